"""The committed profiles belong to the committed code."""
from __future__ import annotations

import bench


def test_the_attention_traffic_figure_is_of_the_present_code():
    """bench.py reports it only under the key of the kernel's and the shared headers' code."""
    n = bench.read_traffic("chunked_hierarchical_sparse_b200/csrc/k_attend_tc.cu")
    assert n is not None and n > 0
