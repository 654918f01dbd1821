"""Refusals of the binding that need no GPU."""
from __future__ import annotations

import pytest
import torch


def test_device_status_of_host_memory_is_refused_as_a_value():
    import chunked_hierarchical_sparse_b200 as m
    with pytest.raises(ValueError):
        m.hsa_device_status(torch.zeros(256, dtype=torch.uint8))
