"""Dense attention on the GPU where its calls are at their limits: waits that run out early,
bad values at the edges of tiles, sizes that take the kernels' other paths.  References and
bounds as in test_dense_attention."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_testutil as dt
from test_dense_attention import DEV, cu_of, decode_inputs, f64, hsa, inputs, run_decode, run_prompt

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("L,G,d", [(1, 8, 128), (100, 8, 128), (130, 3, 64), (300, 16, 128), (520, 1, 64)])
def test_waits_that_run_out_with_every_load_issued(L, G, d):
    """Walks of so few tiles that the loaders have issued everything when the other roles give
    up: each call waits for its copies and products, and the calls behind it are right."""
    m = hsa()
    x = inputs(1, L, 2 * G, 2, d, "bf16", seed=L)
    dx = decode_inputs(3, 2 * L, 100, 2 * G, 2, d, "bf16", [100, 0, 7], seed=L)
    good, gd = run_prompt(x), run_decode(dx)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    for _ in range(20):
        codes = []
        m.hsa_set_wait_limit_ns(1)
        try:
            m.hsa_prompt_fwd(x["q"], x["k"], x["v"], ws=ws)
            codes.append(m.hsa_device_status(ws))
            m.hsa_prompt_bwd(x["q"], x["k"], x["v"], good["o"], x["dO"], good["lse"], ws=ws)
            codes.append(m.hsa_device_status(ws))
            m.hsa_prefix_decode(dx["q"], dx["kp"], dx["vp"], dx["kc"], dx["vc"], dx["lens"], ws=ws)
            codes.append(m.hsa_device_status(ws))
        finally:
            m.hsa_set_wait_limit_ns(0)
        assert codes == [5, 5, 5]
        again, gd2 = run_prompt(x), run_decode(dx)
        assert all(torch.equal(good[n], again[n]) for n in good) and torch.equal(gd["o"], gd2["o"])


@pytest.mark.parametrize("L,G,d", [(200, 16, 64), (330, 8, 128), (700, 8, 64)])
def test_sparse_waits_that_run_out_with_few_loads(L, G, d):
    """The same for the sparse forward and backward beside them."""
    m = hsa()
    K = 4
    x = inputs(1, L, 2 * G, 2, d, "bf16", seed=L)
    qs = x["q"][:, :, ::G].contiguous()
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    good = m.hsa_fwd(x["q"], x["k"], x["v"], qs, K)
    gb = m.hsa_bwd(x["q"], x["k"], x["v"], qs, x["dO"], *good[1:], K)
    for _ in range(10):
        m.hsa_set_wait_limit_ns(1)
        try:
            m.hsa_fwd(x["q"], x["k"], x["v"], qs, K, ws=ws)
            codes = [m.hsa_device_status(ws)]
            m.hsa_bwd(x["q"], x["k"], x["v"], qs, x["dO"], *good[1:], K, ws=ws)
            codes.append(m.hsa_device_status(ws))
        finally:
            m.hsa_set_wait_limit_ns(0)
        assert 5 in codes and all(c in (0, 5) for c in codes)
        again = m.hsa_fwd(x["q"], x["k"], x["v"], qs, K, ws=ws)
        assert m.hsa_device_status(ws) == 0
        # its fp16 sums may be taken in another order: one half-step of fp16 per term, K terms
        assert float((again[0].float() - good[0].float()).abs().max()) <= K * 2 ** -8 * float(good[0].abs().max())
        assert torch.equal(again[2], good[2])
        bb = m.hsa_bwd(x["q"], x["k"], x["v"], qs, x["dO"], *good[1:], K, ws=ws)
        assert m.hsa_device_status(ws) == 0
        for a, b in zip(bb, gb):
            assert float((a.float() - b.float()).norm()) <= 2 ** -7 * float(b.float().norm())


# ------------------------------------------------------------ bad values at the edges of tiles
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G", [1, 3, 5, 6, 7, 8, 12, 16])
def test_a_bad_value_reaches_no_further_back_than_documented(G, dtype):
    """NaN in v at the last token of a tile of 128 keys, and one before and behind it: the rows more
    than 127 tokens before it (126 + floor(128 / G) where G does not divide 128) keep their bits."""
    m = hsa()
    x = inputs(1, 700, 2 * G, 2, 64, dtype, seed=G)
    good = m.hsa_prompt_fwd(x["q"], x["k"], x["v"])[0]
    reach = 127 if 128 % G == 0 else 126 + 128 // G
    for t in (254, 255, 256, 383, 511, 639, 699):
        v = x["v"].clone()
        v[0, 1, t] = np.nan
        o, lse = m.hsa_prompt_fwd(x["q"], x["k"], v)
        assert torch.equal(o[:, :, :G], good[:, :, :G])  # the other group
        assert torch.equal(o[:, :max(0, t - reach)], good[:, :max(0, t - reach)]), t
        assert torch.isnan(o[:, t:, G:]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("lens", [[40, 0, 61], [0, 0]])
def test_fp32_backward_leaves_rows_outside_every_prompt_alone(lens):
    """Nothing of the rows before the first and behind the last prompt reaches even the workspace."""
    m = hsa()
    L = 5 + sum(lens) + 7
    x = inputs(1, L, 6, 2, 64, "fp32", seed=50)
    cu = cu_of(lens, 5)
    b = run_prompt(x, cu)
    outside = np.r_[0:5, L - 7:L]
    o, dO, lse = b["o"], x["dO"], b["lse"]
    for t in (o, dO, lse):
        t[:, outside] = np.nan
    ws = torch.full((m.hsa_prompt_workspace_size(1, L, 6, 2, 64, torch.float32, m.OP_BWD, len(lens)) // 4,), 1.0, device=DEV)
    g = m.hsa_prompt_bwd(x["q"], x["k"], x["v"], o, dO, lse, cu, dq=b["dq"].clone(), dk=b["dk"].clone(), dv=b["dv"].clone(), ws=ws)
    assert m.hsa_device_status(ws) == 0
    assert all(torch.equal(a, b[n]) for a, n in zip(g, ("dq", "dk", "dv")))
    assert not torch.isnan(ws).any()
