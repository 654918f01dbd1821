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


# ------------------------------------------------------------ the kernels' other paths
def plane(x, b, out, g):
    """Batch row b's group g alone: inputs and results of a call."""
    G = x["q"].shape[2] // x["k"].shape[1]
    hs = slice(g * G, (g + 1) * G)
    heads = lambda t: t[b:b + 1, :, hs]
    keys = lambda t: t[b:b + 1, g:g + 1]
    return ({n: heads(x[n]) for n in ("q", "dO")} | {n: keys(x[n]) for n in ("k", "v")},
            {n: heads(out[n]) for n in ("o", "lse", "dq")} | {n: keys(out[n]) for n in ("dk", "dv")})


def check_plane(x, out, b, g, spans, off_by_one, dtype):
    xs, got = plane(x, b, out, g)
    ref = dt.prompt(*(f64(xs[n]) for n in ("q", "k", "v")), spans, off_by_one, f64(xs["dO"]))
    for n in ("o", "lse", "dq", "dk", "dv"):
        dt.check(f64(got[n]), ref, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,L,G,h_kv,d,off_by_one", [(8, 1301, 8, 4, 128, False), (8, 1301, 8, 4, 64, True),
                                                     (11, 1537, 3, 3, 128, True), (20, 900, 1, 4, 64, False)])
def test_prompt_of_many_items(B, L, G, h_kv, d, off_by_one, dtype):
    """Batch rows that fill the GPU: bf16 items of two row tiles, dealt by a counter, and key tiles
    whose rows are not cut, several for every SM; fp32 items of one block each."""
    tt = 128 // G
    rows, steps = -(-L // tt), sum(-(-L // tt) - i * 128 // tt for i in range(-(-L // 128))) * B * h_kv
    # what this test is for: enough pairs of row tiles for every SM, and (the backward's rule) no key tile
    # with more than 9/8 of an SM's share of the steps
    assert B * h_kv * -(-L // (2 * tt)) > 148 and 8 * 148 * rows <= 9 * steps
    x = inputs(B, L, G * h_kv, h_kv, d, dtype, seed=L + G)
    out = run_prompt(x, off_by_one=off_by_one)
    for b, g in ((0, 0), (B // 2, h_kv - 1), (B - 1, 0), (B - 1, h_kv - 1)):
        check_plane(x, out, b, g, [(0, 0, L)], off_by_one, dtype)


@pytest.mark.parametrize("B,L,lens,G,d", [(1, 3000, None, 8, 128), (2, 2049, None, 5, 64),
                                          (1, 3000, [2999, 1], 8, 64), (1, 4100, [1500, 0, 2590], 5, 128)])
def test_prompt_of_cut_key_tiles(B, L, lens, G, d):
    """Key tiles whose rows are walked in pieces, their partials added: every gradient against 64 bits."""
    x = inputs(B, L, 2 * G, 2, d, "bf16", seed=L)
    cu = None if lens is None else cu_of(lens, L - sum(lens))
    spans = [(0, 0, L)] if lens is None else [(0, a, n) for a, n in zip(cu.cpu().tolist(), lens)]
    out = run_prompt(x, cu)
    for b, g in ((0, 1), (B - 1, 0)):
        check_plane(x, out, b, g, spans, False, "bf16")


@pytest.mark.parametrize("L,G,d,off_by_one", [(9001, 4, 128, False), (16384, 2, 64, True)])
def test_prompt_long_against_64_bits(L, G, d, off_by_one):
    """One group of two, all its heads, on the GPU in 64 bits."""
    x = inputs(1, L, 2 * G, 2, d, "bf16", seed=L)
    xs, got = plane(x, 0, run_prompt(x, off_by_one=off_by_one), 1)
    k, v = (xs[n][0, 0].double() for n in ("k", "v"))
    future = torch.ones(L, L, dtype=torch.bool, device=DEV).triu_(1)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    # relative 2-norms.  o, dv: an operand and the output are rounded, 2^-9 rms each at most: 2^-8 in all.
    # dq, dk: dS, D (from the rounded o) and the output: 2^-7
    close = lambda a, b, tol, n: float((a.double() - b).norm() / b.norm()) <= tol or pytest.fail(n)
    for h in range(G):
        q, dO = xs["q"][0, :, h].double(), xs["dO"][0, :, h].double()
        s = (q @ k.T).mul_(d ** -0.5).masked_fill_(future, -np.inf)
        lse = torch.logsumexp(s, 1)
        if off_by_one:
            lse = torch.logaddexp(lse, torch.zeros_like(lse))
        p = s.sub_(lse[:, None]).exp_()
        o = p @ v
        dv += p.T @ dO
        ds = (dO @ v.T).sub_((dO * o).sum(1, keepdim=True)).mul_(p).mul_(d ** -0.5)
        dk += ds.T @ q
        close(got["o"][0, :, h], o, 2 ** -8, "o")
        close(got["dq"][0, :, h], ds @ k, 2 ** -7, "dq")
        assert float((got["lse"][0, :, h].double() - lse).abs().max()) <= 1e-5 * max(1.0, float(lse.abs().max()))
        del s, p, ds
    close(got["dv"][0, 0], dv, 2 ** -8, "dv")
    close(got["dk"][0, 0], dk, 2 ** -7, "dk")


@pytest.mark.parametrize("off_by_one", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [200, 700])
def test_prompt_gradients_of_peaked_rows(L, dtype, off_by_one):
    """Logits of several hundred: one key holds most of a row's weight, and D nearly all of it.

    A logit is a sum of 64 fp32 products of which sum |q_i k_i| / 8 is at most about 1100 here; 64
    additions, each off by at most 2^-23 of the sum so far and of random sign, make 1e-3 of it, and
    the same again for the lse it is compared with: e = 2e-3 is the relative error of a weight, beside
    its rounding U in bf16.  Every bound of the reference is U times a sum that is linear in the
    weights' errors (of o, and through D = dO . o), so e adds e / U of it, in either type."""
    x = inputs(1, L, 4, 1, 64, dtype, seed=60 + L, qscale=30.0)
    x["k"] = x["k"] * (1 + torch.arange(L, device=DEV) / 100).clamp(max=4).to(x["k"].dtype)[None, None, :, None]
    b = run_prompt(x, off_by_one=off_by_one)
    ref = dt.prompt(*(f64(x[n]) for n in ("q", "k", "v")), [(0, 0, L)], off_by_one, f64(x["dO"]))
    assert np.abs(ref["lse"]).max() > 200  # (logits spread by 30 to 120: what the name says of the input)
    for n in ("o", "dq", "dk", "dv"):
        bound = 1e-5 * max(1.0, np.abs(ref[n]).max()) + ((1.02 if dtype == "bf16" else 0.0) + 2e-3 / dt.U) * ref[n + "_b"]
        err = np.abs(f64(b[n]) - ref[n])
        assert np.isfinite(err).all() and (err <= bound).all(), (n, float((err / bound).max()))


@pytest.mark.parametrize("L,lens,G,h_kv,d", [(333, None, 16, 1, 128), (2000, None, 8, 2, 64), (640, [1, 300, 0, 339], 5, 2, 128),
                                             (1500, [700, 800], 1, 4, 64), (257, None, 2, 3, 128)])
def test_many_calls_in_a_row_of_other_shapes(L, lens, G, h_kv, d):
    """As test_many_calls_in_a_row, packed and not, with the decode step in between."""
    m = hsa()
    x = inputs(1, L, G * h_kv, h_kv, d, "bf16", seed=L)
    cu = None if lens is None else cu_of(lens)
    n_seq = 0 if lens is None else len(lens)
    dx = decode_inputs(7, L, 130, G * h_kv, h_kv, d, "bf16", [130, 0, 1, 64, 65, 128, 129], seed=L)
    out = dict(run_prompt(x, cu), od=run_decode(dx)["o"])
    first = {n: t.clone() for n, t in out.items()}
    w = {op: torch.empty(m.hsa_prompt_workspace_size(1, L, G * h_kv, h_kv, d, torch.bfloat16, op, n_seq), dtype=torch.uint8,
                         device=DEV) for op in (m.OP_FWD, m.OP_BWD)}
    w[0] = torch.empty(m.hsa_prefix_workspace_size(7, L, 130, G * h_kv, h_kv, d, torch.bfloat16), dtype=torch.uint8, device=DEV)
    worst = torch.zeros(1, dtype=torch.int32, device=DEV)
    same = torch.ones(1, dtype=torch.bool, device=DEV)
    for i in range(1500):
        m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu, o=out["o"], lse=out["lse"], ws=w[m.OP_FWD])
        m.hsa_prompt_bwd(x["q"], x["k"], x["v"], out["o"], x["dO"], out["lse"], cu, dq=out["dq"], dk=out["dk"], dv=out["dv"],
                         ws=w[m.OP_BWD])
        m.hsa_prefix_decode(dx["q"], dx["kp"], dx["vp"], dx["kc"], dx["vc"], dx["lens"], o=out["od"], ws=w[0])
        for t in w.values():
            torch.maximum(worst, t[:4].view(torch.int32), out=worst)
        if i % 100 == 99:
            for n, t in out.items():
                same &= (t == first[n]).all()
    assert int(worst) == 0 and bool(same)
