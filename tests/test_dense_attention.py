"""Dense attention on the GPU against a plain 64-bit implementation (bounds: dense_testutil)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_testutil as dt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MARK = 77.0  # what the outputs hold before a call


def hsa():
    import chunked_hierarchical_sparse_b200 as m
    m.load_library()
    return m


def tdt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def randn(rng, *shape, dtype, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(DEV, tdt(dtype))


def inputs(B, L, h_q, h_kv, d, dtype, seed=0, qscale=1.0):
    rng = np.random.default_rng(seed)
    return dict(q=randn(rng, B, L, h_q, d, dtype=dtype, scale=qscale), k=randn(rng, B, h_kv, L, d, dtype=dtype),
                v=randn(rng, B, h_kv, L, d, dtype=dtype), dO=randn(rng, B, L, h_q, d, dtype=dtype))


def buffers(x):
    q, k = x["q"], x["k"]
    full = lambda like: torch.full_like(like, MARK)
    return dict(o=full(q), lse=torch.full(q.shape[:3], MARK, dtype=torch.float32, device=DEV), dq=full(q), dk=full(k),
                dv=full(k))


def run_prompt(x, cu=None, off_by_one=False, buf=None):
    m, b = hsa(), buf or buffers(x)
    B, L, h_q, d = x["q"].shape
    n_seq = 0 if cu is None else cu.numel() - 1
    ws = {op: torch.empty(m.hsa_prompt_workspace_size(B, L, h_q, x["k"].shape[1], d, x["q"].dtype, op, n_seq) + 256,
                          dtype=torch.uint8, device=DEV) for op in (m.OP_FWD, m.OP_BWD)}
    ws = {op: w[-w.data_ptr() % 256:] for op, w in ws.items()}
    m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu, off_by_one, o=b["o"], lse=b["lse"], ws=ws[m.OP_FWD])
    m.hsa_prompt_bwd(x["q"], x["k"], x["v"], b["o"], x["dO"], b["lse"], cu, dq=b["dq"], dk=b["dk"], dv=b["dv"],
                     ws=ws[m.OP_BWD])
    assert m.hsa_device_status(ws[m.OP_FWD]) == 0 and m.hsa_device_status(ws[m.OP_BWD]) == 0
    return b


def cu_of(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def spans_of(cu):
    c = cu.cpu().tolist()
    return [(0, a, b - a) for a, b in zip(c, c[1:])]


def check_all(x, b, spans, off_by_one, dtype, names=("o", "lse", "dq", "dk", "dv")):
    ref = dt.prompt(*(f64(x[n]) for n in ("q", "k", "v")), spans, off_by_one, f64(x["dO"]))
    for n in names:
        dt.check(f64(b[n]), ref, n, dtype)
        outside = np.isnan(ref[n])
        assert (f64(b[n])[outside] == MARK).all(), f"{n}: rows outside every prompt were written"


# --------------------------------------------------------------- prompt pass
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [1, 2, 31, 64, 65, 128, 129, 300, 517])
def test_prompt_lengths(L, dtype):
    x = inputs(1, L, 8, 2, 128, dtype, seed=L)
    check_all(x, run_prompt(x), [(0, 0, L)], False, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G,h_kv,d", [(1, 2, 64), (2, 1, 128), (3, 2, 64), (5, 1, 128), (7, 1, 64), (8, 1, 64),
                                      (12, 1, 128), (16, 1, 64), (16, 2, 128)])
def test_prompt_heads(G, h_kv, d, dtype):
    x = inputs(2, 149, G * h_kv, h_kv, d, dtype, seed=G)
    check_all(x, run_prompt(x, off_by_one=G % 2 == 0), [(0, 0, 149), (1, 0, 149)], G % 2 == 0, dtype)


@pytest.mark.parametrize("off_by_one", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,G", [(128, 8), (64, 5)])
def test_prompt_packed(d, G, dtype, off_by_one):
    """Lengths of zero and one, odd ones, rows before the first and behind the last prompt."""
    lens, first, tail = [0, 1, 5, 0, 200, 64, 1, 129, 0], 3, 9
    L = first + sum(lens) + tail
    x = inputs(1, L, G * 2, 2, d, dtype, seed=5)
    for t in ("q", "dO"):
        x[t][:, :first], x[t][:, L - tail:] = np.nan, np.inf
    for t in ("k", "v"):
        x[t][:, :, :first], x[t][:, :, L - tail:] = np.nan, np.nan
    cu = cu_of(lens, first)
    check_all(x, run_prompt(x, cu, off_by_one), spans_of(cu), off_by_one, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_nan_stays_in_its_prompt(dtype):
    lens = [70, 33, 150]
    x = inputs(1, sum(lens), 16, 2, 128, dtype, seed=6)
    for t, s in (("q", np.s_[:, 70:103]), ("dO", np.s_[:, 70:103]), ("k", np.s_[:, :, 70:103]), ("v", np.s_[:, :, 70:103])):
        x[t][s] = np.nan
    cu = cu_of(lens)
    b = run_prompt(x, cu)
    clean = {n: t.clone() for n, t in x.items()}
    for t in ("q", "dO"):
        clean[t][:, 70:103] = 0
    for t in ("k", "v"):
        clean[t][:, :, 70:103] = 0
    ref = dt.prompt(*(f64(clean[n]) for n in ("q", "k", "v")), [s for s in spans_of(cu) if s[1] != 70], False, f64(clean["dO"]))
    for n in ("o", "lse", "dq", "dk", "dv"):
        dt.check(f64(b[n]), ref, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_nan_in_the_future_of_other_tiles(dtype):
    """A bad key at token 400: the rows below 273 stay as they are."""
    x = inputs(1, 500, 8, 1, 128, dtype, seed=7)
    good = run_prompt(x)["o"].clone()
    x["k"][0, 0, 400], x["v"][0, 0, 400] = np.nan, np.inf
    b = run_prompt(x)
    assert torch.equal(b["o"][:, :273], good[:, :273])
    assert torch.isnan(b["o"][:, 400:]).all()


@pytest.mark.parametrize("off_by_one", [False, True])
@pytest.mark.parametrize("qscale", [0.0, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_extreme_logits(dtype, qscale, off_by_one):
    """Logits up to several hundred: the running maximum moves in many tiles; and all equal."""
    x = inputs(1, 400, 4, 1, 64, dtype, seed=8, qscale=qscale)
    x["k"] = x["k"] * (1 + torch.arange(400, device=DEV) / 100).to(x["k"].dtype)[None, None, :, None]
    names = ("o", "lse", "dv") if qscale else ("o", "lse", "dq", "dk", "dv")
    if dtype == "fp32" and qscale:
        # logits near 700 carry 700 * 2^-24 * sqrt(64) = 3e-4 of error each, in the exponent: the
        # weights are off by as much, relatively, so o is held to 1e-3 of max |v| and lse to 1e-3
        ref = dt.prompt(*(f64(x[n]) for n in ("q", "k", "v")), [(0, 0, 400)], off_by_one)
        b = run_prompt(x, off_by_one=off_by_one)
        assert np.abs(f64(b["o"]) - ref["o"]).max() <= 1e-3 * float(x["v"].abs().max())
        assert np.abs(f64(b["lse"]) - ref["lse"]).max() <= 1e-3
        return
    if qscale:
        # bf16 operands are exact in the product, so the same 3e-4 stands beside the 2^-8 of the bound
        ref = dt.prompt(*(f64(x[n]) for n in ("q", "k", "v")), [(0, 0, 400)], off_by_one)
        b = run_prompt(x, off_by_one=off_by_one)
        assert (np.abs(f64(b["o"]) - ref["o"]) <= 1.02 * ref["o_b"] + 1e-3 * float(x["v"].abs().max())).all()
        assert np.abs(f64(b["lse"]) - ref["lse"]).max() <= 1e-3
        return
    check_all(x, run_prompt(x, off_by_one=off_by_one), [(0, 0, 400)], off_by_one, dtype, names)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_very_negative_logits_off_by_one(dtype):
    """exp(-200) beside the added 1: output 0, lse 0, and no NaN in either direction."""
    x = inputs(1, 150, 8, 1, 64, dtype, seed=9)
    x["q"].fill_(5.0)
    x["k"].fill_(-5.0)
    b = run_prompt(x, off_by_one=True)
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert f64(b[n]).any() == False, n  # noqa: E712


def test_prompt_many_prompts():
    """More prompts than a block has threads, most of them of a few tokens."""
    rng = np.random.default_rng(10)
    lens = rng.integers(0, 4, 1500)
    lens[700] = 333
    x = inputs(1, int(lens.sum()), 4, 2, 64, "bf16", seed=10)
    cu = cu_of(lens)
    check_all(x, run_prompt(x, cu), spans_of(cu), False, "bf16")


@pytest.mark.parametrize("bad", [[0, 40, 30, 100], [-1, 40, 50, 100], [0, 40, 50, 101]])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_bad_bounds_are_reported(bad, dtype):
    m = hsa()
    x = inputs(1, 100, 8, 1, 64, dtype)
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    for op in (m.OP_FWD, m.OP_BWD):
        b = buffers(x)
        ws = torch.empty(m.hsa_prompt_workspace_size(1, 100, 8, 1, 64, tdt(dtype), op, 3) + 256, dtype=torch.uint8, device=DEV)
        ws = ws[-ws.data_ptr() % 256:]
        if op == m.OP_FWD:
            m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu, o=b["o"], lse=b["lse"], ws=ws)
        else:
            m.hsa_prompt_bwd(x["q"], x["k"], x["v"], b["o"], x["dO"], b["lse"], cu, dq=b["dq"], dk=b["dk"], dv=b["dv"], ws=ws)
        assert m.hsa_device_status(ws) == 6
        assert all((t == MARK).all() for t in b.values())


def test_waits_that_run_out_are_reported():
    """Every wait bounded by 1 ns: a timeout in the status word, a usable device, a clean next call."""
    m = hsa()
    x = inputs(1, 700, 16, 2, 128, "bf16", seed=21)
    good = run_prompt(x)
    dx = decode_inputs(5, 900, 300, 16, 2, 128, "bf16", [300, 1, 0, 77, 128], seed=22)
    gd = run_decode(dx)
    m.hsa_set_wait_limit_ns(1)
    try:
        codes = []
        b = {n: t.clone() for n, t in good.items()}
        ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
        m.hsa_prompt_fwd(x["q"], x["k"], x["v"], o=b["o"], ws=ws)
        codes.append(m.hsa_device_status(ws))
        m.hsa_prompt_bwd(x["q"], x["k"], x["v"], good["o"], x["dO"], good["lse"], ws=ws)
        codes.append(m.hsa_device_status(ws))
        m.hsa_prefix_decode(dx["q"], dx["kp"], dx["vp"], dx["kc"], dx["vc"], dx["lens"], ws=ws)
        codes.append(m.hsa_device_status(ws))
    finally:
        m.hsa_set_wait_limit_ns(0)
    assert codes == [5, 5, 5]
    again = run_prompt(x)
    assert all(torch.equal(good[n], again[n]) for n in good)
    assert torch.equal(gd["o"], run_decode(dx)["o"])


def test_prompt_empty():
    m = hsa()
    for B, L in ((0, 5), (2, 0)):
        q, k = torch.empty(B, L, 4, 64, device=DEV), torch.empty(B, 2, L, 64, device=DEV)
        o, lse = m.hsa_prompt_fwd(q, k, k)
        dq, dk, dv = m.hsa_prompt_bwd(q, k, k, o, q, lse)
        assert o.shape == q.shape and lse.shape == (B, L, 4) and dq.shape == q.shape and dk.shape == dv.shape == k.shape
    q, k = torch.empty(1, 0, 4, 64, device=DEV), torch.empty(1, 2, 0, 64, device=DEV)
    m.hsa_prompt_fwd(q, k, k, torch.zeros(4, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_same_bits_every_call(dtype):
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 300, 12)
    x = inputs(1, int(lens.sum()), 16, 2, 128, dtype, seed=11)
    cu = cu_of(lens)
    a = run_prompt(x, cu)
    for _ in range(3):
        b = run_prompt(x, cu)
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_prompt_gradients_against_differences():
    """fp32: the loss moved along a random direction, the op's own forward on both sides."""
    m = hsa()
    x = inputs(1, 90, 6, 2, 64, "fp32", seed=12)
    cu = cu_of([50, 40])
    b = run_prompt(x, cu, True)
    rng = np.random.default_rng(13)
    for n in ("q", "k", "v"):
        u = randn(rng, *x[n].shape, dtype="fp32")
        loss = []
        for s in (1, -1):
            y = dict(x)
            y[n] = x[n] + s * 1e-2 * u
            o, _ = m.hsa_prompt_fwd(y["q"], y["k"], y["v"], cu, True)
            loss.append(float((f64(o) * f64(x["dO"])).sum()))
        got, want = float((f64(b["d" + n]) * f64(u)).sum()), (loss[0] - loss[1]) / 2e-2
        # 90*6*64 outputs of size 1, each off by up to 1e-6 (rounding) over 2e-2: sqrt(35e3) * 1e-6 / 2e-2
        # = 0.01; third derivatives: 1e-4 of the change
        assert abs(got - want) <= 0.02 + 1e-3 * abs(want), n


def test_prompt_on_a_side_stream_and_in_graphs():
    """Two captured graphs with their own workspaces, replayed interleaved on new inputs."""
    m = hsa()
    cu = cu_of([60, 1, 139])
    x = inputs(1, 200, 8, 2, 64, "bf16", seed=14)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu, stream=side)
    g = m.hsa_prompt_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, cu, stream=side)
    side.synchronize()
    ref = run_prompt(x, cu)
    assert torch.equal(o, ref["o"]) and all(torch.equal(a, ref[n]) for a, n in zip(g, ("dq", "dk", "dv")))
    graphs = []
    for _ in range(2):
        st = {n: t.clone() for n, t in x.items()}
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o, lse = m.hsa_prompt_fwd(st["q"], st["k"], st["v"], cu)
            out = (o, *m.hsa_prompt_bwd(st["q"], st["k"], st["v"], o, st["dO"], lse, cu))
        graphs.append((gr, st, out))
    for seed in (15, 16):
        xs = [inputs(1, 200, 8, 2, 64, "bf16", seed=seed + 10 * i) for i in range(2)]
        for (gr, st, _), y in zip(graphs, xs):
            for n in st:
                st[n].copy_(y[n])
        for gr, _, _ in graphs:
            gr.replay()
        for (_, _, out), y in zip(graphs, xs):
            r = run_prompt(y, cu)
            assert all(torch.equal(a, r[n]) for a, n in zip(out, ("o", "dq", "dk", "dv")))


# ------------------------------------------------------- shared-prefix decode
def decode_inputs(B, P, cap, h_q, h_kv, d, dtype, lens, room=0, seed=0):
    rng = np.random.default_rng(seed)
    x = dict(q=randn(rng, B, h_q, d, dtype=dtype), kp=randn(rng, h_kv, P + room, d, dtype=dtype),
             vp=randn(rng, h_kv, P + room, d, dtype=dtype), kc=randn(rng, B, h_kv, cap, d, dtype=dtype),
             vc=randn(rng, B, h_kv, cap, d, dtype=dtype), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    x["kp"][:, P:] = np.nan  # memory that is not the prefix's
    x["vp"][:, P:] = np.nan
    for b, n in enumerate(lens):
        x["kc"][b, :, n:] = np.nan
        x["vc"][b, :, n:] = np.inf
    x["kp"], x["vp"] = x["kp"][:, :P], x["vp"][:, :P]
    return x


def run_decode(x, off_by_one=False, status=0):
    m = hsa()
    B, h_q, d = x["q"].shape
    h_kv, P, cap = x["kp"].shape[0], x["kp"].shape[1], x["kc"].shape[2]
    ws = torch.empty(m.hsa_prefix_workspace_size(B, P, cap, h_q, h_kv, d, x["q"].dtype) + 256, dtype=torch.uint8, device=DEV)
    ws = ws[-ws.data_ptr() % 256:]
    o, lse = m.hsa_prefix_decode(x["q"], x["kp"], x["vp"], x["kc"], x["vc"], x["lens"], off_by_one, ws=ws)
    assert m.hsa_device_status(ws) == status
    return {"o": o, "lse": lse}


def check_decode(x, r, off_by_one, dtype, lens=None):
    lens = x["lens"].cpu().tolist() if lens is None else lens
    z = {n: np.nan_to_num(f64(x[n]), posinf=0.0) for n in ("kc", "vc")}
    ref = dt.decode(f64(x["q"]), f64(x["kp"]), f64(x["vp"]), z["kc"], z["vc"], lens, off_by_one)
    for n in ("o", "lse"):
        dt.check(f64(r[n]), ref, n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,P,cap,lens", [
    (1, 0, 1, [1]), (1, 1, 1, [0]), (2, 0, 5, [0, 5]), (3, 64, 130, [0, 1, 130]), (5, 129, 64, [64, 63, 0, 1, 7]),
    (17, 300, 40, list(range(17))), (20, 1000, 257, [257, 256, 255, 128, 129] * 4), (3, 700, 0, [0, 0, 0]),
    (33, 513, 12, [i % 13 for i in range(33)])])
def test_decode(B, P, cap, lens, dtype):
    for off_by_one in (False, True):
        x = decode_inputs(B, P, cap, 16, 2, 128, dtype, lens, room=3 * (P % 2), seed=B + P)
        check_decode(x, run_decode(x, off_by_one), off_by_one, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("G,h_kv,d", [(1, 3, 64), (3, 2, 128), (5, 1, 64), (7, 2, 64), (8, 4, 128), (12, 1, 64), (16, 1, 128)])
def test_decode_heads(G, h_kv, d, dtype):
    lens = [0, 3, 150, 77, 149, 1, 150, 12, 64, 65, 2]
    x = decode_inputs(11, 333, 150, G * h_kv, h_kv, d, dtype, lens, room=11, seed=G)
    check_decode(x, run_decode(x), False, dtype)


def test_decode_no_keys_at_all():
    x = decode_inputs(2, 0, 4, 8, 2, 64, "bf16", [0, 2])
    r = run_decode(x)
    assert (r["o"][0] == 0).all() and (r["lse"][0] == -np.inf).all()
    r = run_decode(x, True)
    assert (r["o"][0] == 0).all() and (r["lse"][0] == 0).all()
    x = decode_inputs(2, 0, 0, 8, 2, 64, "fp32", [0, 0])
    r = run_decode(x)
    assert (r["o"] == 0).all() and (r["lse"] == -np.inf).all()
    m = hsa()
    e = torch.empty(0, 8, 64, device=DEV)
    assert m.hsa_prefix_decode(e, x["kp"], x["vp"], x["kc"][:0], x["vc"][:0], x["lens"][:0])[0].shape == e.shape


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_bad_lengths_are_reported(dtype):
    x = decode_inputs(3, 70, 20, 8, 1, 64, dtype, [20, 0, 5])
    x["lens"].copy_(torch.tensor([25, -3, 5]))
    check_decode(x, run_decode(x, status=6), False, dtype, lens=[20, 0, 5])


def test_decode_cache_beyond_32_bit_offsets():
    """The last sequence's cache begins 2^31 elements into the buffer."""
    B, cap, d = 9, 1 << 21, 128
    x = dict(q=randn(np.random.default_rng(1), B, 4, d, dtype="bf16"), kp=randn(np.random.default_rng(2), 1, 100, d, dtype="bf16"),
             vp=randn(np.random.default_rng(3), 1, 100, d, dtype="bf16"),
             kc=torch.zeros(B, 1, cap, d, dtype=torch.bfloat16, device=DEV))
    x["vc"] = torch.zeros_like(x["kc"])
    tail = randn(np.random.default_rng(4), B, 1, 50, d, dtype="bf16")
    x["kc"][:, :, :50], x["vc"][:, :, :50] = tail, tail.flip(2)
    x["lens"] = torch.full((B,), 50, dtype=torch.int32, device=DEV)
    r = run_decode(x)
    small = {**x, "kc": x["kc"][:, :, :50].contiguous(), "vc": x["vc"][:, :, :50].contiguous()}
    check_decode(small, r, False, "bf16")
    # and a whole cache of equal keys behind the prefix: its mean value
    x["kc"].zero_()
    x["vc"].fill_(0.5)
    x["lens"][:] = torch.tensor([1] * (B - 1) + [cap], dtype=torch.int32)
    r = run_decode(x)
    w = np.exp(f64(x["q"])[-1] @ f64(x["kp"])[0].T / np.sqrt(d))
    want = (w @ f64(x["vp"])[0] + 0.5 * cap) / (w.sum(1, keepdims=True) + cap)
    assert np.abs(f64(r["o"])[-1] - want).max() <= 2.0 ** -8 * 1.1


def test_decode_same_bits_and_graph():
    m = hsa()
    x = decode_inputs(6, 900, 200, 16, 2, 128, "bf16", [0, 200, 13, 64, 199, 128], seed=3)
    a = run_decode(x)
    for _ in range(3):
        assert torch.equal(a["o"], run_decode(x)["o"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = m.hsa_prefix_decode(x["q"], x["kp"], x["vp"], x["kc"], x["vc"], x["lens"])
    x["q"].mul_(0.5)
    x["lens"].copy_(torch.tensor([5, 0, 13, 64, 100, 128]))
    for n in ("kc", "vc"):  # longer by design: values for the tokens that joined
        x[n][0, :, :5] = 0.25
    g.replay()
    r = run_decode(x)
    assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])


# --------------------------------------------------------------- as they are used
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_then_decode(dtype):
    """A prompt's own k and v serve as the prefix: decoding its last tokens one by one gives the
    rows that the prompt pass gives, and the sparse forward runs on the same tensors."""
    m = hsa()
    T, P, h_q, h_kv, d = 420, 384, 16, 2, 128
    x = inputs(1, T, h_q, h_kv, d, dtype, seed=20)
    o, lse = m.hsa_prompt_fwd(x["q"], x["k"], x["v"])
    oracle = dt.prompt(*(f64(x[n]) for n in ("q", "k", "v")), [(0, 0, T)], False)
    dt.check(f64(o), oracle, "o", dtype)
    sparse = m.hsa_fwd(x["q"], x["k"], x["v"], x["q"][:, :, ::8].contiguous(), 4)[0]
    assert sparse.shape == o.shape and torch.isfinite(sparse).all()
    n = T - P  # the sequences of the batch are the same text at different lengths
    kc = x["k"][:, :, P:].expand(n, -1, -1, -1).contiguous()
    vc = x["v"][:, :, P:].expand(n, -1, -1, -1).contiguous()
    lens = torch.arange(1, n + 1, dtype=torch.int32, device=DEV)
    od, ld = m.hsa_prefix_decode(x["q"][0, P:].contiguous(), x["k"][0, :, :P], x["v"][0, :, :P], kc, vc, lens)
    ref = {k_: oracle[k_][0, P:] for k_ in ("o", "o_b", "lse", "lse_b")}
    dt.check(f64(od), ref, "o", dtype)
    dt.check(f64(ld), ref, "lse", dtype)


# ------------------------------------------------------------- calls side by side
def test_two_streams_at_once():
    """Prompt passes and decode steps issued on two streams without waiting in between."""
    m = hsa()
    xs = [inputs(1, 900 + 100 * i, 16, 2, 128, "bf16", seed=30 + i) for i in range(2)]
    ds = [decode_inputs(9, 700 + i, 150, 16, 2, 128, "bf16", [150, 0, 3, 149, 64, 65, 1, 2, 150], seed=32 + i) for i in range(2)]
    want = [run_prompt(x) for x in xs]
    wantd = [run_decode(d) for d in ds]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            x, d = xs[i], ds[i]
            o, lse = m.hsa_prompt_fwd(x["q"], x["k"], x["v"], stream=st)
            g = m.hsa_prompt_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, stream=st)
            od, _ = m.hsa_prefix_decode(d["q"], d["kp"], d["vp"], d["kc"], d["vc"], d["lens"], stream=st)
            got[i].append((o, *g, od))
    torch.cuda.synchronize()
    for i in range(2):
        for o, dq, dk, dv, od in got[i]:
            w = want[i]
            assert all(torch.equal(a, w[n]) for a, n in ((o, "o"), (dq, "dq"), (dk, "dk"), (dv, "dv")))
            assert torch.equal(od, wantd[i]["o"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_workspace_for_calls_of_different_sizes(dtype):
    """What a call left in the workspace does not matter to the next."""
    m = hsa()
    ws = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    for L, G, seed in ((700, 8, 40), (33, 3, 41), (512, 1, 42)):
        x = inputs(1, L, 2 * G, 2, 64, dtype, seed=seed)
        cu = cu_of([L // 3, 0, L - L // 3])
        want = run_prompt(x, cu)
        ws.random_(0, 255)
        o, lse = m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu, ws=ws)
        ws.random_(0, 255)
        g = m.hsa_prompt_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, cu, ws=ws)
        assert torch.equal(o, want["o"]) and all(torch.equal(a, want[n]) for a, n in zip(g, ("dq", "dk", "dv")))
        d = decode_inputs(5, L, 40, 2 * G, 2, 64, dtype, [40, 1, 0, 39, 7], seed=seed)
        wd = run_decode(d)
        ws.random_(0, 255)
        assert torch.equal(m.hsa_prefix_decode(d["q"], d["kp"], d["vp"], d["kc"], d["vc"], d["lens"], ws=ws)[0], wd["o"])


@pytest.mark.parametrize("L,n_seq", [(3000, 1), (5000, 3), (2600, 40)])
def test_prompt_long_and_packed_cut(L, n_seq):
    """Sizes at which streams split the keys and key tiles are cut into pieces, against fp64 on the GPU
    for one head and, for the rest, against the same prompts computed one at a time."""
    rng = np.random.default_rng(L)
    ends = np.sort(rng.integers(0, L + 1, n_seq - 1))
    lens = np.diff(np.concatenate([[0], ends, [L]]))
    x = inputs(1, L, 10, 2, 128, "bf16", seed=L)
    cu = cu_of(lens)
    b = run_prompt(x, cu, True)
    for _, t, n in spans_of(cu):
        if n == 0:
            continue
        ts = slice(t, t + n)
        one = {nm: x[nm][:, ts].contiguous() for nm in ("q", "dO")} | {nm: x[nm][:, :, ts].contiguous() for nm in ("k", "v")}
        r = run_prompt(one, None, True)
        # the same sums in another grouping: fp32 sums of bf16 products, so a rounding of the output
        # (2^-8 of it, both sides) and of the operands p and dS (2^-8 of a sum's terms each side)
        for nm, sl in (("o", np.s_[:, ts]), ("dq", np.s_[:, ts]), ("dk", np.s_[:, :, ts]), ("dv", np.s_[:, :, ts])):
            u, w = b[nm][sl].double(), r[nm].double()
            assert float((u - w).norm() / w.norm()) <= 2 ** -8, nm
    q, k, v, dO = (x[nm].double() for nm in ("q", "k", "v", "dO"))
    h, g = 7, 1  # one head of the second group
    o = torch.zeros(L, 128, dtype=torch.float64, device=DEV)
    dq = torch.zeros_like(o)
    for _, t, n in spans_of(cu):
        ts = slice(t, t + n)
        s = (q[0, ts, h] @ k[0, g, ts].T) / 128 ** 0.5
        s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu(1), -np.inf)
        p = torch.exp(s) / (1 + torch.exp(s).sum(1, keepdim=True))
        o[ts] = p @ v[0, g, ts]
        dp = dO[0, ts, h] @ v[0, g, ts].T
        dq[ts] = (p * (dp - (dO[0, ts, h] * o[ts]).sum(1, keepdim=True))) @ k[0, g, ts] / 128 ** 0.5
    # relative 2-norms: p and the output are rounded (2^-9 rms at most each): 2^-8; dS, dq and D: 2^-7
    assert float((b["o"][0, :, h].double() - o).norm() / o.norm()) <= 2 ** -8
    assert float((b["dq"][0, :, h].double() - dq).norm() / dq.norm()) <= 2 ** -7


def test_prompt_strided_views_are_refused():
    m = hsa()
    x = inputs(1, 64, 8, 2, 64, "bf16")
    with pytest.raises(ValueError):
        m.hsa_prompt_fwd(x["q"].transpose(1, 2), x["k"], x["v"])
    with pytest.raises(ValueError):
        m.hsa_prompt_fwd(x["q"], x["k"].transpose(2, 3).contiguous().transpose(2, 3), x["v"])
    d = decode_inputs(2, 64, 8, 8, 2, 64, "bf16", [8, 8])
    with pytest.raises(m.HsaError):  # planes that overlap
        m.hsa_prefix_decode(d["q"], d["kp"][:1].expand(2, -1, -1), d["vp"][:1].expand(2, -1, -1), d["kc"], d["vc"], d["lens"])
    with pytest.raises(ValueError):
        m.hsa_prefix_decode(d["q"], d["kp"][:, ::2], d["vp"][:, ::2], d["kc"], d["vc"], d["lens"])
    with pytest.raises(TypeError):
        m.hsa_prefix_decode(d["q"], d["kp"], d["vp"], d["kc"], d["vc"], d["lens"].long())


def test_missing_tensors_are_refused():
    m = hsa()
    x = inputs(1, 64, 8, 2, 64, "bf16")
    with pytest.raises(TypeError):
        m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu_seqlens=[0, 64])
    with pytest.raises(TypeError):
        m.hsa_prompt_fwd(x["q"], x["k"], None)
    with pytest.raises(TypeError):
        m.hsa_prompt_bwd(x["q"], x["k"], x["v"], x["q"], x["dO"], None)
    d = decode_inputs(2, 64, 8, 8, 2, 64, "bf16", [8, 8])
    with pytest.raises(ValueError):
        m.hsa_prefix_decode(d["q"], d["kp"], None, d["kc"], d["vc"], d["lens"])
    with pytest.raises(TypeError):
        m.hsa_prefix_decode(d["q"], d["kp"], d["vp"], d["kc"], d["vc"], None)


@pytest.mark.parametrize("d", [64, 128])
def test_many_calls_in_a_row(d):
    """No wait of a kernel may depend on how fast its roles run beside one another: thousands
    of calls, queued without a pause, report nothing and give the same bits."""
    m = hsa()
    x = inputs(1, 889, 6, 3, d, "bf16", seed=d)
    b = buffers(x)
    ws = {op: torch.empty(m.hsa_prompt_workspace_size(1, 889, 6, 3, d, torch.bfloat16, op), dtype=torch.uint8, device=DEV)
          for op in (m.OP_FWD, m.OP_BWD)}
    worst, first = torch.zeros(1, dtype=torch.int32, device=DEV), None
    for i in range(4000):
        m.hsa_prompt_fwd(x["q"], x["k"], x["v"], o=b["o"], lse=b["lse"], ws=ws[m.OP_FWD])
        m.hsa_prompt_bwd(x["q"], x["k"], x["v"], b["o"], x["dO"], b["lse"], dq=b["dq"], dk=b["dk"], dv=b["dv"],
                         ws=ws[m.OP_BWD])
        for w in ws.values():
            torch.maximum(worst, w[:4].view(torch.int32), out=worst)
        if i == 0:
            first = {n: t.clone() for n, t in b.items()}
    assert int(worst) == 0
    for n, t in b.items():
        assert torch.equal(t, first[n]), n
