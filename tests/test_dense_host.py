"""Dense attention without a GPU: refusals of the C ABI and of the binding, and the
64-bit reference's gradients against differences."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import dense_testutil as dt


@pytest.fixture(scope="module")
def lib():
    from chunked_hierarchical_sparse_b200 import build, load_library
    build.build()
    return load_library()


P = ctypes.c_void_p
GOOD, ODD, WS = P(1 << 20), P((1 << 20) + 8), P(1 << 24)


def _prompt_shape(**kw):
    from chunked_hierarchical_sparse_b200 import HsaPromptShape
    d = dict(B=1, L=512, h_q=16, h_kv=2, d=128, n_seq=0, off_by_one=0, dtype=1)
    d.update(kw)
    return HsaPromptShape(**d)


def _prefix_shape(**kw):
    from chunked_hierarchical_sparse_b200 import HsaPrefixShape
    d = dict(B=4, P=512, cap=64, h_q=16, h_kv=2, d=128, off_by_one=0, dtype=1, prefix_stride=512 * 128)
    d.update(kw)
    return HsaPrefixShape(**d)


def _fwd(lib, sh, q=GOOD, k=GOOD, v=GOOD, cu=None, o=GOOD, lse=GOOD, ws=WS, n=1 << 30):
    return lib.hsa_prompt_fwd(ctypes.byref(sh) if sh is not None else None, q, k, v, cu, o, lse, ws, n, None)


def _bwd(lib, sh, q=GOOD, k=GOOD, v=GOOD, o=GOOD, dO=GOOD, lse=GOOD, cu=None, dq=GOOD, dk=GOOD, dv=GOOD, ws=WS, n=1 << 30):
    return lib.hsa_prompt_bwd(ctypes.byref(sh), q, k, v, o, dO, lse, cu, dq, dk, dv, ws, n, None)


def _dec(lib, sh, q=GOOD, kp=GOOD, vp=GOOD, kc=GOOD, vc=GOOD, lens=GOOD, o=GOOD, lse=GOOD, ws=WS, n=1 << 30):
    return lib.hsa_prefix_decode(ctypes.byref(sh), q, kp, vp, kc, vc, lens, o, lse, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(L=-1), 1), (dict(h_q=0), 1), (dict(h_kv=0), 1), (dict(h_q=15), 1), (dict(d=0), 1),
    (dict(dtype=2), 1), (dict(off_by_one=2), 1), (dict(n_seq=-1), 1), (dict(d=96), 2), (dict(h_q=34), 2),
    (dict(B=1 << 15, L=1 << 15), 2)])
def test_prompt_shapes_refused(lib, kw, code):
    sh = _prompt_shape(**kw)
    assert _fwd(lib, sh) == code
    assert _bwd(lib, sh) == code
    for op in (2, 4):
        assert lib.hsa_prompt_workspace_size(ctypes.byref(sh), op) == 0


def test_prompt_arguments_refused(lib):
    sh = _prompt_shape()
    assert _fwd(lib, None) == 1
    for name in ("q", "k", "v", "o"):
        assert _fwd(lib, sh, **{name: None}) == 1 and _fwd(lib, sh, **{name: ODD}) == 1, name
    assert _fwd(lib, sh, lse=ODD) == 1
    for name in ("q", "k", "v", "o", "dO", "lse", "dq", "dk", "dv"):
        assert _bwd(lib, sh, **{name: None}) == 1 and _bwd(lib, sh, **{name: ODD}) == 1, name
    # cu_seqlens and n_seq go together; packing needs B = 1
    assert _fwd(lib, sh, cu=GOOD) == 1
    assert _fwd(lib, _prompt_shape(n_seq=3)) == 1
    assert _fwd(lib, _prompt_shape(n_seq=3, B=2), cu=GOOD) == 1
    assert _fwd(lib, _prompt_shape(n_seq=3), cu=P((1 << 20) + 2)) == 1
    # workspace: missing, misaligned, too small
    assert _fwd(lib, sh, ws=None) == 1 and _fwd(lib, sh, ws=P((1 << 24) + 16)) == 1
    assert _fwd(lib, sh, n=255) == 3
    need = lib.hsa_prompt_workspace_size(ctypes.byref(sh), 4)
    assert need > lib.hsa_prompt_workspace_size(ctypes.byref(sh), 2) >= 256
    assert _bwd(lib, sh, n=need - 1) == 3
    assert lib.hsa_prompt_workspace_size(ctypes.byref(sh), 3) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(P=-1), 1), (dict(cap=-1), 1), (dict(h_q=15), 1), (dict(dtype=3), 1),
    (dict(off_by_one=-1), 1), (dict(prefix_stride=511 * 128), 1), (dict(prefix_stride=512 * 128 + 4), 1),
    (dict(d=32), 2), (dict(h_q=34), 2), (dict(P=1 << 30, prefix_stride=1 << 40), 2)])
def test_prefix_shapes_refused(lib, kw, code):
    sh = _prefix_shape(**kw)
    assert _dec(lib, sh) == code
    assert lib.hsa_prefix_workspace_size(ctypes.byref(sh)) == 0


def test_prefix_arguments_refused(lib):
    sh = _prefix_shape()
    for name in ("q", "kp", "vp", "kc", "vc", "o"):
        assert _dec(lib, sh, **{name: None}) == 1 and _dec(lib, sh, **{name: ODD}) == 1, name
    assert _dec(lib, sh, lens=None) == 1 and _dec(lib, sh, lens=P((1 << 20) + 1)) == 1
    assert _dec(lib, sh, lse=ODD) == 1 and _dec(lib, sh, ws=None) == 1
    assert _dec(lib, sh, n=lib.hsa_prefix_workspace_size(ctypes.byref(sh)) - 1) == 3


def test_binding_refuses_wrong_tensors():
    import chunked_hierarchical_sparse_b200 as m
    q, k = torch.zeros(1, 8, 4, 64), torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError):
        m.hsa_prompt_fwd(q, k, k)              # not on a GPU
    with pytest.raises(ValueError):
        m.hsa_prompt_fwd(q[0], k, k)
    with pytest.raises(TypeError):
        m.hsa_prompt_fwd(q.half(), k.half(), k.half())
    with pytest.raises(ValueError):
        m.hsa_prefix_decode(q[:, 0], k[0], k[0], k, k[:, :1], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        m.hsa_prefix_decode(q, k[0], k[0], k, k, torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("off_by_one", [False, True])
def test_reference_gradients_are_differences(off_by_one):
    rng = np.random.default_rng(3)
    n, d = 7, 8
    x = {c: rng.standard_normal((n, d)) for c in "qkv"}
    dO = rng.standard_normal((n, d))
    vis = np.tril(np.ones((n, n), bool))
    r = dt.attend(x["q"], x["k"], x["v"], vis, off_by_one, dO)
    f = lambda: float((dO * dt.attend(x["q"], x["k"], x["v"], vis, off_by_one)["o"]).sum())
    eps = 1e-5
    for c in "qkv":
        for i in range(n):
            for j in range(d):
                x[c][i, j] += eps
                up = f()
                x[c][i, j] -= 2 * eps
                dn = f()
                x[c][i, j] += eps
                assert abs((up - dn) / (2 * eps) - r["d" + c][i, j]) < 1e-7
