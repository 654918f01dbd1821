"""Plain 64-bit dense attention, its gradients, and per-element error bounds.

Bounds (u = 2^-8, half a step of bf16 relative to the value):
  o     the weights p are rounded once to bf16 as an operand, the output once:
        |err| <= u (sum p |v| + |o|)
  dv    likewise                    u (sum p |dO| + |dv|)
  dq    ds = p (dO.v - D) is rounded once as an operand and the output once;
        D = dO . o is taken from the rounded o, off by e_D <= sum |dO| |err o|:
        u (sum |ds| |k| + |dq|) + e_D sum p |k|     (all times 1/sqrt(d))
  dk    likewise over the rows      u (sum |ds| |q| + |dk|) + sum p e_D |q|
  lse   logits are fp32 sums: 1e-5 max(1, max |lse|)
Everything is computed in fp32 besides, with exp and log good to a few 2^-22:
F = 1e-5 of the largest value of the tensor (at least 1) is added, which is also
the whole bound in fp32 (a sum of n products of random sign is off by about
sqrt(n) 2^-24 of its terms; 1e-5 is 168 such steps, for n <= 2048).  The factor
1.02 covers second-order terms (products of two relative roundings).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8


def attend(q, k, v, visible, off_by_one, dO=None):
    """One head: q [n, d], k, v [m, d], visible [n, m].  Returns a dict with o, lse and, given
    dO, dq, dk, dv, each with a bound "<name>_b" of the bf16 error (without F)."""
    d = q.shape[1]
    sc = 1.0 / np.sqrt(d)
    x = np.where(visible, q @ k.T * sc, -np.inf)
    m = x.max(1, initial=-np.inf, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    if off_by_one:
        m = np.maximum(m, 0.0)
    e = np.exp(x - m)
    z = e.sum(1, keepdims=True) + (np.exp(-m) if off_by_one else 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        p = np.where(z > 0, e / z, 0.0)
        lse = (m + np.log(z))[:, 0]
    r = {"o": p @ v, "lse": lse}
    r["o_b"] = U * (p @ np.abs(v) + np.abs(r["o"]))
    r["lse_b"] = np.zeros_like(lse)
    if dO is not None:
        D = (dO * r["o"]).sum(1, keepdims=True)
        eD = (np.abs(dO) * r["o_b"]).sum(1, keepdims=True)
        ds = p * (dO @ v.T - D)
        r["dq"], r["dk"], r["dv"] = ds @ k * sc, ds.T @ q * sc, p.T @ dO
        r["dq_b"] = U * (np.abs(ds) @ np.abs(k) * sc) + eD * (p @ np.abs(k)) * sc
        r["dk_b"] = U * (np.abs(ds).T @ np.abs(q) * sc) + (p * eD).T @ np.abs(q) * sc
        r["dv_b"] = U * (p.T @ np.abs(dO))
    return r


def prompt(q, k, v, spans, off_by_one, dO=None):
    """q, dO [B, L, h_q, d], k, v [B, h_kv, L, d] (fp64); spans [(batch row, first, tokens)].
    Rows outside every span are NaN in the result."""
    B, L, h_q, d = q.shape
    h_kv = k.shape[1]
    G = h_q // h_kv
    out = {}
    for n, shape in (("o", q.shape), ("lse", q.shape[:3]), ("dq", q.shape), ("dk", k.shape), ("dv", k.shape)):
        for s in ("", "_b"):
            out[n + s] = np.full(shape, np.nan)
    for b, t, n in spans:
        i = np.arange(n)
        vis = i[None, :] <= i[:, None]
        ts = slice(t, t + n)
        for nm in ("dk", "dv"):
            out[nm][b, :, ts] = out[nm + "_b"][b, :, ts] = 0.0
        for h in range(h_q):
            g = h // G
            r = attend(q[b, ts, h], k[b, g, ts], v[b, g, ts], vis, off_by_one, None if dO is None else dO[b, ts, h])
            for nm in ("o", "lse", "dq"):
                if nm in r:
                    out[nm][b, ts, h], out[nm + "_b"][b, ts, h] = r[nm], r[nm + "_b"]
            for nm in ("dk", "dv"):
                if nm in r:
                    out[nm][b, g, ts] += r[nm]
                    out[nm + "_b"][b, g, ts] += r[nm + "_b"]
    if dO is not None:
        for nm in ("dq", "dk", "dv"):  # one rounding of the finished gradient
            out[nm + "_b"] += U * np.abs(out[nm])
    return out


def decode(q, kp, vp, kc, vc, lens, off_by_one):
    """q [B, h_q, d], kp, vp [h_kv, P, d], kc, vc [B, h_kv, cap, d] (fp64)."""
    B, h_q, d = q.shape
    G = h_q // kp.shape[0]
    out = {n: np.zeros((B, h_q) + ((d,) if n[0] == "o" else ())) for n in ("o", "o_b", "lse", "lse_b")}
    for b in range(B):
        n = int(lens[b])
        for h in range(h_q):
            g = h // G
            k, v = np.concatenate([kp[g], kc[b, g, :n]]), np.concatenate([vp[g], vc[b, g, :n]])
            r = attend(q[b, h][None], k, v, np.ones((1, len(k)), bool), off_by_one)
            for nm in out:
                out[nm][b, h] = r[nm][0]
    return out


def check(got, ref, name, dtype):
    """got: fp64 array; compares wherever ref is not NaN."""
    want, seen = ref[name], ~np.isnan(ref[name])
    g, w = got[seen], want[seen]
    inf = np.isinf(w)
    assert np.array_equal(g[inf], w[inf]), f"{name}: infinite values differ"
    g, w = g[~inf], w[~inf]
    if not w.size:
        return
    bound = np.full(w.shape, 1e-5 * max(1.0, np.abs(w).max()))
    if dtype == "bf16":
        bound += 1.02 * ref[name + "_b"][seen][~inf]
    err = np.abs(g - w)
    assert np.isfinite(g).all(), f"{name}: {np.count_nonzero(~np.isfinite(g))} values are not finite"
    worst = float((err / bound).max())
    print(f"[dense] {name} ({dtype}, {w.size}): max|err| {err.max():.3e}, at most {worst:.3f} of its bound")
    assert worst <= 1.0, f"{name}: error {err.max():.3e} is {worst:.2f} times its bound"
