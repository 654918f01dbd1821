"""What is measured of the dense attention operators, and their plain forms.

Three operators stand beside the sparse ones of this library, in its layouts
(q, o [B, L, h_q, d]; k, v [B, h_kv, L, d]; group g serves the heads
g*G .. g*G + G-1, G = h_q / h_kv; logits x = q . k / sqrt(d)):

  prompt   causal attention over whole prompts, one per batch row or several
           packed behind one another (cu_seqlens):
           o_t = sum_{j <= t} e^{x_tj} v_j / Z_t, lse_t = log Z_t,
           Z_t = [1 +] sum_{j <= t} e^{x_tj}   (the 1: softmax-off-by-one)
  train    the same and its gradients of sum(dO * o):
           p_tj = e^{x_tj - lse_t}, D_t = dO_t . o_t, s_tj = p_tj (dO_t . v_j - D_t),
           dq_t = sum_j s_tj k_j / sqrt(d), dk_j = sum s_tj q_t / sqrt(d) and
           dv_j = sum p_tj dO_t, both over the tokens and heads that read j
  decode   one new token per sequence; every sequence has the same first P
           tokens (the prefix, stored once) and lens[b] tokens of its own

A case is one call (train: the forward and the backward) with its sizes.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda:0"


# --------------------------------------------------------------------- cases
def _prompt(name, kind, B, L, h_q, h_kv, d, dtype="bf16", off_by_one=False, n_seq=0, cut=0):
    """n_seq = 0: each batch row is one prompt; else n_seq prompts whose ends are drawn from `cut`."""
    c = dict(kind=kind, B=B, L=L, h_q=h_q, h_kv=h_kv, d=d, dtype=dtype, off_by_one=off_by_one, n_seq=n_seq, cut=cut)
    return dict(name=name, **c) if name else c


def _decode(name, B, P, cap, h_q, h_kv, d, dtype="bf16", off_by_one=False, room=0, cut=0):
    """cap: tokens a sequence's own cache can hold; room: unused tokens behind the prefix in its buffer."""
    c = dict(kind="decode", B=B, P=P, cap=cap, h_q=h_q, h_kv=h_kv, d=d, dtype=dtype, off_by_one=off_by_one,
             room=room, cut=cut)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # a handful of very short prompts that arrive together: latency is all that counts
        _prompt("prompt-short", "prompt", 1, 64, 16, 2, 128, n_seq=3, cut=5),
        # a serving batch's prompts packed to 16K tokens, ragged, single tokens among them
        _prompt("prompt-packed-16k", "prompt", 1, 16384, 16, 2, 128, n_seq=13, cut=11),
        # the benchmark's long context: one prompt of 64K tokens
        _prompt("prompt-64k", "prompt", 1, 65536, 16, 2, 128),
        # the small full-precision workload of the tests
        _prompt("prompt-fp32", "prompt", 1, 1024, 4, 1, 64, dtype="fp32", off_by_one=True),
        # a short packed fine-tuning batch, head dimension 64
        _prompt("train-short", "train", 1, 777, 8, 2, 64, off_by_one=True, n_seq=5, cut=3),
        # the training workload of the benchmark: four sequences of 16K tokens
        _prompt("train-16k", "train", 4, 16384, 16, 2, 128),
        # documents packed for training, with a head count that divides nothing evenly
        _prompt("train-packed-odd", "train", 1, 6001, 15, 3, 128, n_seq=9, cut=7),
        # a gradient check in full precision
        _prompt("train-fp32", "train", 2, 500, 4, 2, 64, dtype="fp32"),
        # a few users behind a short system prompt, just started
        _decode("decode-small", 3, 100, 16, 16, 2, 128, cut=1),
        # the decode workload of the benchmark (16 sequences, 16K tokens) with the context shared
        _decode("decode-16k", 16, 16384, 512, 16, 2, 128, room=64, cut=2),
        # many samples of one long document
        _decode("decode-256", 256, 32768, 2048, 16, 2, 128, cut=3),
        # full precision, off-by-one
        _decode("decode-fp32", 5, 1000, 64, 4, 2, 64, dtype="fp32", off_by_one=True, cut=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "train", "decode"])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    h_kv, G, d = rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), rng.choice([64, 128])
    sink, cut, h_q = rng.random() < 0.4, rng.randrange(1 << 20), h_kv * G
    if kind == "decode":
        B = _log(rng, 1, 256)
        P = 0 if rng.random() < 0.1 else _log(rng, 1, 4096 if dtype == "fp32" else 32768)
        cap = _log(rng, 1, max(2, min(8192, (2048 * 256) // B)) if dtype == "bf16" else 512)
        while B * cap * h_kv > 256 * 2048 * 2 or h_q * B * (P + cap) > 16 * 256 * (32768 + 1024):
            cap = max(1, cap // 2)
            P //= 2
        return _decode(None, B, P, cap, h_q, h_kv, d, dtype, sink, rng.choice([0, 0, 1, 77]), cut)
    top = 2048 if dtype == "fp32" else (16384 if kind == "train" else 65536)
    B, L = (1, _log(rng, 1, top)) if rng.random() < 0.6 else (rng.choice([2, 3, 4]), _log(rng, 1, top // 4))
    n_seq = 0 if B > 1 or rng.random() < 0.3 else _log(rng, 1, 40)
    # no dearer than the largest listed case of its kind (whole rows: an upper bound for packed ones)
    budget = (1 << 34) if kind == "train" else (1 << 36)
    while B * h_q * L * L > budget:
        L = (L * 2) // 3
    return _prompt(None, kind, B, L, h_q, h_kv, d, dtype, sink, n_seq, cut)


def _spans(c):
    """[(batch row, first token, tokens)] of a prompt case's sequences."""
    if not c["n_seq"]:
        return [(b, 0, c["L"]) for b in range(c["B"])]
    r = random.Random(c["cut"])
    ends = sorted(r.randrange(c["L"] + 1) for _ in range(c["n_seq"] - 1))
    cu = [0] + ends + [c["L"]]
    if c["n_seq"] > 2:  # one prompt of a single token
        cu[1] = min(1, cu[2])
    return [(0, a, b - a) for a, b in zip(cu, cu[1:])]


def _lens(c):
    """Tokens of their own that the sequences of a decode case hold (0 to cap)."""
    r = random.Random(c["cut"])
    lens = [r.randint(0, c["cap"]) for _ in range(c["B"])]
    lens[-1] = c["cap"]
    return lens


# -------------------------------------------------------------------- inputs
def _dt(c):
    return torch.float32 if c["dtype"] == "fp32" else torch.bfloat16


def _normal(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _keys(gen, planes, n, d, dtype):
    """Keys ~ N(0, 1) plus one N(0, 0.5^2) offset vector per 64 of them: neighbours are alike."""
    k = torch.randn(planes, n, d, generator=gen, device=DEV)
    off = 0.5 * torch.randn(planes, (n + 63) // 64, d, generator=gen, device=DEV)
    return (k + off.repeat_interleave(64, 1)[:, :n]).to(dtype)


def prepare(case, seed):
    c, gen = case, torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    h_q, h_kv, d, dt = c["h_q"], c["h_kv"], c["d"], _dt(c)
    if c["kind"] == "decode":
        B, P, cap = c["B"], c["P"], c["cap"]
        x = dict(q=_normal(gen, B, h_q, d, dtype=dt),
                 k_prefix=_keys(gen, h_kv, P + c["room"], d, dt)[:, :P],
                 v_prefix=_normal(gen, h_kv, P + c["room"], d, dtype=dt)[:, :P],
                 k_cache=_keys(gen, B * h_kv, cap, d, dt).view(B, h_kv, cap, d),
                 v_cache=_normal(gen, B, h_kv, cap, d, dtype=dt),
                 lens=torch.tensor(_lens(c), dtype=torch.int32, device=DEV))
    else:
        B, L = c["B"], c["L"]
        x = dict(q=_normal(gen, B, L, h_q, d, dtype=dt), k=_keys(gen, B * h_kv, L, d, dt).view(B, h_kv, L, d),
                 v=_normal(gen, B, h_kv, L, d, dtype=dt))
        if c["kind"] == "train":
            x["dO"] = _normal(gen, B, L, h_q, d, dtype=dt)
        spans = _spans(c)
        x["spans"] = spans
        x["cu"] = None
        if c["n_seq"]:
            x["cu"] = torch.tensor([s[1] for s in spans] + [c["L"]], dtype=torch.int32, device=DEV)
    x["case"] = c
    if own:
        import chunked_hierarchical_sparse_b200 as hsa
        hsa.load_library()
        x["hsa"] = hsa
    return x


# --------------------------------------------------------------- the calls
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own_decode(state) if kind == "decode" else _own_prompt(state)
    return _plain_decode(state) if kind == "decode" else _plain_prompt(state)


def _own_prompt(x):
    m, c = x["hsa"], x["case"]
    o, lse = m.hsa_prompt_fwd(x["q"], x["k"], x["v"], cu_seqlens=x["cu"], off_by_one=c["off_by_one"])
    if c["kind"] == "prompt":
        return o, lse
    dq, dk, dv = m.hsa_prompt_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, cu_seqlens=x["cu"])
    return o, lse, dq, dk, dv


def _own_decode(x):
    return x["hsa"].hsa_prefix_decode(x["q"], x["k_prefix"], x["v_prefix"], x["k_cache"], x["v_cache"], x["lens"],
                                      off_by_one=x["case"]["off_by_one"])


# ------------------------------------------------------ plain forms (32 bits)
def _softmax_parts(s, off_by_one):
    """(weights, log of the normaliser) of each row's visible logits (-inf: masked)."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    if off_by_one:
        m = m.clamp(min=0)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    if off_by_one:
        z = z + torch.exp(-m)
    p = torch.where(z > 0, e / z, torch.zeros_like(e))
    return p, (m + torch.log(z)).squeeze(-1)


def _plain_prompt(x):
    c = x["case"]
    dt, G, d, train = _dt(c), c["h_q"] // c["h_kv"], c["d"], c["kind"] == "train"
    q, k, v = x["q"], x["k"], x["v"]
    scale = 1.0 / math.sqrt(d)
    o = torch.zeros(q.shape, dtype=dt, device=DEV)
    lse = torch.zeros(q.shape[:3], dtype=torch.float32, device=DEV)
    if train:
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, t0, n in x["spans"]:
        rows = max(16, min(n, (1 << 27) // max(1, n * G)))  # scores of one block: at most 512 MB
        for g in range(c["h_kv"]):
            kk, vv = k[b, g, t0:t0 + n].float(), v[b, g, t0:t0 + n].float()
            if train:
                gk, gv = torch.zeros_like(kk), torch.zeros_like(vv)
            hs = slice(g * G, g * G + G)
            for r0 in range(0, n, rows):
                r1 = min(n, r0 + rows)
                ts = slice(t0 + r0, t0 + r1)
                qq = q[b, ts, hs].float().transpose(0, 1)                      # [G, r, d]
                s = (qq @ kk[:r1].T) * scale
                future = (torch.arange(r1, device=DEV)[None, :] > torch.arange(r0, r1, device=DEV)[:, None])
                s.masked_fill_(future, -math.inf)
                p, z = _softmax_parts(s, c["off_by_one"])
                del s
                oo = p @ vv[:r1]
                o[b, ts, hs] = oo.transpose(0, 1).to(dt)
                lse[b, ts, hs] = z.T
                if train:
                    do = x["dO"][b, ts, hs].float().transpose(0, 1)
                    dp = do @ vv[:r1].T
                    ds = p * (dp - (do * oo).sum(-1, keepdim=True)) * scale
                    dq[b, ts, hs] = (ds @ kk[:r1]).transpose(0, 1).to(dt)
                    gk[:r1] += ds.flatten(0, 1).T @ qq.flatten(0, 1)
                    gv[:r1] += p.flatten(0, 1).T @ do.flatten(0, 1)
            if train:
                dk[b, g, t0:t0 + n] = gk.to(dt)
                dv[b, g, t0:t0 + n] = gv.to(dt)
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _plain_decode(x):
    c = x["case"]
    B, P, cap, h_kv, d = c["B"], c["P"], c["cap"], c["h_kv"], c["d"]
    G = c["h_q"] // h_kv
    q = x["q"].float().view(B, h_kv, G, d)
    s = torch.empty(B, h_kv, G, P + cap, device=DEV)
    qg = q.transpose(0, 1).reshape(h_kv, B * G, d)
    s[..., :P] = (qg @ x["k_prefix"].float().transpose(1, 2)).view(h_kv, B, G, P).transpose(0, 1)
    s[..., P:] = q @ x["k_cache"].float().transpose(2, 3)
    s *= 1.0 / math.sqrt(d)
    absent = torch.arange(cap, device=DEV)[None, :] >= x["lens"][:, None]
    s[..., P:].masked_fill_(absent[:, None, None, :], -math.inf)
    p, lse = _softmax_parts(s, c["off_by_one"])
    o = p[..., P:] @ x["v_cache"].float()
    pg = p[..., :P].transpose(0, 1).reshape(h_kv, B * G, P)
    o = o + (pg @ x["v_prefix"].float()).view(h_kv, B, G, d).transpose(0, 1)
    return o.reshape(B, c["h_q"], d).to(_dt(c)), lse.reshape(B, c["h_q"])


# ------------------------------------------------- work, and the exact values
def work(case):
    c = case
    h_q, h_kv, d, e = c["h_q"], c["h_kv"], c["d"], 4 if c["dtype"] == "fp32" else 2
    if c["kind"] == "decode":
        n = sum(_lens(c))
        return {"bytes": e * d * (2 * c["B"] * h_q + 2 * h_kv * (c["P"] + n)) + 4 * c["B"] * (h_q + 1),
                "flops": 4 * d * h_q * (c["B"] * c["P"] + n)}
    pairs = sum(n * (n + 1) // 2 for _, _, n in _spans(c))
    toks = c["B"] * c["L"]
    if c["kind"] == "prompt":  # q, k, v in; o, lse out
        return {"bytes": toks * (e * d * (2 * h_q + 2 * h_kv) + 4 * h_q), "flops": 4 * d * h_q * pairs}
    # q, k, v, dO in; o, lse, dq, dk, dv out; two products forward, five backward
    return {"bytes": toks * (e * d * (4 * h_q + 4 * h_kv) + 4 * h_q), "flops": 14 * d * h_q * pairs}


def exact(case, seed):
    """The definitions in 64 bits: head by head, weights from the normaliser Z of each row."""
    c, x = case, prepare(case, seed)
    h_q, h_kv, d = c["h_q"], c["h_kv"], c["d"]
    G, one = h_q // h_kv, 1.0 if c["off_by_one"] else 0.0
    f8 = torch.float64
    if c["kind"] == "decode":
        o = torch.zeros(c["B"], h_q, d, dtype=f8, device=DEV)
        lse = torch.zeros(c["B"], h_q, dtype=f8, device=DEV)
        for b, n in enumerate(_lens(c)):
            for g in range(h_kv):
                keys = torch.cat([x["k_prefix"][g], x["k_cache"][b, g, :n]]).to(f8)
                vals = torch.cat([x["v_prefix"][g], x["v_cache"][b, g, :n]]).to(f8)
                h = slice(g * G, g * G + G)
                a = torch.einsum("hd,nd->hn", x["q"][b, h].to(f8), keys) / math.sqrt(d)
                if a.shape[1] == 0:  # nothing to attend to: output 0, log of an empty sum
                    lse[b, h] = 0.0 if one else -math.inf
                    continue
                top = a.max(1).values
                w = (a - top[:, None]).exp()
                Z = w.sum(1) + one * (-top).exp()
                o[b, h] = torch.einsum("hn,nd->hd", w, vals) / Z[:, None]
                lse[b, h] = top + Z.log()
        return o, lse
    train = c["kind"] == "train"
    o = torch.zeros(x["q"].shape, dtype=f8, device=DEV)
    lse = torch.zeros(x["q"].shape[:3], dtype=f8, device=DEV)
    dq = torch.zeros_like(o)
    dk = torch.zeros(x["k"].shape, dtype=f8, device=DEV)
    dv = torch.zeros_like(dk)
    for b, first, n in _spans(c):
        step = max(1, min(n, (1 << 27) // max(1, n)))
        for h in range(h_q):
            g = h // G
            K, V = x["k"][b, g, first:first + n].to(f8), x["v"][b, g, first:first + n].to(f8)
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                at = slice(first + lo, first + hi)
                Q = x["q"][b, at, h].to(f8)
                a = torch.mm(Q, K[:hi].t()).div_(math.sqrt(d))
                seen = torch.ones(hi - lo, hi, dtype=torch.bool, device=DEV).tril_(lo)
                top = a.masked_fill(~seen, -math.inf).max(1).values
                w = a.sub_(top[:, None]).exp_().mul_(seen)
                Z = w.sum(1) + one * (-top).exp()
                w /= Z[:, None]
                out = torch.mm(w, V[:hi])
                o[b, at, h] = out
                lse[b, at, h] = top + Z.log()
                if train:
                    D = x["dO"][b, at, h].to(f8)
                    dv[b, g, first:first + hi] += torch.mm(w.t(), D)
                    t = torch.mm(D, V[:hi].t()).sub_((D * out).sum(1)[:, None]).mul_(w).div_(math.sqrt(d))
                    dq[b, at, h] = torch.mm(t, K[:hi])
                    dk[b, g, first:first + hi] += torch.mm(t.t(), Q)
    return (o, lse, dq, dk, dv) if train else (o, lse)
