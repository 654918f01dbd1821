// dense_api.cu -- the extern "C" entry points of the dense attention operators:
// argument checks, workspace carving, and the kernel sequence of each call.
#include <algorithm>
#include <climits>
#include <cmath>
#include <initializer_list>

#include "dense.cuh"

using namespace hsa;
using namespace hsa::dense;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool all_ok(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!p || !aligned16(p)) return false;
    return true;
}
bool opt_ok(const void *p) { return !p || aligned16(p); }
bool ws_ok(const void *ws) { return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0; }

hsa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? HSA_OK : HSA_ERR_CUDA; }

struct Carver {
    char *base;
    size_t off = kWsHeader;
    template <typename T> T *take(size_t count) {
        T *p = base ? reinterpret_cast<T *>(base + off) : nullptr;
        off += round_up((int64_t)(count * sizeof(T)), 256);
        return p;
    }
};

int32_t *word(void *ws, int i) { return static_cast<int32_t *>(ws) + i; }

hsa_status_t check_heads(int h_q, int h_kv, int d, int off_by_one, int dtype) {
    if (h_q < 1 || h_kv < 1 || d < 1 || h_q % h_kv != 0) return HSA_ERR_INVALID_ARG;
    if (off_by_one != 0 && off_by_one != 1) return HSA_ERR_INVALID_ARG;
    if (dtype != HSA_F32 && dtype != HSA_BF16) return HSA_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || h_q / h_kv > kMaxG) return HSA_ERR_UNSUPPORTED;
    return HSA_OK;
}

// ------------------------------------------------------------------ prompt pass
hsa_status_t check_prompt(const hsa_prompt_shape_t *s) {
    if (!s || s->B < 0 || s->L < 0 || s->n_seq < 0) return HSA_ERR_INVALID_ARG;
    hsa_status_t r = check_heads(s->h_q, s->h_kv, s->d, s->off_by_one, s->dtype);
    if (r != HSA_OK) return r;
    if (s->n_seq > 0 && s->B != 1) return HSA_ERR_INVALID_ARG;
    // token rows, planes and work items are int32 (a tile holds one token at least)
    if ((int64_t)s->B * s->L >= (1 << 30) || (int64_t)s->B * s->h_kv >= (1 << 30)) return HSA_ERR_UNSUPPORTED;
    if (((int64_t)s->B * s->L + s->n_seq) * s->h_kv >= (1 << 30)) return HSA_ERR_UNSUPPORTED;
    return HSA_OK;
}

struct PromptWs {
    int4 *plan, *kplan, *kpiece, *cut;
    float *delta, *part;
    size_t bytes;
};

bool tensor_cores(const hsa_prompt_shape_t &s) { return s.dtype == HSA_BF16; }
int group(const hsa_prompt_shape_t &s) { return s.h_q / s.h_kv; }
int64_t row_items(const hsa_prompt_shape_t &s, int tok) {
    return s.n_seq > 0 ? plan_cap(s.L, s.n_seq, tok) * s.h_kv : (int64_t)s.B * s.h_kv * ceil_div(s.L, tok);
}

// Forward, tensor cores, not packed: two row tiles per item where that fills the GPU, else
// one, whose streams split the keys (one prompt of 1K
// tokens, 16 heads in 2 groups: 16 us, 23 without).
bool fwd_split(const hsa_prompt_shape_t &s) {
    return tensor_cores(s) && s.n_seq == 0 && row_items(s, 2 * (128 / group(s))) <= kPlanSms;
}
// tokens of a row item: 64 rows on the CUDA cores (fp32), 128-row tiles on the tensor cores
int fwd_tok(const hsa_prompt_shape_t &s) {
    return tensor_cores(s) ? (fwd_split(s) ? 1 : 2) * (128 / group(s)) : kSimtRows / group(s);
}
int bwd_tok(const hsa_prompt_shape_t &s) { return (tensor_cores(s) ? 128 : kSimtRows) / group(s); }
int key_tile(const hsa_prompt_shape_t &s) { return tensor_cores(s) ? 128 : kSimtRows; }

// Backward, tensor cores: steps of the key pass (not packed: exactly; packed: at most) and
// whether some key tile's rows are cut into pieces.
uint64_t key_steps(const hsa_prompt_shape_t &s) {
    const int tt = 128 / group(s);
    const int64_t n = ceil_div(s.L, 128), rows = ceil_div(s.L, tt);
    uint64_t w = 0;
    for (int64_t i = 0; i < n; ++i) w += rows - i * 128 / tt;
    return w * s.h_kv * s.B;
}
bool key_pieces(const hsa_prompt_shape_t &s) {
    if (!tensor_cores(s)) return false;
    return s.n_seq > 0 || cut_rows((int)ceil_div(s.L, 128 / group(s)), key_steps(s));
}

PromptWs carve_prompt(const hsa_prompt_shape_t &s, void *ws, bool bwd) {
    Carver c{static_cast<char *>(ws)};
    PromptWs w{};
    // a packed forward may cut every sequence into half-size items
    if (s.n_seq > 0)
        w.plan = c.take<int4>(plan_cap(s.L, s.n_seq, bwd ? bwd_tok(s) : tensor_cores(s) ? 128 / group(s) : fwd_tok(s)));
    if (bwd) {
        w.delta = c.take<float>((size_t)s.B * s.L * s.h_q);
        const bool pieces = key_pieces(s);
        if (pieces || s.n_seq > 0) {
            const int64_t n = s.n_seq > 0 ? plan_cap(s.L, s.n_seq, key_tile(s)) : (int64_t)s.B * ceil_div(s.L, key_tile(s));
            w.kplan = c.take<int4>(n + (pieces ? kMaxPieces : 0));
            if (pieces) {
                w.kpiece = c.take<int4>(n + kMaxPieces);
                w.cut = c.take<int4>(std::min<int64_t>(n, kMaxPieces));
                // pieces have more than 2 row tiles, which bounds their number for short rows
                const int64_t most = n * s.h_kv * (1 + ceil_div(s.L, 128 / group(s)) / 2);
                w.part = c.take<float>((size_t)std::min<int64_t>(kMaxPieces, most) * 2 * 128 * s.d);
            }
        }
    }
    w.bytes = c.off;
    return w;
}

Args prompt_args(const hsa_prompt_shape_t &s, const void *q, const void *k, const void *v, void *ws, const PromptWs &w,
                 int tok) {
    Args a{};
    a.B = s.B; a.L = s.L; a.hq = s.h_q; a.hkv = s.h_kv; a.G = group(s);
    a.tok = tok;
    a.off_by_one = s.off_by_one;
    a.scale = 1.0f / sqrtf((float)s.d);
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)s.d));
    a.plan = w.plan;
    a.plan_n = word(ws, kWordPlanN);
    a.tiles = (int)ceil_div(s.L, a.tok);
    a.q = q; a.k[0] = k; a.v[0] = v;
    a.plane[0] = (int64_t)s.L * s.d;
    a.ds = static_cast<DevStatus *>(ws);
    return a;
}

PlanJob plan_job(const hsa_prompt_shape_t &s, PlanKind kind, const int32_t *cu, int tok, int4 *plan, int4 *piece, int32_t *n) {
    PlanJob j{};
    j.kind = kind;
    j.cu = cu;
    j.n_seq = cu ? s.n_seq : s.B;
    j.L = s.L; j.tok = tok; j.G = group(s); j.hkv = s.h_kv;
    j.plan = plan; j.piece = piece; j.n = n;
    return j;
}

// checks shared by the two directions; *empty: nothing to read or write
hsa_status_t check_prompt_call(const hsa_prompt_shape_t *shape, const int32_t *cu, int op, void *ws, size_t ws_bytes,
                               bool *empty) {
    hsa_status_t s = check_prompt(shape);
    if (s != HSA_OK) return s;
    *empty = (int64_t)shape->B * shape->L == 0;
    if (!ws_ok(ws)) return HSA_ERR_INVALID_ARG;
    if ((shape->n_seq > 0) != (cu != nullptr)) return HSA_ERR_INVALID_ARG;
    if (cu && (reinterpret_cast<uintptr_t>(cu) & 3u)) return HSA_ERR_INVALID_ARG;
    if (ws_bytes < hsa_prompt_workspace_size(shape, op)) return HSA_ERR_WORKSPACE;
    return HSA_OK;
}

// ------------------------------------------------------------------ shared-prefix decode
constexpr int kSms = 148;

struct PrefixPlan {
    int tok, split, pre_tiles, pre_sub, pre_slots, suf_sub, suf_slots;
    size_t po, plse, bytes;  // workspace offsets
};

hsa_status_t check_prefix(const hsa_prefix_shape_t *s) {
    if (!s || s->B < 0 || s->P < 0 || s->cap < 0) return HSA_ERR_INVALID_ARG;
    hsa_status_t r = check_heads(s->h_q, s->h_kv, s->d, s->off_by_one, s->dtype);
    if (r != HSA_OK) return r;
    if (s->P > 0) {
        const int per16 = s->dtype == HSA_BF16 ? 8 : 4;
        if (s->prefix_stride < (int64_t)s->P * s->d || s->prefix_stride % per16) return HSA_ERR_INVALID_ARG;
    }
    if ((int64_t)s->B * s->h_q >= (1 << 24) || s->P >= (1 << 30) || s->cap >= (1 << 30)) return HSA_ERR_UNSUPPORTED;
    return HSA_OK;
}

// keys per slot: about `want` slots in all for `jobs` independent jobs of `keys` keys, in whole tiles
int slot_keys(int64_t keys, int64_t jobs, int64_t want, int tile) {
    if (keys == 0) return 0;
    const int64_t n = std::clamp<int64_t>(want / std::max<int64_t>(jobs, 1), 1, ceil_div(keys, tile));
    return (int)round_up(ceil_div(keys, n), tile);
}

PrefixPlan plan_prefix(const hsa_prefix_shape_t &s) {
    PrefixPlan p{};
    const bool tc = s.dtype == HSA_BF16;
    const int G = s.h_q / s.h_kv, fit = (tc ? 128 : kSimtRows) / G;
    // tensor cores: a batch beyond one row tile shares the keys between two row tiles, a
    // smaller one splits them between the two streams
    p.split = tc && s.B <= fit;
    p.tok = tc && !p.split ? 2 * fit : fit;
    p.pre_tiles = (int)ceil_div(s.B, p.tok);
    if (tc) {
        // The prefix: one item per SM, of two tiles of 128 keys at least (a second round of
        // items costs more than it balances: 256 sequences behind 32K tokens with up to 2K of
        // their own 107 us, 124 with two rounds).  Where it keeps every SM for long (8 steps of
        // 256 x 128 and more), it leaves to the own caches, which are bound by HBM, as many SMs
        // as let them finish beside it: a step takes about 1.8 us (d = 128), an SM reads about
        // 110 GB/s, and half of cap is taken as used, since the lengths are on the device.  That
        // step without the SMs left free: 123 us; every cache full 149, 167 without; 128 sequences
        // with up to 8K tokens of their own 112, 135 without.  Where the caches are all but empty
        // the SMs are left free for nothing: up to 32 tokens in a cap of 2K 90 us, 81 without, up
        // to 64 in a cap of 8K 67, 47 without.
        const int64_t jobs = (int64_t)s.h_kv * p.pre_tiles;
        const double steps = (double)jobs * (p.split ? 0.5 : 1.0) * ceil_div(s.P, 128);
        const double pre_us = steps * 1.8 * s.d / 128, suf_us = 0.5 * s.B * s.h_kv * (double)s.cap * 4 * s.d / 110e3;
        int sms = kSms;
        if (steps >= 8 * kSms) sms -= (int)std::min(kSms * suf_us / (pre_us + suf_us), kSms / 2.0);
        p.pre_sub = slot_keys(s.P, jobs, sms, 256);
        // The own caches: three blocks fit an SM, ragged lengths want several rounds of them (the
        // first step above with ranges of 2048, 1024 and 512 keys: 112, 107, 111 us; with every
        // cache full 142, 149, 152).
        p.suf_sub = slot_keys(s.cap, (int64_t)s.h_kv * s.B, 8 * kSms, 256);
    } else {  // about two blocks of 64-key tiles per SM
        p.pre_sub = slot_keys(s.P, (int64_t)s.h_kv * p.pre_tiles, 2 * kSms, kSimtRows);
        p.suf_sub = slot_keys(s.cap, (int64_t)s.h_kv * s.B, 2 * kSms, kSimtRows);
    }
    p.pre_slots = p.pre_sub ? (int)ceil_div(s.P, p.pre_sub) : 0;
    p.suf_slots = p.suf_sub ? (int)ceil_div(s.cap, p.suf_sub) : 0;
    Carver c{nullptr};
    const size_t rows = (size_t)s.B * s.h_q * (p.pre_slots + p.suf_slots);
    p.po = c.off;
    c.take<float>(rows * s.d);
    p.plse = c.off;
    c.take<float>(rows);
    p.bytes = c.off;
    return p;
}

}  // namespace

extern "C" {

size_t hsa_prompt_workspace_size(const hsa_prompt_shape_t *shape, int op) {
    if (check_prompt(shape) != HSA_OK || (op != HSA_OP_FWD && op != HSA_OP_BWD)) return 0;
    return carve_prompt(*shape, nullptr, op == HSA_OP_BWD).bytes;
}

hsa_status_t hsa_prompt_fwd(const hsa_prompt_shape_t *shape, const void *q, const void *k, const void *v,
                            const int32_t *cu_seqlens, void *o, float *lse, void *ws, size_t ws_bytes, void *stream) {
    bool empty = false;
    hsa_status_t s = check_prompt_call(shape, cu_seqlens, HSA_OP_FWD, ws, ws_bytes, &empty);
    if (s != HSA_OK) return s;
    if (!empty && (!all_ok({q, k, v, o}) || !opt_ok(lse))) return HSA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (empty) return cuda_status(cudaMemsetAsync(ws, 0, kWsHeader, st));
    cudaError_t e = cudaSuccess;  // the first launch clears the header
    const PromptWs w = carve_prompt(*shape, ws, false);
    Args a = prompt_args(*shape, q, k, v, ws, w, fwd_tok(*shape));
    a.split = fwd_split(*shape);
    a.o = o;
    a.lse = lse;
    TimedLaunch tl(HSA_K_PROMPT_FWD, cu_seqlens ? 2 : 1, st);
    if (cu_seqlens)
        e = launch_plan(plan_job(*shape, tensor_cores(*shape) ? kRowsSplit : kRows, cu_seqlens, a.tok, w.plan, nullptr,
                                 word(ws, kWordPlanN)),
                        nullptr, a.ds, st);
    if (e == cudaSuccess) {
        const int64_t items = row_items(*shape, a.tok);
        e = tensor_cores(*shape) ? launch_fwd_tc(a, shape->d, items, word(ws, kWordNext), st)
                                     : launch_fwd_simt(a, shape->d, items, st);
    }
    return cuda_status(e);
}

hsa_status_t hsa_prompt_bwd(const hsa_prompt_shape_t *shape, const void *q, const void *k, const void *v, const void *o,
                            const void *dO, const float *lse, const int32_t *cu_seqlens, void *dq, void *dk, void *dv,
                            void *ws, size_t ws_bytes, void *stream) {
    bool empty = false;
    hsa_status_t s = check_prompt_call(shape, cu_seqlens, HSA_OP_BWD, ws, ws_bytes, &empty);
    if (s != HSA_OK) return s;
    if (!empty && !all_ok({q, k, v, o, dO, lse, dq, dk, dv})) return HSA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const PromptWs w = carve_prompt(*shape, ws, true);
    const bool planned = w.kplan != nullptr, tc = tensor_cores(*shape);
    // (the plan kernel and the fp32 kernels clear the header themselves)
    cudaError_t e = empty || (tc && !planned) ? cudaMemsetAsync(ws, 0, kWsHeader, st) : cudaSuccess;
    if (empty || e != cudaSuccess) return cuda_status(e);
    BwdArgs b{};
    b.a = prompt_args(*shape, q, k, v, ws, w, bwd_tok(*shape));
    b.kplan = w.kplan;
    b.kpiece = w.kpiece;
    b.kplan_n = word(ws, kWordKPlanN);
    b.ktiles = (int)ceil_div(shape->L, key_tile(*shape));
    b.part = w.part;
    b.cut = w.cut;
    b.n_cut = word(ws, kWordCutN);
    b.o = o; b.dO = dO; b.lse = lse; b.delta = w.delta;
    b.dq = dq; b.dk = dk; b.dv = dv;
    TimedLaunch tl(HSA_K_PROMPT_BWD, (tc ? 2 : 3) + planned + (w.part != nullptr), st);
    if (planned) {
        PlanJob keys = plan_job(*shape, tc ? kKeysSplit : kKeys, cu_seqlens, key_tile(*shape), w.kplan, w.kpiece,
                                word(ws, kWordKPlanN));
        keys.cut = w.cut;
        keys.n_cut = word(ws, kWordCutN);
        if (cu_seqlens)
            e = launch_plan(plan_job(*shape, kRows, cu_seqlens, b.a.tok, w.plan, nullptr, word(ws, kWordPlanN)), &keys,
                            b.a.ds, st);
        else
            e = launch_plan(keys, nullptr, b.a.ds, st);
    }
    if (e == cudaSuccess && !tc) e = launch_delta(b, shape->d, cu_seqlens, shape->n_seq, st);
    if (e == cudaSuccess) {
        const int64_t rows = row_items(*shape, b.a.tok), keys = row_items(*shape, key_tile(*shape)) + (w.part ? kMaxPieces : 0);
        e = tc ? launch_bwd_tc(b, shape->d, rows, keys, word(ws, kWordNext), st)
               : launch_bwd_simt(b, shape->d, rows, keys, st);
    }
    if (e == cudaSuccess && w.part) e = launch_add_pieces(b, shape->d, st);
    return cuda_status(e);
}

size_t hsa_prefix_workspace_size(const hsa_prefix_shape_t *shape) {
    return check_prefix(shape) == HSA_OK ? plan_prefix(*shape).bytes : 0;
}

hsa_status_t hsa_prefix_decode(const hsa_prefix_shape_t *shape, const void *q, const void *k_prefix,
                               const void *v_prefix, const void *k_cache, const void *v_cache, const int32_t *lens,
                               void *o, float *lse, void *ws, size_t ws_bytes, void *stream) {
    hsa_status_t s = check_prefix(shape);
    if (s != HSA_OK) return s;
    if (!ws_ok(ws)) return HSA_ERR_INVALID_ARG;
    const PrefixPlan p = plan_prefix(*shape);
    if (ws_bytes < p.bytes) return HSA_ERR_WORKSPACE;
    if (shape->B > 0) {
        if (!all_ok({q, o}) || !opt_ok(lse)) return HSA_ERR_INVALID_ARG;
        if (shape->P > 0 && !all_ok({k_prefix, v_prefix})) return HSA_ERR_INVALID_ARG;
        if (shape->cap > 0 && (!all_ok({k_cache, v_cache}) || !lens || (reinterpret_cast<uintptr_t>(lens) & 3u)))
            return HSA_ERR_INVALID_ARG;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (shape->B == 0) return cuda_status(cudaMemsetAsync(ws, 0, kWsHeader, st));
    cudaError_t e = cudaSuccess;
    const bool bf16 = shape->dtype == HSA_BF16;
    Args a{};
    a.decode = 1;
    a.B = shape->B; a.L = shape->P; a.hq = shape->h_q; a.hkv = shape->h_kv; a.G = shape->h_q / shape->h_kv;
    a.tok = p.tok;
    a.off_by_one = shape->off_by_one;
    a.scale = 1.0f / sqrtf((float)shape->d);
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)shape->d));
    a.cap = shape->cap; a.lens = lens;
    a.split = p.split;
    a.pre_tiles = p.pre_tiles; a.pre_sub = p.pre_sub; a.pre_slots = p.pre_slots;
    a.suf_sub = p.suf_sub; a.suf_slots = p.suf_slots;
    a.q = q;
    a.k[0] = k_prefix; a.v[0] = v_prefix; a.plane[0] = shape->prefix_stride;
    a.k[1] = k_cache; a.v[1] = v_cache; a.plane[1] = (int64_t)shape->cap * shape->d;
    a.o = o; a.lse = lse;
    a.po = reinterpret_cast<float *>(static_cast<char *>(ws) + p.po);
    a.plse = reinterpret_cast<float *>(static_cast<char *>(ws) + p.plse);
    a.ds = static_cast<DevStatus *>(ws);
    const int np = pre_items(a), ns = suf_items(a);
    TimedLaunch tl(HSA_K_PREFIX, 1 + (bf16 ? (np > 0) + (ns > 0) : np + ns > 0), st);
    if (bf16) {
        if (np > 0) {
            Args pre = a;
            pre.suf_slots = 0;
            e = launch_fwd_tc(pre, shape->d, np, word(ws, kWordNext), st);
        }
        if (e == cudaSuccess && ns > 0) e = launch_cache(a, shape->d, np == 0, st);
    } else if (np + ns > 0) {
        e = launch_fwd_simt(a, shape->d, (int64_t)np + ns, st);
    }
    if (np + ns == 0) e = cudaMemsetAsync(ws, 0, kWsHeader, st);
    if (e == cudaSuccess) e = launch_combine(a, shape->d, bf16, st);
    return cuda_status(e);
}

}  // extern "C"
