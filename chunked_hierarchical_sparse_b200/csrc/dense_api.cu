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

// words of the workspace header behind the status word (all cleared by every call)
constexpr int kWordPlanN = 8, kWordKPlanN = 9, kWordNext = 32;
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
    int4 *plan, *kplan;
    float *delta;
    size_t bytes;
};

// tokens of a row item: 64 rows on the CUDA cores (fp32), two tiles of 128 rows on the
// tensor cores (bf16)
int row_tile(const hsa_prompt_shape_t &s) {
    const int G = s.h_q / s.h_kv;
    return s.dtype == HSA_BF16 ? 2 * (128 / G) : kSimtRows / G;
}
// the backward's: one tile of rows, and its tiles of keys
int bwd_row_tile(const hsa_prompt_shape_t &s) { return (s.dtype == HSA_BF16 ? 128 : kSimtRows) / (s.h_q / s.h_kv); }
int bwd_key_tile(const hsa_prompt_shape_t &s) { return s.dtype == HSA_BF16 ? 128 : kSimtRows; }

PromptWs carve_prompt(const hsa_prompt_shape_t &s, void *ws, bool bwd) {
    Carver c{static_cast<char *>(ws)};
    PromptWs w{};
    if (s.n_seq > 0) w.plan = c.take<int4>(plan_cap(s.L, s.n_seq, bwd ? bwd_row_tile(s) : row_tile(s)));
    if (bwd) {
        if (s.n_seq > 0) w.kplan = c.take<int4>(plan_cap(s.L, s.n_seq, bwd_key_tile(s)));
        w.delta = c.take<float>((size_t)s.B * s.L * s.h_q);
    }
    w.bytes = c.off;
    return w;
}

Args prompt_args(const hsa_prompt_shape_t &s, const void *q, const void *k, const void *v, void *ws, const PromptWs &w,
                 int tok) {
    Args a{};
    a.B = s.B; a.L = s.L; a.hq = s.h_q; a.hkv = s.h_kv; a.G = s.h_q / s.h_kv;
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

int64_t max_items(const hsa_prompt_shape_t &s, int tok) {
    return s.n_seq > 0 ? plan_cap(s.L, s.n_seq, tok) * s.h_kv : (int64_t)s.B * s.h_kv * ceil_div(s.L, tok);
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
    // the prefix: one item per SM (a second round of them costs more than it balances: 256 x 32K
    // tokens 80 us, 96 with two rounds), of two tiles of 128 keys at least; on the CUDA cores
    // about two blocks of 64-key tiles per SM
    p.pre_sub = slot_keys(s.P, (int64_t)s.h_kv * p.pre_tiles, tc ? kSms : 2 * kSms, tc ? 256 : kSimtRows);
    p.pre_slots = p.pre_sub ? (int)ceil_div(s.P, p.pre_sub) : 0;
    // the own caches: two blocks of four stages of 64 keys and more per SM
    p.suf_sub = slot_keys(s.cap, (int64_t)s.h_kv * s.B, 2 * kSms, tc ? 256 : kSimtRows);
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
    Args a = prompt_args(*shape, q, k, v, ws, w, row_tile(*shape));
    a.o = o;
    a.lse = lse;
    TimedLaunch tl(HSA_K_PROMPT_FWD, cu_seqlens ? 2 : 1, st);
    if (cu_seqlens) e = launch_plan(cu_seqlens, shape->n_seq, shape->L, a.tok, false, w.plan, word(ws, kWordPlanN), a.ds, true, st);
    if (e == cudaSuccess) {
        const int64_t items = max_items(*shape, a.tok);
        e = shape->dtype == HSA_BF16 ? launch_fwd_tc(a, shape->d, items, word(ws, kWordNext), st)
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
    // the first kernel of a packed call clears the header itself
    cudaError_t e = empty || !cu_seqlens ? cudaMemsetAsync(ws, 0, kWsHeader, st) : cudaSuccess;
    if (empty || e != cudaSuccess) return cuda_status(e);
    const PromptWs w = carve_prompt(*shape, ws, true);
    const bool bf16 = shape->dtype == HSA_BF16;
    BwdArgs b{};
    b.a = prompt_args(*shape, q, k, v, ws, w, bwd_row_tile(*shape));
    b.kplan = w.kplan;
    b.kplan_n = word(ws, kWordKPlanN);
    b.ktiles = (int)ceil_div(shape->L, bwd_key_tile(*shape));
    b.o = o; b.dO = dO; b.lse = lse; b.delta = w.delta;
    b.dq = dq; b.dk = dk; b.dv = dv;
    TimedLaunch tl(HSA_K_PROMPT_BWD, cu_seqlens ? 5 : 3, st);
    if (cu_seqlens) {
        e = launch_plan(cu_seqlens, shape->n_seq, shape->L, b.a.tok, false, w.plan, word(ws, kWordPlanN), b.a.ds, true, st);
        if (e == cudaSuccess)
            e = launch_plan(cu_seqlens, shape->n_seq, shape->L, bwd_key_tile(*shape), true, w.kplan, word(ws, kWordKPlanN), b.a.ds, false, st);
    }
    if (e == cudaSuccess) e = launch_delta(b, shape->d, bf16, st);
    if (e == cudaSuccess) {
        const int64_t row_items = max_items(*shape, b.a.tok), key_items = max_items(*shape, bwd_key_tile(*shape));
        e = bf16 ? launch_bwd_tc(b, shape->d, row_items, key_items, word(ws, kWordNext), st)
                 : launch_bwd_simt(b, shape->d, row_items, key_items, st);
    }
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
