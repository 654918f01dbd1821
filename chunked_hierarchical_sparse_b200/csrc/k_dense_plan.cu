// k_dense_plan.cu -- work lists, and joining partials (of the decode step, of the backward).
#include <type_traits>

#include "dense.cuh"

namespace hsa {
namespace dense {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;

// One block per job.  An item's cost is the number of tiles it walks; a counting sort over
// kBins cost classes puts the dearest first.  Inside a class the order is not fixed, nor is
// the numbering of the partial slots: every item is computed by itself, and partials are
// added in the order of their ranges, so neither changes a result.  (What is cut, and
// where, follows from integer sums alone.)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanJob job0,
                                                            const __grid_constant__ PlanJob job1, DevStatus *ds,
                                                            int clear) {
    const PlanJob &J = blockIdx.x ? job1 : job0;
    __shared__ int hist[kBins];
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int bad, slots, cuts;
    __shared__ unsigned long long work;
    __shared__ int bounds[kPlanThreads + 1];  // cu, where it fits: read once
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    hist[tid] = 0;
    if (tid == 0) {
        bad = slots = cuts = 0;
        work = 0;
    }
    dependency_wait();
    if (clear && blockIdx.x == 0 && tid < kHeaderWords && !header_word_of_plan(tid)) reinterpret_cast<int32_t *>(ds)[tid] = 0;
    __syncthreads();
    dependents_may_start();
    const int tt = 128 / J.G;  // tokens of a 128-row tile
    const bool fits = J.n_seq <= kPlanThreads;
    auto bound = [&](int s) { return fits ? bounds[s] : J.cu[s]; };
    auto seq = [&](int s, int &a, int &len) {
        a = J.cu ? bound(s) : s * J.L;
        len = J.cu ? bound(s + 1) - a : J.L;
    };
    auto key_rows = [&](int i, int len) { return (len + tt - 1) / tt - i * 128 / tt; };  // row tiles that see key tile i
    if (J.cu && fits) {
        for (int s = tid; s <= J.n_seq; s += kPlanThreads) bounds[s] = J.cu[s];
        __syncthreads();
    }
    for (int s = tid; J.cu && s < J.n_seq; s += kPlanThreads) {
        const int a = bound(s), b = bound(s + 1);
        if (a < 0 || b < a || b > J.L) {
            bad = 1;
            report(ds, HSA_ERR_DEVICE_CHECK, kKDense, s, b);
        }
    }
    __syncthreads();
    if (bad) {
        if (tid == 0) {
            *J.n = 0;
            if (J.kind == kKeysSplit) *J.n_cut = 0;
        }
        return;
    }
    if (J.kind == kRowsSplit || J.kind == kKeysSplit) {  // tile steps of the whole job, for one group
        for (int s = warp; s < J.n_seq; s += kPlanThreads / 32) {
            int a, len;
            seq(s, a, len);
            const int n = (len + J.tok - 1) / J.tok;
            unsigned long long w = 0;
            for (int i = lane; i < n; i += 32)
                w += J.kind == kKeysSplit ? key_rows(i, len) : (min((i + 1) * J.tok, len) + 127) / 128;
            for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            if (lane == 0 && w) atomicAdd(&work, w);
        }
        __syncthreads();
    }
    const int limit = J.kind == kKeysSplit   ? key_limit(work * J.hkv)
                      : J.kind == kRowsSplit ? (int)max(2ull, (work * J.hkv + kPlanSms - 1) / kPlanSms)
                                             : 0x7fffffff;
    const int top = (J.kind == kRows || J.kind == kKeys ? (J.L + J.tok - 1) / J.tok
                     : J.kind == kRowsSplit             ? (J.L + 127) / 128
                                                        : (J.L + tt - 1) / tt) + 1;
    // calls f(bin, tile or first token, pieces, tiles per piece) for every tile of sequence s
    auto tiles = [&](int len, auto &&f) {
        const bool halve = J.kind == kRowsSplit && (len + 127) / 128 > limit;
        const int tok = halve ? J.tok / 2 : J.tok, n = (len + tok - 1) / tok;
        for (int i = lane; i < n; i += 32) {
            int cost = i + 1, pieces = 1, per = 0;
            if (J.kind == kKeys) cost = n - i;
            if (J.kind == kRowsSplit) cost = ((min((i + 1) * tok, len) + 127) / 128 + halve) >> halve;
            if (J.kind == kKeysSplit) {
                const int r = key_rows(i, len);
                if (cut_rows(r, work * J.hkv)) pieces = (r + limit - 1) / limit;
                cost = per = (r + pieces - 1) / pieces;
            }
            f(kBins - 1 - (int)min((int64_t)kBins - 1, (int64_t)cost * kBins / top), i, tok, halve, pieces, per);
        }
    };
    for (int s = warp; s < J.n_seq; s += kPlanThreads / 32) {
        int a, len;
        seq(s, a, len);
        tiles(len, [&](int bin, int, int, bool, int pieces, int) { atomicAdd(&hist[bin], pieces); });
    }
    __syncthreads();
    // exclusive scan of the histogram (one bin per thread)
    const int own = hist[tid];
    int x = own;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sum[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    hist[tid] = x - own + (warp ? warp_sum[warp - 1] : 0);
    if (tid == kPlanThreads - 1) *J.n = hist[tid] + own;
    __syncthreads();
    for (int s = warp; s < J.n_seq; s += kPlanThreads / 32) {
        int a, len;
        seq(s, a, len);
        tiles(len, [&](int bin, int i, int tok, bool halve, int pieces, int per) {
            const int at = atomicAdd(&hist[bin], pieces);
            if (J.kind != kKeysSplit) {
                J.plan[at] = make_int4(a, len, J.kind == kKeys ? i : i * tok, halve);
                return;
            }
            const int first = i * 128 / tt, end = (len + tt - 1) / tt;
            int slot = -1;
            if (pieces > 1) {
                slot = atomicAdd(&slots, pieces * J.hkv);
                J.cut[atomicAdd(&cuts, 1)] = make_int4(a, len, i, slot | pieces << 16);
            }
            for (int c = 0; c < pieces; ++c) {
                J.plan[at + c] = make_int4(a, len, i, c);
                J.piece[at + c] = make_int4(first + c * per, min(end, first + (c + 1) * per),
                                            slot < 0 ? -1 : slot + c * J.hkv, 0);
            }
        });
    }
    __syncthreads();
    if (tid == 0 && J.kind == kKeysSplit) *J.n_cut = cuts;
}

// dk, dv of the key tiles whose rows were cut: their partials added in order.  A unit is 16
// keys of dk or dv of one tile and group, one float4 of each piece per thread and pass;
// latency-bound (the partials are in L2), so the units are small and every thread's reads of
// the pieces are in flight together.
template <int D>
__global__ void __launch_bounds__(256) add_pieces_kernel(const __grid_constant__ BwdArgs b) {
    constexpr int kSlab = 16;
    dependency_wait();
    const int units = *b.n_cut * b.a.hkv * 2 * (128 / kSlab);
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int slab = u % (128 / kSlab), which = u / (128 / kSlab) % 2;  // 0: dv, 1: dk
        const int g = u / (256 / kSlab) % b.a.hkv;
        const int4 c = b.cut[u / (256 / kSlab) / b.a.hkv];
        const int row = c.x / b.a.L, n0 = c.z * 128 + slab * kSlab, keys = min(kSlab, c.y - n0);
        const int slot = (c.w & 0xffff) + g, pieces = c.w >> 16;
        const int64_t at = (int64_t)(row * b.a.hkv + g) * b.a.plane[0] + (int64_t)(c.x % b.a.L + n0) * D;
        const int64_t stride = (int64_t)b.a.hkv * 2 * 128 * D;  // from one piece's partial to the next's
        const float f = which ? b.a.scale : 1.f;
        const float *p = b.part + (((int64_t)slot * 2 + which) * 128 + slab * kSlab) * D;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(which ? b.dk : b.dv) + at;
        for (int j = threadIdx.x * 4; j < keys * D; j += 1024) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int q = 0; q < pieces; ++q) {
                const float4 x = *reinterpret_cast<const float4 *>(p + q * stride + j);
                v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
            }
            *reinterpret_cast<__nv_bfloat162 *>(o + j) = __floats2bfloat162_rn(v.x * f, v.y * f);
            *reinterpret_cast<__nv_bfloat162 *>(o + j + 2) = __floats2bfloat162_rn(v.z * f, v.w * f);
        }
    }
}

// Joining the partials of a (sequence, head) row with weights e^{lse_i - max}.  W of the
// block's 8 warps share a row, each taking every W-th slot (a warp reads a slot's d values
// as one line), their sums added in a fixed order.  Latency-bound: with few rows and many
// slots W = 8 keeps enough reads in flight (256 rows of 64 slots); where the rows alone fill
// the GPU a warp per row is enough (4096 rows of 11 slots: 20 us with W = 8, 8 with 1).
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 2048, kJoinSlots = 8;  // fewer rows and at least as many slots: W = 8

template <typename T, int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) combine_kernel(const __grid_constant__ Args a) {
    constexpr int E = D / 32;
    typedef typename std::conditional<E == 4, float4, float2>::type Vec;
    __shared__ float part[kJoinWarps][D + 1];
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, warp = wid % W;
    const int64_t rows = (int64_t)a.B * a.hq;
    const int row = blockIdx.x * (kJoinWarps / W) + wid / W;
    dependency_wait();
    if (row >= rows) return;  // (W = 1 only)
    const int len = a.cap > 0 ? own_len(a, row / a.hq) : 0;
    if (a.cap > 0 && row % a.hq == 0 && warp == 0 && lane == 0 && a.lens[row / a.hq] != len)
        report(a.ds, HSA_ERR_DEVICE_CHECK, kKDense, row / a.hq, a.lens[row / a.hq]);
    const int n = a.pre_slots + (len > 0 ? (len + a.suf_sub - 1) / a.suf_sub : 0);
    float m = a.off_by_one ? 0.f : -INFINITY;  // off-by-one: the added 1 is a logit of 0
    for (int i = lane; i < n; i += 32) m = fmaxf(m, a.plse[i * rows + row]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mm = m == -INFINITY ? 0.f : m;
    float z = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += W) {
        const float w = __expf(a.plse[i * rows + row] - mm);
        const Vec p = *reinterpret_cast<const Vec *>(a.po + (i * rows + row) * D + lane * E);
        z += w;
        acc[0] += w * p.x;
        acc[1] += w * p.y;
        if constexpr (E == 4) {
            acc[2] += w * p.z;
            acc[3] += w * p.w;
        }
    }
    T *o = static_cast<T *>(a.o) + (int64_t)row * D;
    const float one = a.off_by_one ? __expf(-mm) : 0.f;
    if constexpr (W == 1) {
        z += one;
#pragma unroll
        for (int e = 0; e < E; ++e) Elem<T>::store(o + lane * E + e, z == 0.f ? 0.f : acc[e] / z);
        if (a.lse && lane == 0) a.lse[row] = mm + logf(z);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) part[wid][lane * E + e] = acc[e];
        if (lane == 0) part[wid][D] = z;
        __syncthreads();
        if (threadIdx.x >= D) return;
        float s = 0.f;
        z = one;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            s += part[i][threadIdx.x];
            z += part[i][D];
        }
        // no key at all: output 0, lse = log 0; a NaN stays one
        Elem<T>::store(o + threadIdx.x, z == 0.f ? 0.f : s / z);
        if (a.lse && threadIdx.x == 0) a.lse[row] = mm + logf(z);
    }
}

template <typename T, int D> cudaError_t combine(const Args &a, cudaStream_t st) {
    const bool behind = pre_items(a) + suf_items(a) > 0;  // else it is the call's first kernel
    const int rows = a.B * a.hq;
    if (rows < kJoinRows && a.pre_slots + a.suf_slots >= kJoinSlots)
        return launch_next(behind, combine_kernel<T, D, kJoinWarps>, rows, kJoinWarps * 32, 0, st, 1, a);
    return launch_next(behind, combine_kernel<T, D, 1>, (rows + kJoinWarps - 1) / kJoinWarps, kJoinWarps * 32, 0, st, 1, a);
}

}  // namespace

cudaError_t launch_plan(const PlanJob &job0, const PlanJob *job1, DevStatus *ds, cudaStream_t st) {
    return launch_next(false, plan_kernel, job1 ? 2 : 1, kPlanThreads, 0, st, 1, job0, job1 ? *job1 : job0, ds, 1);
}

cudaError_t launch_add_pieces(const BwdArgs &b, int d, cudaStream_t st) {
    return d == 128 ? launch_next(true, add_pieces_kernel<128>, 8 * kPlanSms, 256, 0, st, 1, b)
                    : launch_next(true, add_pieces_kernel<64>, 8 * kPlanSms, 256, 0, st, 1, b);
}

cudaError_t launch_combine(const Args &a, int d, bool bf16, cudaStream_t st) {
    if (bf16) return d == 128 ? combine<__nv_bfloat16, 128>(a, st) : combine<__nv_bfloat16, 64>(a, st);
    return d == 128 ? combine<float, 128>(a, st) : combine<float, 64>(a, st);
}

}  // namespace dense
}  // namespace hsa
