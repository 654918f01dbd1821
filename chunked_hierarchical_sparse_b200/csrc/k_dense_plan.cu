// k_dense_plan.cu -- work lists of packed prompts, and joining the decode partials.
#include <type_traits>

#include "dense.cuh"

namespace hsa {
namespace dense {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;

// One block.  A tile's cost is the number of keys (or rows) it meets, which is
// linear in its index, so a counting sort over kBins index classes puts the
// dearest first; inside a class the order does not matter (and is not fixed:
// every tile is computed by itself, so it changes no result).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int32_t *cu, int n_seq, int L, int tok,
                                                            int first_dear, int4 *plan, int32_t *plan_n,
                                                            DevStatus *ds, int clear) {
    __shared__ int hist[kBins];
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    hist[tid] = 0;
    if (tid == 0) bad = 0;
    dependency_wait();
    dependents_may_start();
    if (clear && tid < (int)kWsHeader / 4) reinterpret_cast<int32_t *>(ds)[tid] = 0;
    __syncthreads();
    for (int s = tid; s < n_seq; s += kPlanThreads) {
        const int a = cu[s], b = cu[s + 1];
        if (a < 0 || b < a || b > L) {
            bad = 1;
            report(ds, HSA_ERR_DEVICE_CHECK, kKDense, s, b);
        }
    }
    __syncthreads();
    if (bad) {
        if (tid == 0) *plan_n = 0;
        return;
    }
    const int top = (L + tok - 1) / tok;  // tiles of the longest possible sequence
    auto bin = [&](int i, int n) {        // 0: dearest
        const int64_t rank = first_dear ? n - 1 - i : i;
        return kBins - 1 - (int)(rank * kBins / max(top, 1));
    };
    for (int s = warp; s < n_seq; s += kPlanThreads / 32) {
        const int n = (cu[s + 1] - cu[s] + tok - 1) / tok;
        for (int i = lane; i < n; i += 32) atomicAdd(&hist[bin(i, n)], 1);
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
    if (tid == kPlanThreads - 1) *plan_n = hist[tid] + own;
    __syncthreads();
    for (int s = warp; s < n_seq; s += kPlanThreads / 32) {
        const int a = cu[s], len = cu[s + 1] - a, n = (len + tok - 1) / tok;
        for (int i = lane; i < n; i += 32) plan[atomicAdd(&hist[bin(i, n)], 1)] = make_int4(a, len, i, 0);
    }
}

// Joining the partials of a (sequence, head) row with weights e^{lse_i - max}.  W of the
// block's 8 warps share a row, each taking every W-th slot (a warp reads a slot's d values
// as one line), their sums added in a fixed order.  Latency-bound: with many slots per row
// W = 8 keeps enough reads in flight (16 x 16 rows of 64 slots: 3 us of the 16.7 us step),
// with few of them and many rows a warp per row is enough.
constexpr int kJoinWarps = 8;
constexpr int kJoinMany = 8;  // slots from which a block takes one row

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
    if (a.pre_slots + a.suf_slots >= kJoinMany)
        return launch_next(behind, combine_kernel<T, D, kJoinWarps>, rows, kJoinWarps * 32, 0, st, a);
    return launch_next(behind, combine_kernel<T, D, 1>, (rows + kJoinWarps - 1) / kJoinWarps, kJoinWarps * 32, 0, st, a);
}

}  // namespace

cudaError_t launch_plan(const int32_t *cu, int n_seq, int L, int tok, bool first_dear, int4 *plan, int32_t *plan_n,
                        DevStatus *ds, bool clear, cudaStream_t st) {
    return launch_next(!clear, plan_kernel, 1, kPlanThreads, 0, st, cu, n_seq, L, tok, (int)first_dear, plan, plan_n, ds,
                       (int)clear);
}

cudaError_t launch_combine(const Args &a, int d, bool bf16, cudaStream_t st) {
    if (bf16) return d == 128 ? combine<__nv_bfloat16, 128>(a, st) : combine<__nv_bfloat16, 64>(a, st);
    return d == 128 ? combine<float, 128>(a, st) : combine<float, 64>(a, st);
}

}  // namespace dense
}  // namespace hsa
