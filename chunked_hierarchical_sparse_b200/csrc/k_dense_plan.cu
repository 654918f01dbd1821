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

// Joining the partials of a (sequence, head) row: weights e^{lse_i - max}, one block per
// row, its warps taking every kJoinWarps-th slot (a warp reads a slot's d values as one
// 512-byte line), their sums added in a fixed order.  Latency-bound: the slots of a row are
// spread over as many warps as the reads need to be in flight together.
constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) combine_kernel(const __grid_constant__ Args a) {
    constexpr int E = D / 32;
    typedef typename std::conditional<E == 4, float4, float2>::type Vec;
    __shared__ float part[kJoinWarps][D + 1];
    const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.B * a.hq;
    dependency_wait();
    const int len = a.cap > 0 ? min(max(a.lens[row / a.hq], 0), a.cap) : 0;
    const int n = a.pre_slots + (a.suf_sub > 0 ? (len + a.suf_sub - 1) / a.suf_sub : 0);
    float m = a.off_by_one ? 0.f : -INFINITY;  // off-by-one: the added 1 is a logit of 0
    for (int i = lane; i < n; i += 32) m = fmaxf(m, a.plse[i * rows + row]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mm = m == -INFINITY ? 0.f : m;
    float z = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += kJoinWarps) {
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
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
    if (lane == 0) part[warp][D] = z;
    __syncthreads();
    if (threadIdx.x >= D) return;
    float s = 0.f;
    z = a.off_by_one ? __expf(-mm) : 0.f;
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
        s += part[i][threadIdx.x];
        z += part[i][D];
    }
    // no key at all: output 0, lse = log 0; a NaN stays one
    Elem<T>::store(static_cast<T *>(a.o) + (int64_t)row * D + threadIdx.x, z == 0.f ? 0.f : s / z);
    if (a.lse && threadIdx.x == 0) a.lse[row] = mm + logf(z);
}

}  // namespace

cudaError_t launch_plan(const int32_t *cu, int n_seq, int L, int tok, bool first_dear, int4 *plan, int32_t *plan_n,
                        DevStatus *ds, bool clear, cudaStream_t st) {
    return launch_next(!clear, plan_kernel, 1, kPlanThreads, 0, st, cu, n_seq, L, tok, (int)first_dear, plan, plan_n, ds,
                       (int)clear);
}

cudaError_t launch_combine(const Args &a, int d, bool bf16, cudaStream_t st) {
    const int grid = a.B * a.hq;
    const bool behind = pre_items(a) + suf_items(a) > 0;  // else it is the call's first kernel
    auto go = [&](auto *kernel) { return launch_next(behind, kernel, grid, kJoinWarps * 32, 0, st, a); };
    if (bf16) return d == 128 ? go(combine_kernel<__nv_bfloat16, 128>) : go(combine_kernel<__nv_bfloat16, 64>);
    return d == 128 ? go(combine_kernel<float, 128>) : go(combine_kernel<float, 64>);
}

}  // namespace dense
}  // namespace hsa
