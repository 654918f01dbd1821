// k_dense_plan.cu -- work lists of packed prompts, and joining the decode partials.
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
                                                            DevStatus *ds) {
    __shared__ int hist[kBins];
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    hist[tid] = 0;
    if (tid == 0) bad = 0;
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

// One warp per (sequence, head): the partials of its slots weighted by e^{lse_i - max}.
template <typename T, int D>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ Args a) {
    constexpr int E = D / 32;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rows = a.B * a.hq;
    if (row >= rows) return;
    const int len = a.cap > 0 ? min(max(a.lens[row / a.hq], 0), a.cap) : 0;
    const int n_suf = a.suf_sub > 0 ? (len + a.suf_sub - 1) / a.suf_sub : 0;
    const int n = a.pre_slots + n_suf;
    float m = a.off_by_one ? 0.f : -INFINITY;  // off-by-one: the added 1 is a logit of 0
    for (int i = lane; i < n; i += 32) m = fmaxf(m, a.plse[(size_t)i * rows + row]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mm = m == -INFINITY ? 0.f : m;
    float z = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float w = __expf(a.plse[(size_t)i * rows + row] - mm);
        z += w;
        const float *p = a.po + ((size_t)i * rows + row) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += w * p[e];
    }
    if (a.off_by_one) z += __expf(-mm);
    const float r = z > 0.f ? 1.f / z : 0.f;  // no key at all: output 0, lse = log 0
    T *o = static_cast<T *>(a.o) + (size_t)row * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) Elem<T>::store(o + e, acc[e] * r);
    if (a.lse && lane == 0) a.lse[row] = mm + logf(z);
}

}  // namespace

cudaError_t launch_plan(const int32_t *cu, int n_seq, int L, int tok, bool first_dear, int4 *plan, int32_t *plan_n,
                        DevStatus *ds, cudaStream_t st) {
    plan_kernel<<<1, kPlanThreads, 0, st>>>(cu, n_seq, L, tok, first_dear, plan, plan_n, ds);
    return cudaGetLastError();
}

cudaError_t launch_combine(const Args &a, int d, bool bf16, cudaStream_t st) {
    const int grid = (int)ceil_div((int64_t)a.B * a.hq, 4);
    if (bf16 && d == 128) combine_kernel<__nv_bfloat16, 128><<<grid, 128, 0, st>>>(a);
    else if (bf16) combine_kernel<__nv_bfloat16, 64><<<grid, 128, 0, st>>>(a);
    else if (d == 128) combine_kernel<float, 128><<<grid, 128, 0, st>>>(a);
    else combine_kernel<float, 64><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dense
}  // namespace hsa
