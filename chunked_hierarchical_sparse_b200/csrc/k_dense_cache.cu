// k_dense_cache.cu -- the own-cache part of the shared-prefix decode step (bf16).
//
// Mathematics.  One new token of a sequence: its G query heads of a group against that
// group's lens[b] cached keys, S = Q K^T, online softmax, O += P V; the partial
// (O / l, lse) of each range of keys goes to its slot.
//
// Bound: HBM -- every key and value is read once, for 4 G d FLOP per 4 d bytes.  With
// G <= 16 rows per key a 128-row tcgen05 tile would be 7/8 padding or more, its two
// products and the softmax of one row per thread take 2.2 us per 128 KB of cache, and
// nothing overlaps the ends of a sequence: measured 81 us for 133 MB (256 sequences of
// 1024 tokens on average).  So warp-level MMAs (m16n8k16, the G rows padded to 16):
// a block of 4 warps walks its keys in stages of 64 loaded by TMA (a fifth warp), warp w
// taking keys 16 w .. 16 w + 15 of each with its own running maximum, sum and output in
// registers, so that the warps never wait for one another; their four states are joined
// at the end.  Three blocks per SM with 64 KB of stages each keep 192 KB in flight and
// cover one another's ends (two of 96 KB: 112 instead of 106 us for a step of 256
// sequences, 32K tokens shared and up to 2K of their own).
#include <algorithm>

#include "dense_tc.cuh"

namespace hsa {
namespace dense {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kKeys = 64;  // keys per stage

template <int D> struct Smem {
    static constexpr int NH = D / 64;
    static constexpr int HALF = kKeys * 128;           // 64 keys x 64 columns
    static constexpr int TILE = NH * HALF;
    static constexpr int ST = D == 128 ? 2 : 4;
    static constexpr int OFF_STATE = ST * 2 * TILE;    // m, l of the warps' 16 rows
    static constexpr int OFF_BAR = OFF_STATE + 2 * kWarps * 16 * 4;
    static constexpr int OFF_MISC = OFF_BAR + 128;
    static constexpr int ALLOC = OFF_MISC + 16 + 1024;
};
static_assert(kWarps * 16 * 128 * 4 <= Smem<128>::OFF_STATE && kWarps * 16 * 64 * 4 <= Smem<64>::OFF_STATE,
              "the warps' outputs are joined in the stages' memory");
static_assert(3 * (Smem<128>::ALLOC + 1024) <= 233472 && 3 * (Smem<64>::ALLOC + 1024) <= 233472, "three blocks per SM");

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                         const __grid_constant__ CUtensorMap tm_v,
                                                         const __grid_constant__ Args a, int clear, uint64_t wait_ns) {
    using L = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *state = reinterpret_cast<float *>(sm + L::OFF_STATE);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR), *empty = full + L::ST;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blocks in item order: the ranges of one sequence's groups are neighbours
    const int g = blockIdx.x % a.hkv, r = blockIdx.x / a.hkv, b = r % a.B, s = r / a.B;
    if (clear && blockIdx.x == 0 && threadIdx.x == 0) *a.ds = DevStatus{};
    // Its inputs are the caller's, so its blocks work beside the prefix kernel's.  Only the last
    // waits for that kernel, at its end: this one is then complete when both are, which is what
    // the join kernel waits for (a block that waited would keep its SM meanwhile).
    dependents_may_start();
    const bool last_block = blockIdx.x == gridDim.x - 1;
    const int key0 = s * a.suf_sub, nkeys = min(a.suf_sub, own_len(a, b) - key0);
    if (nkeys <= 0) {
        if (last_block) dependency_wait();
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::ST; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], kWarps); }
        *abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();
    const int stages = (nkeys + kKeys - 1) / kKeys;
    auto wait = [&](uint64_t *x, uint32_t par, int role) { return warp_wait(x, par & 1, wait_ns, abort_flag, a.ds, role); };
    bool ok = true;
    float o[D / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    if (warp == kWarps) {
        // ============================================================ loads
        const int plane = b * a.hkv + g;
        int j = 0;
        for (; j < stages; ++j) {
            const int st = j % L::ST;
            if (j >= L::ST && !(ok = wait(&empty[st], j / L::ST - 1, 31))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[st], 2 * L::TILE);
#pragma unroll
                for (int h = 0; h < L::NH; ++h) {
                    tma_load_3d(sm + st * 2 * L::TILE + h * L::HALF, &tm_k, h * 64, key0 + j * kKeys, plane, &full[st]);
                    tma_load_3d(sm + st * 2 * L::TILE + L::TILE + h * L::HALF, &tm_v, h * 64, key0 + j * kKeys, plane, &full[st]);
                }
            }
        }
        if (lane == 0) land(full, j, L::ST);
        __syncwarp();
    } else {
        // ============================================================ 16 keys of every stage
        const int qr = lane >> 2, qc = (lane & 3) * 2;
        uint32_t q[D / 16][4];  // the group's rows as the first operand; rows >= G are zeros
        {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                                   ((int64_t)b * a.hq + g * a.G) * D);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = qr + (i & 1) * 8, col = ks * 16 + qc + (i >> 1) * 8;
                    q[ks][i] = row < a.G ? p[(row * D + col) / 2] : 0u;
                }
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        // ldmatrix row addresses (16-byte chunk c of row r is stored at c ^ (r & 7))
        const int mi = lane >> 3, mr = lane & 7;
        const int krow = warp * 16 + (mi >> 1) * 8 + mr, vrow = warp * 16 + (mi & 1) * 8 + mr;
        const uint32_t kbase = smem_u32(sm) + krow * 128, vbase = smem_u32(sm) + L::TILE + vrow * 128;
        const float c = a.scale_log2;
        for (int j = 0; j < stages; ++j) {
            const int st = j % L::ST;
            if (!(ok = wait(&full[st], j / L::ST, 32))) break;
            const int left = nkeys - j * kKeys - warp * 16;  // keys of this warp's 16 that exist
            if (left > 0) {
                float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t kf[4];
                    const int ch = (ks & 3) * 2 + (mi & 1);
                    ldm4(kf, kbase + st * 2 * L::TILE + (ks >> 2) * L::HALF + ((ch ^ mr) << 4));
                    mma16(x[0], q[ks], kf[0], kf[1]);
                    mma16(x[1], q[ks], kf[2], kf[3]);
                }
                uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // pairs of keys of the second product that exist
                if (left < 16) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (t * 8 + qc + (i & 1) >= left) x[t][i] = -INFINITY;
                    keep0 = (qc < left ? 0xffffu : 0u) | (qc + 1 < left ? 0xffff0000u : 0u);
                    keep1 = (qc + 8 < left ? 0xffffu : 0u) | (qc + 9 < left ? 0xffff0000u : 0u);
                }
                float mx[2];
                bool moved = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // rows qr and qr + 8
                    float v = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1])) * c;
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    mx[i] = fmaxf(m[i], v);
                    moved |= mx[i] > m[i];
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float f = mx[i] > m[i] ? ex2(m[i] - mx[i]) : 1.f;
                        m[i] = mx[i];
                        l[i] *= f;
#pragma unroll
                        for (int e = 0; e < D / 8; ++e) {
                            o[e][2 * i] *= f;
                            o[e][2 * i + 1] *= f;
                        }
                    }
                }
                uint32_t p[4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mm = m[i] == -INFINITY ? 0.f : m[i];
                        const float e0 = ex2(fmaf(x[t][2 * i], c, -mm)), e1 = ex2(fmaf(x[t][2 * i + 1], c, -mm));
                        l[i] += e0 + e1;
                        p[t * 2 + i] = bf16_pair(e0, e1);
                    }
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    uint32_t vf[4];
                    const int ch = (e & 3) * 2 + (mi >> 1);
                    ldm4t(vf, vbase + st * 2 * L::TILE + (e >> 2) * L::HALF + ((ch ^ mr) << 4));
                    // values behind the last key may be anything: 0 * NaN is NaN
                    mma16(o[2 * e], p, vf[0] & keep0, vf[1] & keep1);
                    mma16(o[2 * e + 1], p, vf[2] & keep0, vf[3] & keep1);
                }
            }
            __syncwarp();
            mbar_arrive_lane0(&empty[st], lane);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // the four lanes of a row hold parts of its sum
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
    }
    // ================================================================ joining the warps
    __syncthreads();  // every stage has been read; their memory now holds the outputs
    const bool good = *abort_flag == 0;
    float *out = reinterpret_cast<float *>(sm);
    if (warp < kWarps) {
        const int qr = lane >> 2, qc = (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = qr + 8 * i;
            if ((lane & 3) == 0) {
                state[warp * 16 + row] = m[i];
                state[kWarps * 16 + warp * 16 + row] = l[i];
            }
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
                *reinterpret_cast<float2 *>(out + (warp * 16 + row) * D + e * 8 + qc) = make_float2(o[e][2 * i], o[e][2 * i + 1]);
        }
    }
    __syncthreads();
    if (good) {
        const int64_t rows = (int64_t)a.B * a.hq, first = (a.pre_slots + s) * rows + (int64_t)b * a.hq + g * a.G;
        for (int i = threadIdx.x; i < a.G * (D / 4); i += kThreads) {
            const int row = i / (D / 4), col = (i % (D / 4)) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, state[w * 16 + row]);
            const float mm = top == -INFINITY ? 0.f : top;
            float z = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(state[w * 16 + row] - mm);
                const float4 x = *reinterpret_cast<const float4 *>(out + (w * 16 + row) * D + col);
                z += f * state[kWarps * 16 + w * 16 + row];
                v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
            }
            const float inv = z == 0.f ? 0.f : 1.f / z;  // a NaN stays one
            *reinterpret_cast<float4 *>(a.po + (first + row) * D + col) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            if (col == 0) a.plse[first + row] = (mm + log2f(z)) * kLn2;
        }
    }
    if (last_block) dependency_wait();
}

template <int D> cudaError_t launch(const Args &a, bool first, cudaStream_t st) {
    CUtensorMap mk, mv;
    const uint64_t planes = (uint64_t)a.B * a.hkv;
    if (!make_map3(&mk, a.k[1], D, a.cap, D, planes, a.plane[1], kKeys, 1) ||
        !make_map3(&mv, a.v[1], D, a.cap, D, planes, a.plane[1], kKeys, 1))
        return cudaErrorInvalidValue;
    const cudaError_t e = set_smem_once((const void *)cache_kernel<D>, Smem<D>::ALLOC);
    if (e != cudaSuccess) return e;
    return launch_next(!first, cache_kernel<D>, a.hkv * a.B * a.suf_slots, kThreads, Smem<D>::ALLOC, st, 1, mk, mv, a,
                       (int)first, wait_limit_ns());
}

}  // namespace

cudaError_t launch_cache(const Args &a, int d, bool first, cudaStream_t st) {
    return d == 128 ? launch<128>(a, first, st) : launch<64>(a, first, st);
}

}  // namespace dense
}  // namespace hsa
