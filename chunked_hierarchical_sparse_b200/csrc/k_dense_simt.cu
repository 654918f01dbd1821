// k_dense_simt.cu -- dense attention and its backward in fp32, on the CUDA cores.
//
// A block takes one tile of 64 (token, head) rows of a group and walks the keys
// in tiles of 64 (the key-major backward kernel: a tile of 64 keys, walking the
// rows).  Every product of a tile pair is a 64 x 64 (or 64 x d) fp32 outer-product
// loop out of shared memory: thread (ty, tx) of 16 x 16 owns rows ty + 16 i and
// columns tx + 16 j, so that the lanes of a warp read different rows of a padded
// tile (stride d + 4 floats: 16-byte reads without bank conflicts).  Softmax state
// (running maximum, sum, output) stays in fp32 registers.
//
// Few items (small problems are what fp32 is for) are shared by a cluster of C blocks, each
// taking every C-th tile of the walk; their states are joined through distributed shared
// memory, in rank order, each block finishing 64 / C of the rows.  No partial goes through
// global memory and no second kernel is needed.
//
// Bound: FFMA issue fed by shared memory (8 16-byte reads per 64 FMAs); the tiles
// of keys come from L2 and cost little beside it.
#include <cooperative_groups.h>

#include "dense.cuh"

namespace hsa {
namespace dense {

namespace {

namespace cg = cooperative_groups;

constexpr int kT = kSimtRows;
constexpr int kThr = 256;
constexpr int kPS = kT + 4;  // row stride of a 64 x 64 tile

// 64 rows of d values into a padded tile; row r comes from src(r) (null: zeros)
template <int D, typename F> __device__ __forceinline__ void load_tile(float *dst, F &&src) {
    constexpr int V = D / 4;
    for (int i = threadIdx.x; i < kT * V; i += kThr) {
        const int r = i / V, c = (i % V) * 4;
        const float *p = src(r);
        const float4 x = p ? *reinterpret_cast<const float4 *>(p + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + c) = x;
    }
}

// acc[i][j] = A[ty + 16 i] . B[tx + 16 j] over d: even and odd columns of d are summed apart, two
// FMAs an instruction
template <int D> __device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float *A, const float *B, int ty, int tx) {
    float2 s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * (D + 4) + c);
            y[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * (D + 4) + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), s[i][j]);
                s[i][j] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}

// acc[i][64 h + 4 tx + e] += sum_n P[ty + 16 i][n] B[n][64 h + 4 tx + e]
template <int D>
__device__ __forceinline__ void accum_tile(float (&acc)[4][D / 16], const float *P, const float *B, int ty, int tx) {
#pragma unroll 2
    for (int n = 0; n < kT; n += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(P + (ty + 16 * i) * kPS + n);
            p[i][0] = v.x; p[i][1] = v.y; p[i][2] = v.z; p[i][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const float4 b = *reinterpret_cast<const float4 *>(B + (n + e) * (D + 4) + h * 64 + tx * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 pp = make_float2(p[i][e], p[i][e]);
                    float2 *y = reinterpret_cast<float2 *>(&acc[i][h * 4]);
                    y[0] = fma2(pp, make_float2(b.x, b.y), y[0]);
                    y[1] = fma2(pp, make_float2(b.z, b.w), y[1]);
                }
            }
    }
}

__device__ __forceinline__ float row_max16(float x) {  // over the 16 lanes that share a row
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum16(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

// a thread's part of a 64 x d accumulator into a padded tile
template <int D> __device__ __forceinline__ void put_tile(float *dst, const float (&acc)[4][D / 16], int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<float4 *>(dst + (ty + 16 * i) * (D + 4) + h * 64 + tx * 4) =
                make_float4(acc[i][h * 4], acc[i][h * 4 + 1], acc[i][h * 4 + 2], acc[i][h * 4 + 3]);
}
__device__ __forceinline__ void add4(float4 &v, float4 x, float f) {
    v.x = fmaf(f, x.x, v.x); v.y = fmaf(f, x.y, v.y); v.z = fmaf(f, x.z, v.z); v.w = fmaf(f, x.w, v.w);
}
// Sums a tile that every block of the cluster holds at the same place, in rank order; the
// calling block's 64 / C rows of it go, scaled, to dst(row) + column.
template <int D, int THREADS, typename F>
__device__ __forceinline__ void add_tiles(const cg::cluster_group &cl, float *tile, int rows, float scale, F &&dst) {
    const int C = cl.num_blocks(), rank = cl.block_rank();
    for (int i = threadIdx.x; i < kT / C * (D / 4); i += THREADS) {
        const int r = rank * (kT / C) + i / (D / 4), c = i % (D / 4) * 4;
        if (r >= rows) break;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < C; ++q) add4(v, *reinterpret_cast<const float4 *>(cl.map_shared_rank(tile, q) + r * (D + 4) + c), 1.f);
        store4(dst(r) + c, make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale));
    }
}

// (the kernels here keep no counters in the header and report nothing, so any block may clear it)
__device__ __forceinline__ void clear_header(DevStatus *ds) {
    if (threadIdx.x < kHeaderWords) reinterpret_cast<int32_t *>(ds)[threadIdx.x] = 0;
}

template <int D>
__global__ void __launch_bounds__(kThr, D == 64 ? 2 : 1) fwd_simt_kernel(const __grid_constant__ Args a) {
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + kT * (D + 4), *V = K + kT * (D + 4), *P = V + kT * (D + 4);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    Item it;
    dependency_wait();
    dependents_may_start();
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks(), item = blockIdx.x / C;
    if (!a.plan && blockIdx.x == 0) clear_header(a.ds);
    if (item >= item_count(a) || !get_item(a, item, it)) return;  // (the whole cluster)
    const int rows = it.ntok * a.G;
    const float *q = static_cast<const float *>(a.q);
    const float *kp = static_cast<const float *>(a.k[it.src]) + it.plane * a.plane[it.src] + (int64_t)it.key0 * D;
    const float *vp = static_cast<const float *>(a.v[it.src]) + it.plane * a.plane[it.src] + (int64_t)it.key0 * D;
    auto row_index = [&](int r) { return ((int64_t)it.tok0 + r / a.G) * a.hq + it.g * a.G + r % a.G; };
    load_tile<D>(Q, [&](int r) -> const float * { return r < rows ? q + row_index(r) * D : nullptr; });
    float m[4], z[4], o[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        z[i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[i][c] = 0.f;
    }
    for (int n0 = rank * kT; n0 < it.nkeys; n0 += C * kT) {
        __syncthreads();
        auto key = [&](const float *p, int r) -> const float * { return n0 + r < it.nkeys ? p + (int64_t)(n0 + r) * D : nullptr; };
        load_tile<D>(K, [&](int r) { return key(kp, r); });
        load_tile<D>(V, [&](int r) { return key(vp, r); });
        __syncthreads();
        float s[4][4];
        dot_tile<D>(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = it.off + (ty + 16 * i) / a.G;  // this row's last visible key
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 16 * j;
                s[i][j] = n < it.nkeys && n <= last ? s[i][j] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
            mx = fmaxf(m[i], row_max16(mx));
            const float ms = mx == -INFINITY ? 0.f : mx;
            const float f = exp2f(m[i] - ms);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - ms);
                sum += p;
                P[(ty + 16 * i) * kPS + tx + 16 * j] = p;
            }
            z[i] = z[i] * f + row_sum16(sum);
            m[i] = mx;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) o[i][c] *= f;
        }
        __syncthreads();
        accum_tile<D>(o, P, V, ty, tx);
    }
    // joining the cluster: outputs and statistics in the tiles' memory
    float *st = P;  // m[64], z[64]
    __syncthreads();
    put_tile<D>(K, o, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (tx == 0) {
            st[ty + 16 * i] = m[i];
            st[kT + ty + 16 * i] = z[i];
        }
    cl.sync();
    const int64_t nrow = (int64_t)a.B * a.hq;  // decode rows per slot
    for (int i = threadIdx.x; i < kT / C * (D / 4); i += kThr) {
        const int r = rank * (kT / C) + i / (D / 4), c = i % (D / 4) * 4;
        if (r >= rows) break;
        float mm = -INFINITY;
        for (int q2 = 0; q2 < C; ++q2) mm = fmaxf(mm, cl.map_shared_rank(st, q2)[r]);
        if (mm == -INFINITY) mm = 0.f;
        float zz = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q2 = 0; q2 < C; ++q2) {
            const float *rs = cl.map_shared_rank(st, q2);
            const float f = exp2f(rs[r] - mm);
            zz += f * rs[kT + r];
            add4(v, *reinterpret_cast<const float4 *>(cl.map_shared_rank(K, q2) + r * (D + 4) + c), f);
        }
        float f = 1.f;
        if (!a.decode && a.off_by_one) {  // the added 1 is a logit of 0
            const float top = fmaxf(mm, 0.f);
            f = exp2f(mm - top);
            zz = zz * f + exp2f(-top);
            mm = top;
        }
        const float inv = zz > 0.f ? f / zz : (zz == 0.f ? 0.f : zz);
        const float l = (mm + log2f(zz)) * 0.6931471805599453f;
        const int64_t ri = row_index(r);
        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if (a.decode) store4(a.po + (it.slot * nrow + ri) * D + c, v);
        else store4(static_cast<float *>(a.o) + ri * D + c, v);
        if (c == 0) {
            if (a.decode) a.plse[it.slot * nrow + ri] = l;
            else if (a.lse) a.lse[ri] = l;
        }
    }
    cl.sync();  // no block leaves while another reads its memory
}

// delta[row] = dO . o, one warp per (token, head) row; `header`: to be cleared (null: by a kernel before).
// Packed (`cu`; the plan has looked at it, and has no items where it does not rise): the sequences' rows only.
template <int D>
__global__ void __launch_bounds__(256) delta_kernel(const float *o, const float *dO, float *delta, int64_t rows, DevStatus *header,
                                                    const int32_t *cu, int n_seq, int hq, const int32_t *plan_n) {
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    dependency_wait();
    dependents_may_start();
    if (header && blockIdx.x == 0) clear_header(header);
    if (r >= rows) return;
    if (cu && (*plan_n == 0 || r < (int64_t)cu[0] * hq || r >= (int64_t)cu[n_seq] * hq)) return;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < D; c += 128) {
        if (c + lane * 4 < D) {
            const float4 x = *reinterpret_cast<const float4 *>(o + r * D + c + lane * 4), y = *reinterpret_cast<const float4 *>(dO + r * D + c + lane * 4);
            s += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
    }
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) delta[r] = s;
}

// The backward's two kernels run two groups of 256 threads: one computes S and p, the other dP, on
// different products at the same time.  A step of a small problem is latency, and 8 warps hide little
// of it: one prompt of 1K tokens, 4 heads in a group, 209 us with one group doing both, 150 with two.
// (d = 64, 8K tokens, two such blocks per SM: 15.4 ms, now 16.4; d = 128, 16 x 1K tokens: 9.1, now 7.8.)  Masked places are zeros in both.  The next tiles wait in registers meanwhile.
constexpr int kThr2 = 2 * kThr;

// A 64 x D tile on its way from global memory to a padded one: each thread's part
template <int D> struct Fetch {
    static constexpr int V = D / 4, N = kT * V / kThr2;
    float4 x[N];
    template <typename F> __device__ __forceinline__ void load(F &&src) {  // row r comes from src(r) (null: zeros)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * kThr2;
            const float *p = src(at / V);
            x[i] = p ? *reinterpret_cast<const float4 *>(p + at % V * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void store(float *dst) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = threadIdx.x + i * kThr2;
            store4(dst + at / V * (D + 4) + at % V * 4, x[i]);
        }
    }
};

// acc[i][] += sum_n P[ty + 16 i][n] B[n][columns of tx].  W columns of B's D: 4 per thread of every 64
// (W = 32: 2).
template <int D, int W>
__device__ __forceinline__ void accum2(float2 (&acc)[4][W / 32], const float *P, const float *B, int ty, int tx) {
#pragma unroll 1
    for (int n = 0; n < kT; n += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(P + (ty + 16 * i) * kPS + n);
            p[i][0] = v.x; p[i][1] = v.y; p[i][2] = v.z; p[i][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 b[W / 32];
            const float *row = B + (n + e) * (D + 4);
            if constexpr (W == 32) {
                b[0] = *reinterpret_cast<const float2 *>(row + tx * 2);
            } else {
#pragma unroll
                for (int h = 0; h < W / 64; ++h) {
                    const float4 x = *reinterpret_cast<const float4 *>(row + h * 64 + tx * 4);
                    b[2 * h] = make_float2(x.x, x.y);
                    b[2 * h + 1] = make_float2(x.z, x.w);
                }
            }
#pragma unroll
            for (int h = 0; h < W / 32; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][h] = fma2(make_float2(p[i][e], p[i][e]), b[h], acc[i][h]);
        }
    }
}
// the accumulator's W columns into a padded tile
template <int D, int W> __device__ __forceinline__ void put2(float *dst, const float2 (&acc)[4][W / 32], int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float *row = dst + (ty + 16 * i) * (D + 4);
        if constexpr (W == 32) {
            *reinterpret_cast<float2 *>(row + tx * 2) = acc[i][0];
        } else {
#pragma unroll
            for (int h = 0; h < W / 64; ++h)
                store4(row + h * 64 + tx * 4, make_float4(acc[i][2 * h].x, acc[i][2 * h].y, acc[i][2 * h + 1].x, acc[i][2 * h + 1].y));
        }
    }
}

// dq of a row tile: walks the keys, dq += (p (dO.v - delta)) k
template <int D>
__global__ void __launch_bounds__(kThr2, 1) bwd_dq_simt_kernel(const __grid_constant__ BwdArgs b) {
    extern __shared__ float sm[];
    const Args &a = b.a;
    float *Q = sm, *G = Q + kT * (D + 4), *K = G + kT * (D + 4), *V = K + kT * (D + 4), *S = V + kT * (D + 4);
    const int grp = threadIdx.x / kThr, ty = threadIdx.x % kThr >> 4, tx = threadIdx.x & 15;
    Item it;
    dependency_wait();
    dependents_may_start();
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks(), item = blockIdx.x / C;
    if (item >= item_count(a) || !get_item(a, item, it)) return;
    const int rows = it.ntok * a.G;
    const int64_t pl = it.plane * a.plane[0] + (int64_t)it.key0 * D;
    const float *kp = static_cast<const float *>(a.k[0]) + pl, *vp = static_cast<const float *>(a.v[0]) + pl;
    auto row_index = [&](int r) { return ((int64_t)it.tok0 + r / a.G) * a.hq + it.g * a.G + r % a.G; };
    Fetch<D> fk, fv;
    auto fetch = [&](int n0) {  // (behind the last key: zeros)
        auto key = [&](const float *p, int r) -> const float * { return n0 + r < it.nkeys ? p + (int64_t)(n0 + r) * D : nullptr; };
        fk.load([&](int r) { return key(kp, r); });
        fv.load([&](int r) { return key(vp, r); });
    };
    {
        auto row = [&](const void *p, int r) -> const float * { return r < rows ? static_cast<const float *>(p) + row_index(r) * D : nullptr; };
        fk.load([&](int r) { return row(a.q, r); });
        fv.load([&](int r) { return row(b.dO, r); });
        fk.store(Q);
        fv.store(G);
    }
    fetch(rank * kT);
    float st[4];  // group 0: lse, 1: delta
    float2 dq[4][D / 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
        if (grp == 0) st[i] = r < rows ? b.lse[row_index(r)] * 1.4426950408889634f : INFINITY;
        else st[i] = r < rows ? b.delta[row_index(r)] : 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) dq[i][c] = make_float2(0.f, 0.f);
    }
    for (int n0 = rank * kT; n0 < it.nkeys; n0 += C * kT) {
        __syncthreads();
        fk.store(K);
        fv.store(V);
        __syncthreads();
        if (n0 + C * kT < it.nkeys) fetch(n0 + C * kT);
        float s[4][4];
        dot_tile<D>(s, grp ? G : Q, grp ? V : K, ty, tx);
        // each group gives the other half of its values and multiplies the other half
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int last = it.off + (ty + 16 * i) / a.G;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 16 * j;
                const float x = grp ? s[i][j] - st[i] : exp2f(s[i][j] * a.scale_log2 - st[i]);
                s[i][j] = n < it.nkeys && n <= last ? x : 0.f;
                if (j / 2 != grp) S[(ty + 16 * i) * kPS + tx + 16 * j] = s[i][j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float *y = S + (ty + 16 * i) * kPS + tx + 16 * j + 32 * grp;
                *y *= grp ? s[i][j + 2] : s[i][j];
            }
        __syncthreads();
        accum2<D, D / 2>(dq, S, K + grp * (D / 2), ty, tx);  // half of the columns each
    }
    __syncthreads();
    put2<D, D / 2>(K + grp * (D / 2), dq, ty, tx);
    cl.sync();
    add_tiles<D, kThr2>(cl, K, rows, a.scale, [&](int r) { return static_cast<float *>(b.dq) + row_index(r) * D; });
    cl.sync();
}

// dk, dv of a tile of keys: walks the row tiles that see it, all heads of the group
template <int D>
__global__ void __launch_bounds__(kThr2, 1) bwd_dkv_simt_kernel(const __grid_constant__ BwdArgs b) {
    extern __shared__ float sm[];
    const Args &a = b.a;
    float *K = sm, *V = K + kT * (D + 4), *Q = V + kT * (D + 4), *G = Q + kT * (D + 4), *P = G + kT * (D + 4),
          *S = P + kT * kPS;
    const int grp = threadIdx.x / kThr, ty = threadIdx.x % kThr >> 4, tx = threadIdx.x & 15;
    KeyItem it;
    dependency_wait();
    dependents_may_start();
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks(), item = blockIdx.x / C;
    if (item >= key_item_count(b) || !get_key_item(b, item, kT, it)) return;
    const int64_t pl = it.plane * a.plane[0] + (int64_t)(it.start + it.n0) * D;
    Fetch<D> fq, fg;
    auto row_index = [&](int t0, int r) { return (it.row0 + t0 + r / a.G) * a.hq + it.g * a.G + r % a.G; };
    auto rows_at = [&](int t0) { return min(a.tok, it.len - t0) * a.G; };
    auto fetch = [&](int t0) {
        const int rows = rows_at(t0);
        auto row = [&](const void *p, int r) -> const float * { return r < rows ? static_cast<const float *>(p) + row_index(t0, r) * D : nullptr; };
        fq.load([&](int r) { return row(a.q, r); });
        fg.load([&](int r) { return row(b.dO, r); });
    };
    {
        auto key = [&](const void *p, int r) -> const float * { return r < it.nkeys ? static_cast<const float *>(p) + pl + r * D : nullptr; };
        fq.load([&](int r) { return key(a.k[0], r); });
        fg.load([&](int r) { return key(a.v[0], r); });
        fq.store(K);
        fg.store(V);
    }
    const int t_first = it.n0 + rank * a.tok;
    if (t_first < it.len) fetch(t_first);
    float2 acc[4][D / 32];  // group 0: dv, 1: dk
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[i][c] = make_float2(0.f, 0.f);
    for (int t0 = t_first; t0 < it.len; t0 += C * a.tok) {
        const int rows = rows_at(t0);
        __syncthreads();
        fq.store(Q);
        fg.store(G);
        __syncthreads();
        float st[4];  // group 0: lse, 1: delta, of the rows (columns of the tile)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = tx + 16 * j;
            if (grp == 0) st[j] = r < rows ? b.lse[row_index(t0, r)] * 1.4426950408889634f : INFINITY;
            else st[j] = r < rows ? b.delta[row_index(t0, r)] : 0.f;
        }
        if (t0 + C * a.tok < it.len) fetch(t0 + C * a.tok);
        float s[4][4];  // keys down, rows across: the sums below read P and S along their rows
        dot_tile<D>(s, grp ? V : K, grp ? G : Q, ty, tx);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = tx + 16 * j, tok = t0 + r / a.G - it.n0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = ty + 16 * i;
                const float x = grp ? s[i][j] - st[j] : exp2f(s[i][j] * a.scale_log2 - st[j]);
                s[i][j] = r < rows && n < it.nkeys && n <= tok ? x : 0.f;
                if (grp == 0) P[n * kPS + r] = s[i][j];
            }
        }
        __syncthreads();
        if (grp == 0) {
            accum2<D, D>(acc, P, G, ty, tx);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = (ty + 16 * i) * kPS + tx + 16 * j;
                    S[at] = P[at] * s[i][j];
                }
            asm volatile("bar.sync 1, 256;" ::: "memory");  // (the group)
            accum2<D, D>(acc, S, Q, ty, tx);
        }
    }
    __syncthreads();
    put2<D, D>(grp ? V : K, acc, ty, tx);
    cl.sync();
    add_tiles<D, kThr2>(cl, K, it.nkeys, 1.f, [&](int r) { return static_cast<float *>(b.dv) + pl + (int64_t)r * D; });
    add_tiles<D, kThr2>(cl, V, it.nkeys, a.scale, [&](int r) { return static_cast<float *>(b.dk) + pl + (int64_t)r * D; });
    cl.sync();
}

template <int D> constexpr size_t fwd_smem() { return sizeof(float) * (3 * kT * (D + 4) + kT * kPS); }
template <int D> constexpr size_t bwd_smem() { return sizeof(float) * (4 * kT * (D + 4) + 2 * kT * kPS); }

// Blocks per item: as many as fill the GPU about once (`fit` blocks per SM), each with a tile of
// the walk at least.  Items' walks differ (the first keys are seen by every row), so long ones are
// shared beyond that, by up to 4 blocks that keep 8 tiles each: the first item then ends with the
// rest.  (Backward, one prompt of 2K tokens, 16 heads in 2 groups, d = 128, key tiles shared by 2 / 4 / 8
// blocks: 3.46 / 2.14 / 2.31 ms -- clusters of 8 leave SMs idle --, 4 heads, d = 64: 458 / 306 / 361 us;
// 1K tokens, forward, blocks with 4 / 2 tiles: 37 / 41 us.)
int cluster_size(int64_t items, int walk, int fit) {
    int c = 1;
    while (c < 8 && c * 2 <= walk) {
        const int64_t blocks = items * c * 2, fill = (int64_t)fit * kPlanSms;
        if (blocks > fill && (c >= 4 || walk < 16 * c || blocks > 2 * fill)) break;
        c *= 2;
    }
    return c;
}

template <int D> cudaError_t fwd(const Args &a, int64_t items, cudaStream_t st) {
    cudaError_t e = set_smem_once((const void *)fwd_simt_kernel<D>, fwd_smem<D>());
    if (e != cudaSuccess) return e;
    const int c = a.decode ? 1 : cluster_size(items, (int)ceil_div(a.L, kT), D == 64 ? 2 : 1);
    return launch_next(a.plan != nullptr, fwd_simt_kernel<D>, (int)items * c, kThr, fwd_smem<D>(), st, c, a);
}

template <int D> cudaError_t delta(const BwdArgs &b, const int32_t *cu, int n_seq, cudaStream_t st) {
    const int64_t rows = (int64_t)b.a.B * b.a.L * b.a.hq;
    return launch_next(b.a.plan != nullptr, delta_kernel<D>, (int)ceil_div(rows, 8), 256, 0, st, 1,
                       static_cast<const float *>(b.o), static_cast<const float *>(b.dO), b.delta, rows, b.a.plan ? nullptr : b.a.ds,
                       cu, n_seq, b.a.hq, b.a.plan_n);
}

template <int D> cudaError_t bwd(const BwdArgs &b, int64_t row_items, int64_t key_items, cudaStream_t st) {
    cudaError_t e = set_smem_once((const void *)bwd_dq_simt_kernel<D>, bwd_smem<D>());
    if (e == cudaSuccess) e = set_smem_once((const void *)bwd_dkv_simt_kernel<D>, bwd_smem<D>());
    if (e != cudaSuccess) return e;
    const int ck = cluster_size(key_items, (int)ceil_div(b.a.L, b.a.tok), 1), cr = cluster_size(row_items, (int)ceil_div(b.a.L, kT), 1);
    e = launch_next(true, bwd_dkv_simt_kernel<D>, (int)key_items * ck, kThr2, bwd_smem<D>(), st, ck, b);
    if (e != cudaSuccess) return e;
    return launch_next(true, bwd_dq_simt_kernel<D>, (int)row_items * cr, kThr2, bwd_smem<D>(), st, cr, b);
}

}  // namespace

cudaError_t launch_fwd_simt(const Args &a, int d, int64_t items, cudaStream_t st) {
    return d == 128 ? fwd<128>(a, items, st) : fwd<64>(a, items, st);
}

cudaError_t launch_delta(const BwdArgs &b, int d, const int32_t *cu, int n_seq, cudaStream_t st) {
    return d == 128 ? delta<128>(b, cu, n_seq, st) : delta<64>(b, cu, n_seq, st);
}

cudaError_t launch_bwd_simt(const BwdArgs &b, int d, int64_t row_items, int64_t key_items, cudaStream_t st) {
    return d == 128 ? bwd<128>(b, row_items, key_items, st) : bwd<64>(b, row_items, key_items, st);
}

}  // namespace dense
}  // namespace hsa
