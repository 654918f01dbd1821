// k_dense_bwd_tc.cu -- backward of the dense prompt pass on the tensor cores (bf16).
//
// Mathematics.  With p = 2^(S c - lse log2 e) (S = Q K^T, c = log2(e)/sqrt(d)),
// dP = dO V^T and D = rowsum(dO o):  dS = p (dP - D),  dV = p^T dO,
// dK = dS^T Q / sqrt(d),  dQ = dS K / sqrt(d).
//
// Two passes over the tile pairs, one per stationary operand, instead of one that
// adds dQ tiles into memory: 7 products instead of 5, but no fp32 dQ in memory, no
// atomics (the result does not depend on timing) and nothing but plain stores.
// (Adding 64 KB of fp32 per 128 x 128 tile pair at the 4.8 TB/s that vector
// reductions reach on this GPU takes 2 us per SM, as long as the five products.)
// Both keep every first operand of a second product in tensor memory:
// - key pass: 128 keys per CTA, walking the row tiles that see them (in pieces, with fp32
//   partials added in order afterwards, where there are too few tiles for the GPU).  S^T = K Q^T
//   and dP^T = V dO^T have a key per tensor-memory lane; p and dS go back over them
//   as bf16 and feed dV += p dO, dK += dS Q directly.  The group's heads are rows
//   of the same tiles, so dK and dV of shared heads are summed by the products.
// - row pass: 128 (token, head) rows per CTA, walking the keys: S, dP, then
//   dQ += dS K.  S has two buffers, so the tensor cores run ahead of the exponentials.
// D is written by the row pass, which goes first.  Taken from the stored output (dO . o) it
// carries o's rounding to bf16, 2^-9 of |dO||o|, into every dS of the row; that is small where a
// row averages many values and the largest single error where it averages few.  The row pass
// therefore first sweeps the keys of rows that have at most kSweep tiles of them for D = sum p dP
// (two products more per tile, on a fraction of any long prompt).  The same rows' dS, an operand in
// bf16, keeps in the columns beside it what its rounding takes off, for one product more in either
// pass.  Relative errors of dq and dk against 64 bits (rounding the exact values alone: 0.0017):
// neither 0.0031 (12 tokens), 0.0026 (16K tokens); the sweep 0.0025, 0.0024; both 0.0017, 0.0022.
// The sweep takes about 2 us of a call, the remainders 2 more (2K tokens: 86 -> 88 us); eight tiles
// instead of two gain 0.00002.
// Two compute warpgroups take half of a tile's columns each (64 values of S and of dP
// per thread); the MMAs are issued so that one warpgroup step always has one or two
// products running behind it.
#include <algorithm>

#include "dense_tc.cuh"

namespace hsa {
namespace dense {

namespace {

constexpr int kThreads = 384;
constexpr int kTile = 128;
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpStat = 10, kWarpClear = 11;
constexpr int kItems = 2;
constexpr int kBarriers = 22;    // besides the ring's
constexpr int kSweep = 2;   // row pass: rows of at most so many key tiles take D from a sweep of their own

template <int D, bool KEYS> struct Smem {
    static constexpr int NH = D / 64;
    static constexpr int TILE = NH * 128 * 128;           // bytes of a 128 x D bf16 tile
    static constexpr int ST = D == 128 ? 5 : 10;
    static constexpr int OFF_FIX = 0;                     // the two stationary tiles
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_STAT = OFF_RING + ST * TILE; // key pass: [2][lse, delta][128]; row pass: [2][128]
    static constexpr int OFF_ITEM = OFF_STAT + (KEYS ? 2048 : 1024);
    static constexpr int OFF_BAR = OFF_ITEM + kItems * 64;
    static constexpr int OFF_MISC = OFF_BAR + 384;
    static constexpr int ALLOC = OFF_MISC + 64;
    static_assert((kBarriers + 2 * ST) * 8 <= 384, "barriers");
};
static_assert(Smem<128, true>::ALLOC <= 232448 && Smem<128, false>::ALLOC <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void load64(uint32_t t, float (&x)[64]) {
    float(&x0)[32] = *reinterpret_cast<float(*)[32]>(x);
    float(&x1)[32] = *reinterpret_cast<float(*)[32]>(x + 32);
    tmem_ld32(t, x0);
    tmem_ld32(t + 32, x1);
    wait_loads(x0);
    wait_loads(x1);
}
__device__ __forceinline__ void store64(uint32_t t, const float (&x)[64]) {  // as 32 bf16 pairs
    uint32_t u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
    tmem_st32(t, u);
    tmem_wait_st();
}
// what store64 rounded off, as bf16 pairs in the 32 columns behind its own
__device__ __forceinline__ void store64_rest(uint32_t t, const float (&x)[64]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float a = x[32 * h + 2 * i], b = x[32 * h + 2 * i + 1];
            const uint32_t p = bf16_pair(a, b);
            u[i] = bf16_pair(a - __uint_as_float(p << 16), b - __uint_as_float(p & 0xffff0000u));
        }
        tmem_st16(t + 32 + 16 * h, u);
    }
    tmem_wait_st();
}
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {  // eight bf16 products
    auto two = [](uint32_t x, uint32_t y) {
        return __uint_as_float(x << 16) * __uint_as_float(y << 16) +
               __uint_as_float(x & 0xffff0000u) * __uint_as_float(y & 0xffff0000u);
    };
    return (two(a.x, b.x) + two(a.y, b.y)) + (two(a.z, b.z) + two(a.w, b.w));
}
// one row of a [128 x d] accumulator per lane, scaled, to global memory (as bf16; or fp32 as it is)
template <int D> __device__ __forceinline__ void store_row(uint32_t t, float f, __nv_bfloat16 *dst, bool real, int lane) {
    const QuadRows out(dst, real, lane);
#pragma unroll 1
    for (int h = 0; h < D / 32; ++h) {
        float y[32];
        tmem_ld32(t + h * 32, y);
        wait_loads(y);
        out.store_bf16(y, f, h * 64, lane);
    }
}
template <int D> __device__ __forceinline__ void store_part(uint32_t t, float *dst, bool real, int lane) {
    const QuadRows out(dst, real, lane);
#pragma unroll 1
    for (int h = 0; h < D / 32; ++h) {
        float y[32];
        tmem_ld32(t + h * 32, y);
        wait_loads(y);
        out.store_f32(y, h * 128, lane);
    }
}

struct BwdItem {
    int end, g, plane;
    int tok0, ntok;    // row pass: first token row and tokens; key pass: the sequence's first token row, its length
    int key0, nkeys;   // first key row (inside its plane) and keys
    int off;           // row pass: causal offset; key pass: first key's index in the sequence
    int foreign;
    int j0, j1, slot;  // key pass: row tiles and partial slot (KeyItem)
    int pad[4];
};
static_assert(sizeof(BwdItem) == 64, "item ring");

// ---------------------------------------------------------------------- key pass
template <int D>
__global__ void __launch_bounds__(kThreads, 1) bwd_key_tc_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ BwdArgs b, int32_t *next, uint64_t wait_ns) {
    using L = Smem<D, true>;
    // d = 128: dV, dK, dP and one S fill tensor memory; P is handed over in halves, so that its first
    // product runs under the second half's exponentials.  d = 64: a second S fits, so the next S is
    // computed ahead of the P that the first holds.
    constexpr bool kTwoS = D == 64, kHalves = !kTwoS;
    const Args &a = b.a;
    extern __shared__ __align__(1024) uint8_t sm[];  // (no room to align it by hand)
    if (smem_u32(sm) & 1023) {
        if (threadIdx.x == 0) report(a.ds, HSA_ERR_CUDA, kKDense, 1024, 0);
        return;
    }
    float *stat = reinterpret_cast<float *>(sm + L::OFF_STAT);
    BwdItem *items = reinterpret_cast<BwdItem *>(sm + L::OFF_ITEM);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
    uint64_t *item_full = bar, *item_empty = bar + 2, *fix_full = bar + 4, *fix_empty = bar + 5;
    uint64_t *stat_full = bar + 6, *stat_empty = bar + 8;
    uint64_t *s_full = bar + 20, *dp_full = bar + 11, *p_full = bar + 18, *ds_full = bar + 13, *acc_full = bar + 14;
    uint64_t *done = bar + 15, *clean = bar + 16, *clear_req = bar + 17, *p_half = bar + 10, *ring_full = bar + kBarriers, *ring_empty = ring_full + L::ST;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::OFF_MISC + 16);
    volatile int *clear_job = abort_flag + 1;  // stage, first row, steps

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int tt = 128 / a.G, rows = tt * a.G;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&item_full[i], 1); mbar_init(&item_empty[i], 10);
            mbar_init(&stat_full[i], 1); mbar_init(&stat_empty[i], 8);
        }
        mbar_init(fix_full, 1); mbar_init(fix_empty, 1);
        mbar_init(s_full, 1); mbar_init(s_full + 1, 1); mbar_init(dp_full, 1); mbar_init(p_half, 8); mbar_init(p_full, 8); mbar_init(p_full + 1, 8); mbar_init(ds_full, 8); mbar_init(acc_full, 1);
        mbar_init(done, 1); mbar_init(clean, 1); mbar_init(clear_req, 1);
        for (int i = 0; i < L::ST; ++i) { mbar_init(&ring_full[i], 1); mbar_init(&ring_empty[i], 1); }
        *abort_flag = 0;
        clear_job[2] = 0;
        mbar_fence_init();
    }
    // rows that no box writes (G does not divide 128) take part in the sums over rows: zeros
    if (rows < 128) {
        for (int i = threadIdx.x; i < L::ST * L::TILE / 16; i += kThreads)
            reinterpret_cast<uint4 *>(sm + L::OFF_RING)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == kWarpLoad && lane == 0) {
        prefetch_tmap(&tm_q); prefetch_tmap(&tm_do); prefetch_tmap(&tm_k); prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    dependency_wait();
    dependents_may_start();
    const uint32_t t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + D;
    // A waiter sees a barrier's phases by their parity: the next but one must not complete before it has
    // looked.  With S computed ahead the warpgroups may be a P further than the MMA thread has seen: two
    // barriers, by step.  (The others' next phase needs a product issued behind the wait.)
    auto p_done = [&](int step) { return &p_full[kTwoS ? step & 1 : 0]; };
    auto p_phase = [&](int step) { return (uint32_t)(kTwoS ? step >> 1 : step); };
    // row tile j's rows have at most kSweep key tiles: dS keeps what its rounding takes off (as in the row pass)
    auto few_keys = [&](const BwdItem &t, int j) { return min((j + 1) * tt, t.ntok) <= kSweep * kTile; };
    auto t_s = [&](int step) { return tmem + (kTwoS && (step & 1) ? 384u : 0u); };
    auto wait = [&](uint64_t *x, uint32_t par, int role) { return warp_wait(x, par & 1, wait_ns, abort_flag, a.ds, role); };
    if (warp == kWarpLoad) {
        // ============================================================ items and loads
        const int total = key_item_count(b);
        int idx = blockIdx.x, pos = 0, fixes = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            BwdItem t{};
            KeyItem it;
            t.end = idx >= total || !get_key_item(b, idx, kTile, it);
            if (!t.end) {
                t.g = it.g; t.plane = it.plane; t.tok0 = (int)it.row0; t.ntok = it.len;
                t.key0 = it.start + it.n0; t.nkeys = it.nkeys; t.off = it.n0;
                t.j0 = it.j0; t.j1 = it.j1; t.slot = it.slot;
            }
            const int ib = n % kItems;
            if (n >= kItems && !(ok = wait(&item_empty[ib], n / kItems - 1, 11))) break;
            if (lane == 0) {
                items[ib] = t;
                mbar_arrive(&item_full[ib]);
            }
            __syncwarp();
            if (t.end) break;
            if (n > 0 && !(ok = wait(fix_empty, n - 1, 11))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(fix_full, 2 * L::TILE);
#pragma unroll
                for (int h = 0; h < L::NH; ++h) {
                    tma_load_3d(sm + L::OFF_FIX + h * 16384, &tm_k, h * 64, t.key0, t.plane, fix_full);
                    tma_load_3d(sm + L::OFF_FIX + L::TILE + h * 16384, &tm_v, h * 64, t.key0, t.plane, fix_full);
                }
            }
            ++fixes;
            for (int j = t.j0; ok && j < t.j1; ++j) {
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int st = pos % L::ST;
                    if (pos >= L::ST && !(ok = wait(&ring_empty[st], pos / L::ST - 1, 11))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ring_full[st], L::NH * rows * 128);
#pragma unroll
                        for (int h = 0; h < L::NH; ++h)
                            tma_load_3d(sm + L::OFF_RING + st * L::TILE + h * 16384, o ? &tm_do : &tm_q, h * 64, t.g * a.G,
                                        t.tok0 + j * tt, &ring_full[st]);
                    }
                    ++pos;
                }
            }
            int i = 0;
            if (lane == 0) i = atomicAdd(next, 1);
            idx = __shfl_sync(0xffffffffu, i, 0) + gridDim.x;
        }
        if (lane == 0) {
            land(ring_full, pos, L::ST);
            land(fix_full, fixes, 1);
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ============================================================ MMA issue, a single thread
        if (elect_one()) {
            auto wait1 = [&](uint64_t *x, uint32_t par) { return thread_wait(x, par & 1, wait_ns, abort_flag, a.ds, 12); };
            const uint32_t kb = smem_u32(sm + L::OFF_FIX), vb = kb + L::TILE;
            Ring<L::ST> ring;
            int np = 0, nc = 0;  // np: steps
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const int ib = n % kItems;
                if (!(ok = wait1(&item_full[ib], n / kItems))) break;
                const BwdItem t = items[ib];
                mbar_arrive(&item_empty[ib]);
                if (t.end) break;
                const int j0 = t.j0, j1 = t.j1;
                auto tile = [&](const Ring<L::ST> &r) { return smem_u32(sm + L::OFF_RING + r.st * L::TILE); };
                // Tile j's Q or dO, as loaded next.  Rows behind the sequence's last token are
                // another's (or nothing's): cleared, since the sums run over all 128 rows.
                auto take = [&](int j, Ring<L::ST> &r) -> bool {
                    r = ring;
                    ring.next();
                    if (!wait1(&ring_full[r.st], r.ph)) return false;
                    const int real = (t.ntok - j * tt) * a.G;
                    if (real >= rows) return true;
                    request_clear(clear_req, clear_job, r.st, real);
                    return wait1(clean, nc++);
                };
                Ring<L::ST> q, d, qn;
                if (!(ok = wait1(fix_full, n) && take(j0, q))) break;
                tc_fence_after();
                auto s_done = [&](int step) { return &s_full[kTwoS ? step & 1 : 0]; };
                mma_dots<D>(t_s(np), kb, tile(q));
                mma_commit(s_done(np));
                if (!(ok = take(j0, d))) break;
                mma_dots<D>(t_dp, vb, tile(d));
                mma_commit(dp_full);
                for (int j = j0; j < j1; ++j) {
                    const bool more = j + 1 < j1;
                    clear_job[2] = np + 1;
                    auto next_scores = [&]() -> bool {
                        if (!take(j + 1, qn)) return false;
                        tc_fence_after();
                        mma_dots<D>(t_s(np + 1), kb, tile(qn));
                        mma_commit(s_done(np + 1));
                        return true;
                    };
                    if constexpr (kTwoS) {  // (the loads' order: this tile's dO was taken with its dP)
                        if (more && !(ok = next_scores())) break;
                    } else {
                        if (!(ok = wait1(p_half, np))) break;
                        tc_fence_after();
                        mma_sum<D, 64, 0, 2>(t_dv, t_s(np), tile(d), j > j0);
                        mma_sum<D, 64, 4, 6>(t_dv, t_s(np), tile(d), 1);
                    }
                    if (!(ok = wait1(p_done(np), p_phase(np)))) break;
                    tc_fence_after();
                    if constexpr (kTwoS) {
                        mma_sum<D, 64>(t_dv, t_s(np), tile(d), j > j0);
                    } else {
                        mma_sum<D, 64, 2, 4>(t_dv, t_s(np), tile(d), 1);
                        mma_sum<D, 64, 6, 8>(t_dv, t_s(np), tile(d), 1);
                    }
                    mma_commit(&ring_empty[d.st]);
                    if (!kTwoS && more && !(ok = next_scores())) break;
                    if (!(ok = wait1(ds_full, np++))) break;
                    tc_fence_after();
                    mma_sum<D, 64>(t_dk, t_dp, tile(q), j > j0);
                    if (few_keys(t, j)) mma_sum<D, 64>(t_dk, t_dp + 32, tile(q), 1);
                    mma_commit(&ring_empty[q.st]);
                    if (more) {
                        if (!(ok = take(j + 1, d))) break;
                        tc_fence_after();
                        mma_dots<D>(t_dp, vb, tile(d));
                        mma_commit(dp_full);
                    } else {
                        mma_commit(acc_full);
                        mma_commit(fix_empty);
                    }
                    q = qn;
                }
            }
            request_clear(clear_req, clear_job, -1, 0);
            finish_mma(done);
        }
        __syncwarp();
    } else if (warp == kWarpClear) {
        clear_role(sm + L::OFF_RING, L::TILE, L::NH, clear_req, clean, clear_job, abort_flag, wait_ns, lane);
    } else if (warp == kWarpStat) {
        // ============================================================ row statistics of each tile
        int nt = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const int ib = n % kItems;
            if (!(ok = wait(&item_full[ib], n / kItems, 13))) break;
            const BwdItem t = items[ib];
            __syncwarp();
            mbar_arrive_lane0(&item_empty[ib], lane);
            if (t.end) break;
            for (int j = t.j0; j < t.j1; ++j, ++nt) {
                float l2[4], de[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 32 + lane, tk = j * tt + r / a.G;
                    const bool real = r < rows && tk < t.ntok;
                    const int64_t at = ((int64_t)t.tok0 + tk) * a.hq + t.g * a.G + r % a.G;
                    l2[i] = real ? b.lse[at] * kLog2e : INFINITY;  // p = 2^-inf = 0
                    de[i] = real ? b.delta[at] : 0.f;
                }
                if (nt >= 2 && !(ok = wait(&stat_empty[nt & 1], (nt >> 1) - 1, 13))) break;
                float *s = stat + (nt & 1) * 256;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[i * 32 + lane] = l2[i];
                    s[128 + i * 32 + lane] = de[i];
                }
                __syncwarp();
                mbar_arrive_lane0(&stat_full[nt & 1], lane);
            }
        }
    } else if (warp < 8) {
        // ============================================================ p and dS, 64 columns per warpgroup
        const int w = warp >> 2, key = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t xd = t_dp + lanes + w * 64;
        const float c = a.scale_log2;
        int nt = 0, na = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const int ib = n % kItems;
            if (!(ok = wait(&item_full[ib], n / kItems, 14))) break;
            const BwdItem t = items[ib];
            __syncwarp();
            mbar_arrive_lane0(&item_empty[ib], lane);
            if (t.end) break;
            for (int j = t.j0; j < t.j1; ++j, ++nt) {
                const float4 *s4 = reinterpret_cast<const float4 *>(stat + (nt & 1) * 256 + w * 64);
                if (!(ok = wait(&stat_full[nt & 1], nt >> 1, 14))) break;
                const uint32_t xs = t_s(nt) + lanes + w * 64;
                if (!(ok = wait(kTwoS ? &s_full[nt & 1] : s_full, kTwoS ? nt >> 1 : nt, 14))) break;
                tc_fence_after();
                float x[64];
                load64(xs, x);
                const float2 c2 = make_float2(c, c);
                const bool edge = j * tt < t.off + kTile - 1;  // some row of the tile does not see some of the keys
                const int first = (t.off + key - j * tt) * a.G - w * 64;  // first column that sees this key
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // the first half is multiplied while the second is exponentials
#pragma unroll
                    for (int i = 8 * h; i < 8 * h + 8; ++i) {
                        const float4 l = s4[i];
                        const float2 u = fma2(make_float2(x[4 * i], x[4 * i + 1]), c2, make_float2(-l.x, -l.y));
                        const float2 v = fma2(make_float2(x[4 * i + 2], x[4 * i + 3]), c2, make_float2(-l.z, -l.w));
                        x[4 * i] = ex2(u.x); x[4 * i + 1] = ex2(u.y); x[4 * i + 2] = ex2(v.x); x[4 * i + 3] = ex2(v.y);
                    }
                    if (edge) {
#pragma unroll
                        for (int i = 32 * h; i < 32 * h + 32; ++i) x[i] = i >= first ? x[i] : 0.f;
                    }
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[i] = bf16_pair(x[32 * h + 2 * i], x[32 * h + 2 * i + 1]);
                    tmem_st16(xs + 16 * h, u);
                    if (!h && !kHalves) continue;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_lane0(h ? p_done(nt) : p_half, lane);
                }
                if (!(ok = wait(dp_full, nt, 14))) break;
                tc_fence_after();
                float y[64];
                load64(xd, y);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 d = s4[32 + i];
                    const float2 u = mul2(make_float2(x[4 * i], x[4 * i + 1]), add2(make_float2(y[4 * i], y[4 * i + 1]), make_float2(-d.x, -d.y)));
                    const float2 v = mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), add2(make_float2(y[4 * i + 2], y[4 * i + 3]), make_float2(-d.z, -d.w)));
                    x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = v.x; x[4 * i + 3] = v.y;
                }
                store64(xd, x);
                if (few_keys(t, j)) store64_rest(xd, x);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_lane0(ds_full, lane);
                mbar_arrive_lane0(&stat_empty[nt & 1], lane);
            }
            if (!ok || !(ok = wait(acc_full, na, 14))) break;
            ++na;
            tc_fence_after();
            if (t.slot >= 0) {  // one of several pieces of this tile's rows
                store_part<D>((w ? t_dk : t_dv) + lanes, b.part + (((int64_t)t.slot * 2 + w) * 128 + key) * D, key < t.nkeys, lane);
                tc_fence_before();
                continue;
            }
            const int64_t at = (int64_t)t.plane * a.plane[0] + (int64_t)(t.key0 + key) * D;
            if (w == 0) store_row<D>(t_dv + lanes, 1.f, static_cast<__nv_bfloat16 *>(b.dv) + at, key < t.nkeys, lane);
            else store_row<D>(t_dk + lanes, a.scale, static_cast<__nv_bfloat16 *>(b.dk) + at, key < t.nkeys, lane);
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- row pass
template <int D>
__global__ void __launch_bounds__(kThreads, 1) bwd_row_tc_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
    const __grid_constant__ CUtensorMap tm_do,
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ BwdArgs b, int32_t *next, uint64_t wait_ns) {
    using L = Smem<D, false>;
    const Args &a = b.a;
    extern __shared__ __align__(1024) uint8_t sm[];  // (no room to align it by hand)
    if (smem_u32(sm) & 1023) {
        if (threadIdx.x == 0) report(a.ds, HSA_ERR_CUDA, kKDense, 1024, 0);
        return;
    }
    float *joint = reinterpret_cast<float *>(sm + L::OFF_STAT);  // [2][128]
    BwdItem *items = reinterpret_cast<BwdItem *>(sm + L::OFF_ITEM);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
    uint64_t *item_full = bar, *item_empty = bar + 2, *fix_full = bar + 4, *fix_empty = bar + 5;
    uint64_t *s_full = bar + 6, *dp_full = bar + 8, *dp_read = bar + 9, *ds_full = bar + 17, *acc_full = bar + 11;
    uint64_t *done = bar + 12, *clean = bar + 13, *clear_req = bar + 14, *join = bar + 15, *out_read = bar + 16, *ring_full = bar + kBarriers, *ring_empty = ring_full + L::ST;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::OFF_MISC + 16);
    volatile int *clear_job = abort_flag + 1;  // stage, first row, steps

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int tt = 128 / a.G, rows = tt * a.G;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) { mbar_init(&item_full[i], 1); mbar_init(&item_empty[i], 9); mbar_init(&s_full[i], 1); }
        mbar_init(fix_full, 1); mbar_init(fix_empty, 1);
        mbar_init(dp_full, 1); mbar_init(dp_read, 8); mbar_init(ds_full, 8); mbar_init(ds_full + 1, 8); mbar_init(acc_full, 1);
        mbar_init(join, 8); mbar_init(out_read, 8);
        mbar_init(done, 1); mbar_init(clean, 1); mbar_init(clear_req, 1);
        for (int i = 0; i < L::ST; ++i) { mbar_init(&ring_full[i], 1); mbar_init(&ring_empty[i], 1); }
        *abort_flag = 0;
        clear_job[2] = 0;
        mbar_fence_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == kWarpLoad && lane == 0) {
        prefetch_tmap(&tm_q); prefetch_tmap(&tm_o); prefetch_tmap(&tm_do); prefetch_tmap(&tm_k); prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    dependency_wait();
    dependents_may_start();
    const uint32_t t_s = tmem, t_dp = tmem + 256, t_dq = tmem + 384;  // S: two buffers
    // (S and dP of the next step are issued before the wait for this step's dS, so the warpgroups may
    // finish both before the MMA thread looks: two ds_full, in turns)
    auto wait = [&](uint64_t *x, uint32_t par, int role) { return warp_wait(x, par & 1, wait_ns, abort_flag, a.ds, role); };
    auto tiles = [](int keys) { return (keys + kTile - 1) / kTile; };
    auto sweep = [](int nt) { return nt <= kSweep ? nt : 0; };

    if (warp == kWarpLoad) {
        // ============================================================ items and loads
        const int total = item_count(a);
        int idx = blockIdx.x, pos = 0, fixes = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            BwdItem t{};
            Item it;
            t.end = idx >= total || !get_item(a, idx, it);
            if (!t.end) {
                t.g = it.g; t.plane = it.plane; t.tok0 = it.tok0; t.ntok = it.ntok;
                t.key0 = it.key0; t.nkeys = it.nkeys; t.off = it.off; t.foreign = it.foreign;
            }
            const int ib = n % kItems;
            if (n >= kItems && !(ok = wait(&item_empty[ib], n / kItems - 1, 21))) break;
            if (lane == 0) {
                items[ib] = t;
                mbar_arrive(&item_full[ib]);
            }
            __syncwarp();
            if (t.end) break;
            const int nt = tiles(t.nkeys), sw = sweep(nt), all = nt + sw;
            auto load = [&](const CUtensorMap *m, int bytes, int y, int z) -> bool {
                const int st = pos % L::ST;
                if (pos >= L::ST && !wait(&ring_empty[st], pos / L::ST - 1, 21)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ring_full[st], bytes);
#pragma unroll
                    for (int h = 0; h < L::NH; ++h)
                        tma_load_3d(sm + L::OFF_RING + st * L::TILE + h * 16384, m, h * 64, y, z, &ring_full[st]);
                }
                ++pos;
                return true;
            };
            // the ring's first tiles do not wait for the item before: rows without a sweep, their
            // stored output (for D = dO . o); the first K and V
            if (!sw) ok = load(&tm_o, L::NH * rows * 128, t.g * a.G, t.tok0);
            ok = ok && load(&tm_k, L::TILE, t.key0, t.plane) && load(&tm_v, L::TILE, t.key0, t.plane);
            if (!ok || (n > 0 && !(ok = wait(fix_empty, n - 1, 21)))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(fix_full, 2 * L::NH * rows * 128);
#pragma unroll
                for (int h = 0; h < L::NH; ++h) {
                    tma_load_3d(sm + L::OFF_FIX + h * 16384, &tm_q, h * 64, t.g * a.G, t.tok0, fix_full);
                    tma_load_3d(sm + L::OFF_FIX + L::TILE + h * 16384, &tm_do, h * 64, t.g * a.G, t.tok0, fix_full);
                }
            }
            ++fixes;
            for (int j = 1; ok && j < all; ++j) {
                const int key = t.key0 + (j < sw ? j : j - sw) * kTile;
                ok = load(&tm_k, L::TILE, key, t.plane) && load(&tm_v, L::TILE, key, t.plane);
            }
            int i = 0;
            if (lane == 0) i = atomicAdd(next, 1);
            idx = __shfl_sync(0xffffffffu, i, 0) + gridDim.x;
        }
        if (lane == 0) {
            land(ring_full, pos, L::ST);
            land(fix_full, fixes, 1);
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // ============================================================ MMA issue, a single thread
        if (elect_one()) {
            auto wait1 = [&](uint64_t *x, uint32_t par) { return thread_wait(x, par & 1, wait_ns, abort_flag, a.ds, 22); };
            const uint32_t qb = smem_u32(sm + L::OFF_FIX), ob = qb + L::TILE;
            Ring<L::ST> ring;
            int nt = 0, nc = 0, nd = 0, n_out = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const int ib = n % kItems;
                if (!(ok = wait1(&item_full[ib], n / kItems))) break;
                const BwdItem t = items[ib];
                mbar_arrive(&item_empty[ib]);
                if (t.end) break;
                if (!(ok = wait1(fix_full, n))) break;
                // steps: first the sweep for D (S and dP only), then the keys
                const int nk = tiles(t.nkeys), sw = sweep(nk), nn = sw + nk;
                auto tile = [&](const Ring<L::ST> &r) { return smem_u32(sm + L::OFF_RING + r.st * L::TILE); };
                auto scores = [&](int j, Ring<L::ST> &k) -> bool {  // S of step j, into buffer (nt + j) & 1
                    k = ring;
                    ring.next();
                    if (!wait1(&ring_full[k.st], k.ph)) return false;
                    if (t.foreign && j == nn - 1 && t.nkeys % kTile) {  // dS is 0 there, but 0 * NaN is not
                        request_clear(clear_req, clear_job, k.st, t.nkeys % kTile);
                        if (!wait1(clean, nc++)) return false;
                    }
                    const int sb = (nt + j) & 1;
                    tc_fence_after();
                    mma_dots<D>(t_s + sb * 128, qb, tile(k));
                    mma_commit(&s_full[sb]);
                    if (j < sw) mma_commit(&ring_empty[k.st]);
                    return true;
                };
                auto dprob = [&](int j) -> bool {
                    const Ring<L::ST> v = ring;
                    ring.next();
                    if (!wait1(&ring_full[v.st], v.ph)) return false;
                    if (j > 0 && !wait1(dp_read, nt + j - 1)) return false;
                    tc_fence_after();
                    mma_dots<D>(t_dp, ob, tile(v));
                    mma_commit(dp_full);
                    mma_commit(&ring_empty[v.st]);
                    if (j == nn - 1) mma_commit(fix_empty);
                    return true;
                };
                Ring<L::ST> k, kn;
                const Ring<L::ST> out = ring;
                if (!sw) ring.next();
                ok = scores(0, k) && dprob(0);
                if (ok && !sw) {  // the warpgroups have read the output tile
                    ok = wait1(out_read, n_out++);
                    mbar_arrive(&ring_empty[out.st]);
                }
                for (int j = 0; ok && j < nn; ++j) {
                    clear_job[2] = nt + j + 1;
                    // (S of step j + 1 goes over that of j - 1: read, and its dS multiplied, before dP of j)
                    if (j + 1 < nn) {
                        if (!(ok = scores(j + 1, kn) && dprob(j + 1))) break;
                    } else if (!(ok = wait1(dp_read, nt + j))) {  // the next item's dP overwrites it
                        break;
                    }
                    if (j >= sw) {
                        if (!(ok = wait1(&ds_full[nd & 1], nd >> 1))) break;
                        ++nd;
                        tc_fence_after();
                        mma_sum<D, 64>(t_dq, t_s + ((nt + j) & 1) * 128, tile(k), j > sw);
                        if (sw) mma_sum<D, 64>(t_dq, t_s + ((nt + j) & 1) * 128 + 32, tile(k), 1);
                        mma_commit(&ring_empty[k.st]);
                        if (j == nn - 1) mma_commit(acc_full);
                    }
                    k = kn;
                }
                nt += nn;
            }
            request_clear(clear_req, clear_job, -1, 0);
            finish_mma(done);
        }
        __syncwarp();
    } else if (warp == kWarpClear) {
        clear_role(sm + L::OFF_RING, L::TILE, L::NH, clear_req, clean, clear_job, abort_flag, wait_ns, lane);
    } else if (warp < 8) {
        // ============================================================ dS, 64 keys per warpgroup
        const int w = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t xd = t_dp + lanes + w * 64;
        const float c = a.scale_log2;
        const int rt = r / a.G, rh = r % a.G;
        int nt = 0, na = 0, n_join = 0, pos = 0, nd = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const int ib = n % kItems;
            if (!(ok = wait(&item_full[ib], n / kItems, 24))) break;
            const BwdItem t = items[ib];
            __syncwarp();
            mbar_arrive_lane0(&item_empty[ib], lane);
            if (t.end) break;
            const bool real = r < t.ntok * a.G;
            const int64_t row = ((int64_t)t.tok0 + rt) * a.hq + t.g * a.G + rh;
            const float l2 = real ? b.lse[row] * kLog2e : INFINITY;
            float de = 0.f;
            const int lim = min(t.nkeys - 1, t.off + rt), lim_all = min(t.nkeys - 1, t.off);
            const int nk = tiles(t.nkeys), sw = sweep(nk);
            float dsum = 0.f;
            if (!sw) {  // D = dO . o, half of the columns per warpgroup, from the tiles in shared memory
                const int st = pos % L::ST;
                if (!(ok = wait(fix_full, n, 24) && wait(&ring_full[st], pos / L::ST, 24))) break;
                const int h = D == 128 ? w : 0, c0 = D == 128 ? 0 : 4 * w;  // 64-column half, first 16-byte piece
                const uint8_t *po = sm + L::OFF_RING + st * L::TILE + h * 16384 + r * 128;
                const uint8_t *pd = sm + L::OFF_FIX + L::TILE + h * 16384 + r * 128;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int at = ((c0 + i) ^ (r & 7)) << 4;
                    dsum += dot8(*reinterpret_cast<const uint4 *>(po + at), *reinterpret_cast<const uint4 *>(pd + at));
                }
                if (!real) dsum = 0.f;
                ++pos;
                __syncwarp();
                mbar_arrive_lane0(out_read, lane);
            }
            pos += 2 * (sw + nk);
            if (!sw) {
                joint[w * 128 + r] = dsum;
                __syncwarp();
                mbar_arrive_lane0(join, lane);
                if (!(ok = wait(join, n_join++, 24))) break;
                de = joint[r] + joint[128 + r];
                if (w == 0 && real) b.delta[row] = de;  // for the key pass
            }
            for (int step = 0; step < sw + nk; ++step, ++nt) {
                const bool first = step < sw;
                const int j = first || !sw ? step : step - sw;
                const int sb = nt & 1;
                const uint32_t xs = t_s + lanes + sb * 128 + w * 64;
                if (!(ok = wait(&s_full[sb], nt >> 1, 24))) break;
                tc_fence_after();
                float x[64];
                load64(xs, x);
                const float2 c2 = make_float2(c, c), m2 = make_float2(-l2, -l2);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 u = fma2(make_float2(x[i], x[i + 1]), c2, m2);
                    x[i] = ex2(u.x);
                    x[i + 1] = ex2(u.y);
                }
                if (!(ok = wait(dp_full, nt, 24))) break;
                tc_fence_after();
                float y[64];
                load64(xd, y);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_lane0(dp_read, lane);
                const int last = lim - j * kTile - w * 64;
                const bool edge = j * kTile + kTile - 1 > lim_all;
                if (first) {  // D = sum p dP over the keys this row sees
                    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        float2 u = mul2(make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]));
                        float2 v = mul2(make_float2(x[i + 2], x[i + 3]), make_float2(y[i + 2], y[i + 3]));
                        if (edge) {
                            u.x = i <= last ? u.x : 0.f;
                            u.y = i + 1 <= last ? u.y : 0.f;
                            v.x = i + 2 <= last ? v.x : 0.f;
                            v.y = i + 3 <= last ? v.y : 0.f;
                        }
                        a0 = add2(a0, u);
                        a1 = add2(a1, v);
                    }
                    a0 = add2(a0, a1);
                    dsum += a0.x + a0.y;
                    if (step == sw - 1) {  // the two warpgroups' halves
                        joint[w * 128 + r] = dsum;
                        __syncwarp();
                        mbar_arrive_lane0(join, lane);
                        if (!(ok = wait(join, n_join++, 24))) break;
                        de = joint[r] + joint[128 + r];
                        if (w == 0 && real) b.delta[row] = de;
                    }
                    continue;
                }
                const float2 d2 = make_float2(-de, -de);
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 u = mul2(make_float2(x[i], x[i + 1]), add2(make_float2(y[i], y[i + 1]), d2));
                    x[i] = u.x;
                    x[i + 1] = u.y;
                }
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) x[i] = i <= last ? x[i] : 0.f;
                }
                store64(xs, x);
                if (sw) store64_rest(xs, x);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_lane0(&ds_full[nd++ & 1], lane);
            }
            if (!ok || !(ok = wait(acc_full, na, 24))) break;
            ++na;
            tc_fence_after();
            // each warpgroup stores half of the row
            store_row<D / 2>(t_dq + lanes + w * (D / 2), a.scale, static_cast<__nv_bfloat16 *>(b.dq) + row * D + w * (D / 2), real, lane);
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const BwdArgs &b, int64_t row_items, int64_t key_items, int32_t *next, cudaStream_t st) {
    const Args &a = b.a;
    CUtensorMap mq, mo, mg, mk, mv;
    const uint64_t toks = (uint64_t)a.B * a.L, tt = 128 / a.G, planes = (uint64_t)a.B * a.hkv;
    if (!make_map3(&mq, a.q, D, a.hq, D, toks, (uint64_t)a.hq * D, a.G, (uint32_t)tt) ||
        !make_map3(&mo, b.o, D, a.hq, D, toks, (uint64_t)a.hq * D, a.G, (uint32_t)tt) ||
        !make_map3(&mg, b.dO, D, a.hq, D, toks, (uint64_t)a.hq * D, a.G, (uint32_t)tt) ||
        !make_map3(&mk, a.k[0], D, a.L, D, planes, a.plane[0], kTile, 1) ||
        !make_map3(&mv, a.v[0], D, a.L, D, planes, a.plane[0], kTile, 1))
        return cudaErrorInvalidValue;
    cudaError_t e = set_smem_once((const void *)bwd_key_tc_kernel<D>, Smem<D, true>::ALLOC);
    if (e == cudaSuccess) e = set_smem_once((const void *)bwd_row_tc_kernel<D>, Smem<D, false>::ALLOC);
    if (e != cudaSuccess) return e;
    // the row pass first: it writes delta for the key pass
    e = launch_next(b.a.plan || b.kplan, bwd_row_tc_kernel<D>, (int)std::min<int64_t>(row_items, sm_count()), kThreads,
                    Smem<D, false>::ALLOC, st, 1, mq, mo, mg, mk, mv, b, next + 1, wait_limit_ns());
    if (e != cudaSuccess) return e;
    return launch_next(true, bwd_key_tc_kernel<D>, (int)std::min<int64_t>(key_items, sm_count()), kThreads,
                       Smem<D, true>::ALLOC, st, 1, mq, mg, mk, mv, b, next, wait_limit_ns());
}

}  // namespace

cudaError_t launch_bwd_tc(const BwdArgs &b, int d, int64_t row_items, int64_t key_items, int32_t *next, cudaStream_t st) {
    return d == 128 ? launch<128>(b, row_items, key_items, next, st) : launch<64>(b, row_items, key_items, next, st);
}

}  // namespace dense
}  // namespace hsa
