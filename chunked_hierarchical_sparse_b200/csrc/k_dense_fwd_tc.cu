// k_dense_fwd_tc.cu -- dense attention on the tensor cores (bf16): the prompt pass
// and the prefix part of the shared-prefix decode step.
//
// Mathematics.  For a tile of 128 (token, head) rows, keys in tiles of 128:
// S = Q K^T, p = 2^(s c - m), l += sum p, O += P V with c = log2(e)/sqrt(d), one
// pass over the keys; o = O / l, lse = (m + log2 l) ln 2.  m is a running
// maximum that is only moved (and O, l rescaled) when a tile exceeds it by more
// than 2^8: p then stays below 256, which neither fp32 sums nor bf16 operands
// mind, and O in tensor memory is almost never touched.  (The online softmax of Milakov
// and Gimelshein, 2018; a maximum moved only beyond a bound, two row tiles in turns and P
// over S in tensor memory are published steps of attention on this generation of GPUs.)
//
// One persistent CTA per SM with two streams, each a 128-row tile with its own S
// and O in tensor memory and its own softmax warpgroup (one thread per row, the
// whole row of S in registers; P goes back over S's columns as bf16 and feeds the
// second product from there).  While one stream's softmax works, the tensor cores
// run the other's products; the MMAs of a stream are issued in the order
// P.V(j), S(j+1), so S may overwrite the P that the product before it reads, and
// a finished S(j+1) means that O holds tiles 0..j.
// - Many rows: the streams are neighbouring row tiles and share the K and V tiles.
// - Few rows (a decode batch of one row tile; a prompt whose row tiles would be too few
//   for the GPU, or one sequence longer than its SM's share of a packed batch): both
//   streams hold the same rows and take half of the keys each; their results are joined
//   in the epilogue.
// Warp 8 deals the items (dynamically, dearest first) and loads K and V by TMA, warp 9
// issues the MMAs, warp 10 clears foreign rows, warp 11 loads Q.
#include <algorithm>
#include <atomic>

#include "dense_tc.cuh"

namespace hsa {
namespace dense {

namespace {

constexpr int kThreads = 384;
constexpr int kKeys = 128;        // keys per tile
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpClear = 10, kWarpQ = 11;
constexpr int kItems = 3;         // item ring
constexpr float kSlack = 8.f;     // log2 of how far a tile may exceed m before it moves

template <int D> struct Smem {
    static constexpr int NH = D / 64;                 // 64-column halves
    static constexpr int TILE = NH * 128 * 128;       // bytes of a 128 x D bf16 tile
    static constexpr int ST = D == 128 ? 5 : 10;      // K / V tile ring
    static constexpr int OFF_Q = 0;                   // [2]
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_ITEM = OFF_KV + ST * TILE;
    static constexpr int OFF_JOINT = OFF_ITEM + 256;  // m and l of stream 1's rows
    static constexpr int OFF_BAR = OFF_JOINT + 1024;
    static constexpr int OFF_MISC = OFF_BAR + 512;
    static constexpr int ALLOC = OFF_MISC + 64 + 1024;  // + alignment to 1 KB
};
static_assert(Smem<128>::ALLOC <= 232448 && Smem<64>::ALLOC <= 232448, "shared memory of a CTA");
static_assert((2 * kItems + 17 + 2 * Smem<64>::ST) * 8 <= 512, "barriers");

struct TcItem {
    int end, plane, g, shared, foreign, slot;
    int tok[2], ntok[2], key0[2], nkeys[2], off[2];
};
static_assert(kItems * sizeof(TcItem) <= 256, "item ring");

// Item i of the call as two streams; false when neither has rows and keys.
__device__ __forceinline__ bool get_tc_item(const Args &a, int i, TcItem &t) {
    Item it;
    const bool some = get_item(a, i, it);
    const int tt = 128 / a.G;  // tokens of one stream's tile
    t.end = 0; t.plane = it.plane; t.g = it.g;
    t.shared = !it.split;
    t.foreign = it.foreign; t.slot = it.slot;
    if (t.shared) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            t.tok[s] = it.tok0 + s * tt;
            t.ntok[s] = min(tt, it.ntok - s * tt);
            t.key0[s] = it.key0;
            t.off[s] = it.off == kNoMask ? kNoMask : it.off + s * tt;
            t.nkeys[s] = t.ntok[s] <= 0 ? 0 : (it.off == kNoMask ? it.nkeys : min(it.nkeys, t.off[s] + t.ntok[s]));
        }
    } else {  // half of the keys each, in whole tiles
        const int half = (it.nkeys + 2 * kKeys - 1) / (2 * kKeys) * kKeys;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            t.tok[s] = it.tok0;
            t.ntok[s] = it.ntok;
            t.key0[s] = it.key0 + s * half;
            t.off[s] = it.off == kNoMask ? kNoMask : it.off - s * half;
            t.nkeys[s] = max(0, min(half, it.nkeys - s * half));
        }
    }
    return some;
}

// this warp's lanes, 16 columns of an accumulator, times f (few registers: the caller holds a row of S)
__device__ __forceinline__ void rescale16(uint32_t t, float f) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    tmem_st16(t, r);
}

// DECODE: the prefix part of a decode step (fp32 partials), else the prompt pass; two kernels,
// since what an item runs once should be as little code as possible (instruction fetch).
template <int D, bool DECODE>
__global__ void __launch_bounds__(kThreads, 1) fwd_tc_kernel(
    const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
    const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ Args a, int32_t *next, uint64_t wait_ns) {
    using L = Smem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    TcItem *items = reinterpret_cast<TcItem *>(sm + L::OFF_ITEM);
    float *joint = reinterpret_cast<float *>(sm + L::OFF_JOINT);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
    uint64_t *item_full = bar, *item_empty = bar + kItems;
    uint64_t *q_full = item_empty + kItems, *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 2, *p_full = s_full + 2, *o_full = p_full + 2;
    uint64_t *p_half = o_full + 2, *clean = p_half + 2, *clear_req = clean + 1, *join_full = clear_req + 1, *join_empty = join_full + 1, *done = join_empty + 1;
    uint64_t *kv_full = done + 1, *kv_empty = kv_full + L::ST;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::OFF_MISC + 16);
    volatile int *clear_job = abort_flag + 1;  // stage, first row, steps

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i) { mbar_init(&item_full[i], 1); mbar_init(&item_empty[i], 10); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1); mbar_init(&p_half[i], 4); mbar_init(&p_full[i], 4); mbar_init(&o_full[i], 1);
        }
        mbar_init(join_full, 4); mbar_init(join_empty, 4);
        mbar_init(done, 1); mbar_init(clean, 1); mbar_init(clear_req, 1);
        for (int i = 0; i < L::ST; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
        *abort_flag = 0;
        clear_job[2] = 0;
        mbar_fence_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == kWarpLoad && lane == 0) {
        prefetch_tmap(&tm_q); prefetch_tmap(&tm_k); prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    dependency_wait();
    // A call of at most one item per block needs no counter and clears its header here: the
    // other blocks report nothing but waits that ran out, seconds later.
    if (!next && blockIdx.x == 0 && threadIdx.x == 0) *a.ds = DevStatus{};
    if (!next) __syncthreads();
    dependents_may_start();
    auto wait = [&](uint64_t *b, uint32_t par, int role) { return warp_wait(b, par & 1, wait_ns, abort_flag, a.ds, role); };
    auto tiles = [](int keys) { return (keys + kKeys - 1) / kKeys; };

    if (warp >= 8) {
        reg_dec<72>();
        if (warp == kWarpLoad) {
            // ======================================================== items and loads
            const int total = item_count(a);
            int idx = blockIdx.x, kv = 0;
            bool ok = true;
            auto next_item = [&]() -> int {  // the first gridDim.x items are dealt by block index
                if (!next) return total;     // there are no more
                int i = 0;
                if (lane == 0) i = atomicAdd(next, 1);
                return __shfl_sync(0xffffffffu, i, 0) + gridDim.x;
            };
            TcItem t, ahead;  // the next item is looked up (two trips to memory) before this one's loads
            auto look_up = [&](TcItem &x) {
                while (idx < total && !get_tc_item(a, idx, x)) idx = next_item();
                x.end = idx >= total;
            };
            look_up(t);
            for (int n = 0; ok; ++n, t = ahead) {
                const int ib = n % kItems;
                if (n >= kItems && !(ok = wait(&item_empty[ib], n / kItems - 1, 1))) break;
                if (lane == 0) {
                    items[ib] = t;
                    mbar_arrive(&item_full[ib]);  // release: the item is visible to those who wait
                }
                __syncwarp();
                if (t.end) break;
                auto load_kv = [&](const CUtensorMap *m, int key) -> bool {
                    const int st = kv % L::ST;
                    if (kv >= L::ST && !wait(&kv_empty[st], kv / L::ST - 1, 1)) return false;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&kv_full[st], L::TILE);
#pragma unroll
                        for (int h = 0; h < L::NH; ++h)
                            tma_load_3d(sm + L::OFF_KV + st * L::TILE + h * 16384, m, h * 64, key, t.plane, &kv_full[st]);
                    }
                    ++kv;
                    return true;
                };
                const int n0 = tiles(t.nkeys[0]), n1 = tiles(t.nkeys[1]);
                ok = load_kv(&tm_k, t.key0[0]);
                if (ok && !t.shared && n1) ok = load_kv(&tm_k, t.key0[1]);
                idx = next_item();
                look_up(ahead);
                if (t.shared) {
                    const int nn = max(n0, n1);
                    for (int j = 0; ok && j < nn; ++j) {
                        ok = load_kv(&tm_v, t.key0[0] + j * kKeys);
                        if (ok && j + 1 < nn) ok = load_kv(&tm_k, t.key0[0] + (j + 1) * kKeys);
                    }
                } else {
                    for (int j = 0; ok && j < n0; ++j) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int ns = s ? n1 : n0;
                            if (ok && j < ns) ok = load_kv(&tm_v, t.key0[s] + j * kKeys);
                            if (ok && j + 1 < ns) ok = load_kv(&tm_k, t.key0[s] + (j + 1) * kKeys);
                        }
                    }
                }
            }
            if (lane == 0) land(kv_full, kv, L::ST);
            __syncwarp();
        } else if (warp == kWarpQ) {
            // ======================================================== rows of Q (beside the other loads, so that
            // the next item's keys and values are on their way before this item's Q tiles are free)
            int nq[2] = {0, 0};
            bool ok = true;
            for (int n = 0; ok; ++n) {
                const int ib = n % kItems;
                if (!(ok = wait(&item_full[ib], n / kItems, 5))) break;
                const TcItem t = items[ib];
                __syncwarp();
                mbar_arrive_lane0(&item_empty[ib], lane);
                if (t.end) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!ok || t.nkeys[s] == 0) continue;
                    if (nq[s] > 0 && !(ok = wait(&q_empty[s], nq[s] - 1, 5))) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[s], L::NH * a.G * (128 / a.G) * 128);
#pragma unroll
                        for (int h = 0; h < L::NH; ++h)
                            tma_load_3d(sm + L::OFF_Q + s * L::TILE + h * 16384, &tm_q, h * 64, t.g * a.G, t.tok[s], &q_full[s]);
                    }
                    ++nq[s];
                }
            }
            if (lane == 0)
                for (int s = 0; s < 2; ++s) land(&q_full[s], nq[s], 1);
            __syncwarp();
        } else if (warp == kWarpMma) {
            // ======================================================== MMA issue, a single thread
            // One thread issues for both streams, in turns: the products then run first come, first
            // served, one stream's while the other's softmax works.  (Two issuing warps interleave
            // the streams' products, both finish late and both softmaxes run at the same time:
            // 1185 instead of 1310 TFLOP/s at 64K tokens.)
            if (elect_one()) {
                auto wait1 = [&](uint64_t *b, uint32_t par) { return thread_wait(b, par & 1, wait_ns, abort_flag, a.ds, 2); };
                Ring<L::ST> kv;
                int nq[2] = {0, 0}, np[2] = {0, 0}, nc = 0, steps = 0;
                bool ok = true;
                for (int n = 0; ok; ++n) {
                    const int ib = n % kItems;
                    if (!(ok = wait1(&item_full[ib], n / kItems))) break;
                    const TcItem t = items[ib];
                    mbar_arrive(&item_empty[ib]);
                    if (t.end) break;
                    const bool shared = t.shared;
                    const int n0 = tiles(t.nkeys[0]), n1 = tiles(t.nkeys[1]), nn = max(n0, n1);
                    // Tiles in the order of the loads: shared, K(j) V(j) for both streams; else K0(0) [K1(0)],
                    // then per j V0(j) K0(j+1) V1(j) K1(j+1), as far as each stream goes.
                    // A shared tile is free once the last stream that reads it has.
                    auto last_reader = [&](int s, int j) { return !shared || s == 1 || j >= n1; };
                    Ring<L::ST> v, k;  // the tiles in hand
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!ok || (s ? n1 : n0) == 0) continue;
                        if (s == 0 || !shared) {
                            k = kv;
                            kv.next();
                            if (!(ok = wait1(&kv_full[k.st], k.ph))) break;
                        }
                        if (!(ok = wait1(&q_full[s], nq[s]++))) break;
                        tc_fence_after();
                        mma_dots<D>(tmem + s * 128, smem_u32(sm + L::OFF_Q + s * L::TILE), smem_u32(sm + L::OFF_KV + k.st * L::TILE));
                        mma_commit(&s_full[s]);
                        if (last_reader(s, 0)) mma_commit(&kv_empty[k.st]);
                        if ((s ? n1 : n0) == 1) mma_commit(&q_empty[s]);
                    }
                    for (int j = 0; ok && j < nn; ++j) {
                        clear_job[2] = ++steps;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int ns = s ? n1 : n0;
                            if (!ok || j >= ns) continue;
                            const bool more = j + 1 < ns;
                            if (!shared || s == 0 || j >= n0) {  // V(j) and K(j+1): the next two tiles
                                v = kv;
                                kv.next();
                                if (!(ok = wait1(&kv_full[v.st], v.ph))) break;
                                if (shared ? j + 1 < nn : more) {
                                    k = kv;
                                    kv.next();
                                }
                            }
                            // values behind the last key belong to something else and may be anything:
                            // their weights are 0, and 0 * NaN is NaN, so warp 10 clears them meanwhile
                            const int last = shared ? max(t.nkeys[0], t.nkeys[1]) : t.nkeys[s];
                            const bool dirty = t.foreign && last % kKeys != 0 && j == (shared ? nn : ns) - 1 &&
                                               (!shared || s == (n0 != nn));
                            if (dirty) request_clear(clear_req, clear_job, v.st, last % kKeys);
                            const uint32_t t_s = tmem + s * 128, t_o = tmem + 256 + s * D;
                            const uint32_t vs = smem_u32(sm + L::OFF_KV + v.st * L::TILE);
                            // the first half of P is multiplied while the second is still exponentials
                            if (!(ok = (!dirty || wait1(clean, nc++)) && wait1(&p_half[s], np[s]))) break;
                            tc_fence_after();
                            mma_sum<D, 32, 0, 4>(t_o, t_s, vs, j > 0);
                            if (!(ok = wait1(&p_full[s], np[s]++))) break;
                            tc_fence_after();
                            mma_sum<D, 32, 4, 8>(t_o, t_s, vs, 1);
                            if (last_reader(s, j)) mma_commit(&kv_empty[v.st]);
                            if (more) {  // (the wait hides behind the products just issued)
                                if (!(ok = wait1(&kv_full[k.st], k.ph))) break;
                                tc_fence_after();
                                mma_dots<D>(t_s, smem_u32(sm + L::OFF_Q + s * L::TILE), smem_u32(sm + L::OFF_KV + k.st * L::TILE));
                                mma_commit(&s_full[s]);
                                if (last_reader(s, j + 1)) mma_commit(&kv_empty[k.st]);
                                if (j + 2 == ns) mma_commit(&q_empty[s]);
                            } else {
                                mma_commit(&o_full[s]);
                            }
                        }
                    }
                }
                request_clear(clear_req, clear_job, -1, 0);
                finish_mma(done);
            }
            __syncwarp();
        } else if (warp == kWarpClear) {
            // ======================================================== values behind the last key
            clear_role(sm + L::OFF_KV, L::TILE, L::NH, clear_req, clean, clear_job, abort_flag, wait_ns, lane);
        }
    } else {
        // ============================================================ softmax, one warpgroup per stream
        reg_inc<216>();
        const int s = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + 256 + s * D;
        const int rt = r / a.G, rh = r % a.G;
        const float c = a.scale_log2;
        int ns_done = 0, no_done = 0, n_join = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const int ib = n % kItems;
            if (!(ok = wait(&item_full[ib], n / kItems, 3))) break;
            const int end = items[ib].end, g = items[ib].g, tok = items[ib].tok[s], ntok = items[ib].ntok[s],
                      nkeys = items[ib].nkeys[s], off = items[ib].off[s], slot = items[ib].slot;
            const bool merge = !items[ib].shared && items[ib].nkeys[1] > 0;  // both streams hold parts of the same rows
            __syncwarp();
            mbar_arrive_lane0(&item_empty[ib], lane);
            if (end) break;
            const int nt = tiles(nkeys);
            if (nt == 0) continue;
            const bool warp_rows = r - lane < ntok * a.G;         // some row of this warp is real
            const int lim = min(nkeys - 1, off + rt);             // last key this row sees
            const int lim_all = min(nkeys - 1, off);              // ... that every row sees
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < nt; ++j) {
                if (!(ok = wait(&s_full[s], ns_done, 3))) break;
                ++ns_done;
                if (warp_rows) {
                    tc_fence_after();
                    float x[128];
                    float(&x0)[32] = *reinterpret_cast<float(*)[32]>(x);
                    float(&x1)[32] = *reinterpret_cast<float(*)[32]>(x + 32);
                    float(&x2)[32] = *reinterpret_cast<float(*)[32]>(x + 64);
                    float(&x3)[32] = *reinterpret_cast<float(*)[32]>(x + 96);
                    tmem_ld32(ts, x0);
                    tmem_ld32(ts + 32, x1);
                    wait_loads(x0);
                    wait_loads(x1);
                    tmem_ld32(ts + 64, x2);  // in flight while the first half is worked on
                    tmem_ld32(ts + 96, x3);
                    const bool edge = j * kKeys + kKeys - 1 > lim_all;
                    const int last = lim - j * kKeys;
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) x[i] = i <= last ? x[i] : -INFINITY;
                    }
                    if (j == 0 || edge) {
                        wait_loads(x2);
                        wait_loads(x3);
                    }
                    if (edge) {
#pragma unroll
                        for (int i = 64; i < 128; ++i) x[i] = i <= last ? x[i] : -INFINITY;
                    }
                    if (j == 0) {
                        float mxs[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) mxs[i] = fmaxf(x[i], x[i + 8]);
#pragma unroll
                        for (int i = 16; i < 128; i += 16)
#pragma unroll
                            for (int e = 0; e < 8; ++e) mxs[e] = fmaxf(fmaxf(mxs[e], x[i + e]), x[i + 8 + e]);
                        m = c * fmaxf(fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])),
                                      fmaxf(fmaxf(mxs[4], mxs[5]), fmaxf(mxs[6], mxs[7])));
                    }
                    // Later tiles take their exponentials from the m so far; the tile's maximum is
                    // found meanwhile (other pipe), and if it exceeds m by too much, once more.
                    const float2 c2 = make_float2(c, c);
                    float2 sum0, sum1;
                    uint32_t u[32];
                    while (true) {
                        const float mn = m == -INFINITY ? 0.f : -m;
                        const float2 m2 = make_float2(mn, mn);
                        float mx0 = x[0], mx1 = x[1];
                        sum0 = sum1 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float2 y0 = fma2(make_float2(x[2 * i], x[2 * i + 1]), c2, m2);
                            float2 y1 = fma2(make_float2(x[2 * i + 2], x[2 * i + 3]), c2, m2);
                            mx0 = fmaxf(fmaxf(mx0, x[2 * i]), x[2 * i + 1]);
                            mx1 = fmaxf(fmaxf(mx1, x[2 * i + 2]), x[2 * i + 3]);
                            y0.x = ex2(y0.x); y0.y = ex2(y0.y);
                            y1.x = ex2(y1.x); y1.y = ex2(y1.y);
                            sum0 = add2(sum0, y0);
                            sum1 = add2(sum1, y1);
                            u[i] = bf16_pair(y0.x, y0.y);
                            u[i + 1] = bf16_pair(y1.x, y1.y);
                        }
                        wait_loads(x2);
                        wait_loads(x3);
                        float mx2 = x[64], mx3 = x[65];
#pragma unroll
                        for (int i = 66; i < 126; i += 4) {
                            mx0 = fmaxf(fmaxf(mx0, x[i]), x[i + 1]);
                            mx1 = fmaxf(fmaxf(mx1, x[i + 2]), x[i + 3]);
                        }
                        mx2 = fmaxf(mx2, x[126]);
                        mx3 = fmaxf(mx3, x[127]);
                        const float mx = c * fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
                        if (!__any_sync(0xffffffffu, mx > m + kSlack)) break;
                        const float f = mx > m + kSlack ? ex2(m - mx) : 1.f;
                        m = mx > m + kSlack ? mx : m;
                        l *= f;
                        if (j == 0) continue;
                        // S(j) is complete, so P.V(j-1) issued before it is, too
#pragma unroll 1
                        for (int h = 0; h < D / 16; ++h) rescale16(to + h * 16, f);
                        tmem_wait_st();
                    }
                    tmem_st32(ts, u);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_lane0(&p_half[s], lane);
                    {
                        const float mn = m == -INFINITY ? 0.f : -m;
                        const float2 m2 = make_float2(mn, mn);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float2 y0 = fma2(make_float2(x[2 * i + 64], x[2 * i + 65]), c2, m2);
                            float2 y1 = fma2(make_float2(x[2 * i + 66], x[2 * i + 67]), c2, m2);
                            y0.x = ex2(y0.x); y0.y = ex2(y0.y);
                            y1.x = ex2(y1.x); y1.y = ex2(y1.y);
                            sum0 = add2(sum0, y0);
                            sum1 = add2(sum1, y1);
                            u[i] = bf16_pair(y0.x, y0.y);
                            u[i + 1] = bf16_pair(y1.x, y1.y);
                        }
                    }
                    tmem_st32(ts + 32, u);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_lane0(&p_full[s], lane);
                    sum0 = add2(sum0, sum1);
                    l += sum0.x + sum0.y;
                } else {
                    mbar_arrive_lane0(&p_half[s], lane);
                    mbar_arrive_lane0(&p_full[s], lane);
                }
            }
            if (!ok || !(ok = wait(&o_full[s], no_done, 3))) break;
            ++no_done;
            tc_fence_after();
            // Streams that split the keys of the same rows: stream 1 hands over m and l, stream 0 reads
            // both O (a warp reaches its 32 rows in every column) and writes one joint result.
            float f1 = 0.f;
            if (merge && s == 1) {
                joint[r] = m;
                joint[128 + r] = l;
                tc_fence_before();
                __syncwarp();
                mbar_arrive_lane0(join_full, lane);
                if (!(ok = wait(join_empty, n_join++, 3))) break;
                continue;
            }
            float z = l, f = 1.f, mm = m == -INFINITY ? 0.f : m;
            if (merge) {
                if (!(ok = wait(join_full, n_join++, 3))) break;
                tc_fence_after();
                const float m1 = joint[r], top = fmaxf(m, m1);
                mm = top == -INFINITY ? 0.f : top;
                f = ex2(m - mm);
                f1 = ex2(m1 - mm);
                z = l * f + joint[128 + r] * f1;
            }
            const bool real = r < ntok * a.G;
            const int64_t row = ((int64_t)tok + rt) * a.hq + g * a.G + rh;
            if (!DECODE && a.off_by_one) {  // the added 1 is a logit of 0
                const float top = fmaxf(mm, 0.f), e = ex2(mm - top);
                f *= e;
                f1 *= e;
                z = z * e + ex2(-top);
                mm = top;
            }
            const float inv = z > 0.f ? f / z : (z == 0.f ? 0.f : z), inv1 = merge && z > 0.f ? f1 / z : 0.f;  // NaN stays NaN
            const float lse = (mm + lg2(z)) * kLn2;
            const int64_t prow = (int64_t)slot * a.B * a.hq + row;
            if (warp_rows && real) {
                if (DECODE) a.plse[prow] = lse;
                else if (a.lse) a.lse[row] = lse;
            }
            const QuadRows out(DECODE ? static_cast<void *>(a.po + prow * D) : static_cast<__nv_bfloat16 *>(a.o) + row * D,
                               warp_rows && real, lane);
            // rolled: this code runs once per item and would be fetched anew each time
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
                if (!warp_rows) break;
                float y[32];
                tmem_ld32(to + h * 32, y);
                wait_loads(y);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] *= inv;
                if (merge) {
                    float y1[32];
                    tmem_ld32(to + D + h * 32, y1);
                    wait_loads(y1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] += y1[i] * inv1;
                }
                if constexpr (DECODE) out.store_f32(y, h * 128, lane);
                else out.store_bf16(y, 1.f, h * 64, lane);
                __syncwarp();
            }
            tc_fence_before();
            if (merge) {
                __syncwarp();
                mbar_arrive_lane0(join_empty, lane);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int D, bool DECODE>
cudaError_t launch(const Args &a, int64_t items, int32_t *next, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    const uint64_t rows = (uint64_t)a.B * (a.decode ? 1 : a.L), planes = (uint64_t)a.hkv * (a.decode ? 1 : a.B);
    if (!make_map3(&mq, a.q, D, a.hq, D, rows, (uint64_t)a.hq * D, a.G, 128 / a.G) ||
        !make_map3(&mk, a.k[0], D, a.L, D, planes, a.plane[0], kKeys, 1) ||
        !make_map3(&mv, a.v[0], D, a.L, D, planes, a.plane[0], kKeys, 1))
        return cudaErrorInvalidValue;
    const size_t smem = Smem<D>::ALLOC;
    cudaError_t e = set_smem_once((const void *)fwd_tc_kernel<D, DECODE>, smem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>(items, sm_count());
    if (!a.plan && items <= grid) next = nullptr;
    else if (!a.plan && (e = cudaMemsetAsync(a.ds, 0, kWsHeader, st)) != cudaSuccess) return e;
    return launch_next(a.plan != nullptr, fwd_tc_kernel<D, DECODE>, grid, kThreads, smem, st, 1, mq, mk, mv, a, next,
                       wait_limit_ns());
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        return EncodeTiledFn(nullptr);
    }();
    return fn;
}

}  // namespace

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && (n = known[dev].load(std::memory_order_relaxed))) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    if (keep) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool make_map3(CUtensorMap *m, const void *base, uint64_t cols, uint64_t n1, uint64_t s1, uint64_t n2, uint64_t s2,
               uint32_t b1, uint32_t b2) {
    EncodeTiledFn enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[3] = {cols, n1, n2};
    cuuint64_t strides[2] = {s1 * 2, s2 * 2};
    cuuint32_t box[3] = {64, b1, b2};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_fwd_tc(const Args &a, int d, int64_t items, int32_t *next, cudaStream_t st) {
    if (a.decode) return d == 128 ? launch<128, true>(a, items, next, st) : launch<64, true>(a, items, next, st);
    return d == 128 ? launch<128, false>(a, items, next, st) : launch<64, false>(a, items, next, st);
}

}  // namespace dense
}  // namespace hsa
