// dense_tc.cuh -- pieces shared by the tensor-core kernels of dense attention:
// tensor maps, waits that give up, and small arithmetic helpers.
#pragma once

#include "dense.cuh"
#include "sm100.cuh"

namespace hsa {
namespace dense {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x with the hardware approximation (relative error about 2^-22, subnormals flushed)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// log2 with the hardware approximation (absolute error about 2^-22 near 1, relative beyond)
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
        "mov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 w, x, y;\n\t"
        "mov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Converged wait of a warp for phase `parity` of `bar`; false once it ran out (the
// first to run out sets *abort and reports) or another role gave up.  A limit below
// the timer's resolution (about 1 us) runs out at once: try_wait alone may sleep longer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns, volatile int *abort,
                                          DevStatus *ds, int role) {
    const bool at_once = limit_ns < 1000;
    bool ok = at_once ? mbar_test(bar, parity) : mbar_try(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = globaltimer();
        while (true) {
            if (__any_sync(0xffffffffu, *abort != 0)) return false;
            if (__any_sync(0xffffffffu, at_once || globaltimer() - t0 > limit_ns)) {
                *abort = 1;
                report(ds, HSA_ERR_TIMEOUT, kKDense, role, (int)((int64_t)(globaltimer() - t0) / 1000));
                return false;
            }
            ok = mbar_try(bar, parity);
            if (__all_sync(0xffffffffu, ok)) break;
        }
    }
    return true;
}

// The same for a role that a single thread plays: no votes, the shortest path from a
// barrier to the next instruction (a converged wait costs the issuing warp about 100
// cycles even when the phase is long complete).
__device__ __forceinline__ bool thread_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns, volatile int *abort,
                                            DevStatus *ds, int role) {
    const bool at_once = limit_ns < 1000;
    if (at_once ? mbar_test(bar, parity) : mbar_try(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (true) {
        if (*abort) return false;
        if (at_once || globaltimer() - t0 > limit_ns) {
            *abort = 1;
            report(ds, HSA_ERR_TIMEOUT, kKDense, role, (int)((int64_t)(globaltimer() - t0) / 1000));
            return false;
        }
        if (mbar_try(bar, parity)) return true;
    }
}

// The loads from tensor memory issued so far are complete; x may be read from here on
// (as an operand of the wait, so that no use can be scheduled before it).
__device__ __forceinline__ void wait_loads(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15])
                 :
                 : "memory");
    asm volatile(""
                 : "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]),
                   "+f"(x[23]), "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]),
                   "+f"(x[30]), "+f"(x[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Rows that the lanes of a warp hold one each (64 bytes at a time) go to global memory in
// pieces of 16 bytes that the four lanes of a quad first exchange, so that a store writes
// 64 consecutive bytes of 8 rows instead of 16 bytes of 32: the load/store unit takes a
// cycle per 128-byte line, and a direct store of a 128 x 128 tile keeps it for 2000.
struct QuadRows {
    char *row[4];  // this quad's rows (null: not stored), for piece `lane & 3`
    __device__ __forceinline__ QuadRows(void *mine, bool real, int lane) {
        const uint64_t p = real ? reinterpret_cast<uint64_t>(mine) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t q = __shfl_sync(0xffffffffu, p, (lane & ~3) + j);
            row[j] = q ? reinterpret_cast<char *>(q) + (lane & 3) * 16 : nullptr;
        }
    }
    // u: 64 bytes of the lane's own row, which start `offset` bytes into it
    __device__ __forceinline__ void store(uint32_t (&u)[16], int offset, int lane) const {
        const bool odd = lane & 1, high = lane & 2;
#pragma unroll
        for (int k = 0; k < 16; k += 8)  // pieces 0 <-> 1, 2 <-> 3 with the neighbour
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = __shfl_xor_sync(0xffffffffu, odd ? u[k + e] : u[k + 4 + e], 1);
                (odd ? u[k + e] : u[k + 4 + e]) = r;
            }
#pragma unroll
        for (int k = 0; k < 8; k += 4)  // pieces 0 <-> 2, 1 <-> 3 with the next pair
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = __shfl_xor_sync(0xffffffffu, high ? u[k + e] : u[k + 8 + e], 2);
                (high ? u[k + e] : u[k + 8 + e]) = r;
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row[j]) *reinterpret_cast<uint4 *>(row[j] + offset) = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
    }
    __device__ __forceinline__ void store_bf16(const float (&y)[32], float f, int offset, int lane) const {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = bf16_pair(y[2 * i] * f, y[2 * i + 1] * f);
        store(u, offset, lane);
    }
    __device__ __forceinline__ void store_f32(const float (&y)[32], int offset, int lane) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(y[16 * h + i]);
            store(u, offset + 64 * h, lane);
        }
    }
};

// One lane of a converged warp, always the same.  The compiler knows that a branch on
// it holds a single thread and keeps the operands of tcgen05.mma in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Descriptor of a 128-byte-swizzled tile at shared address `s` (smem_desc_sw128 with the
// strides of these kernels' tiles: 16 KB between 64-column halves, 1 KB between 8-row
// groups), split so that a step along the tile is one 32-bit addition.
struct Desc {
    uint32_t lo;
    __device__ __forceinline__ explicit Desc(uint32_t s) : lo(((s >> 4) & 0x3FFF) | (16384u >> 4) << 16) {}
    __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
        constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | 2u << 29;
        return (uint64_t)hi << 32 | (lo + (bytes >> 4));
    }
};

// D[128 x 128] = A B^T over d (16 d-columns per step), A and B K-major tiles
template <int D> __device__ __forceinline__ void mma_dots(uint32_t dst, uint32_t a, uint32_t b) {
    constexpr uint32_t id = idesc_bf16_f32(128, 128, false, false);
    const Desc da(a), db(b);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
        mma_bf16_ss(dst, da.at((ks >> 2) * 16384 + (ks & 3) * 32), db.at((ks >> 2) * 16384 + (ks & 3) * 32), id, ks > 0);
}
// D[128 x d] (+)= A B over 128: A in tensor memory as bf16 pairs, the second 64 of the
// contracted indices HALF columns behind the first; B a tile whose rows are contracted.
// Steps [K0, K1) of 16 indices.
template <int D, int HALF, int K0 = 0, int K1 = 8>
__device__ __forceinline__ void mma_sum(uint32_t dst, uint32_t a, uint32_t b, uint32_t add) {
    constexpr uint32_t id = idesc_bf16_f32(128, D, false, true);
    const Desc db(b);
#pragma unroll
    for (int ks = K0; ks < K1; ++ks)
        mma_bf16_ts(dst, a + (ks >> 2) * HALF + (ks & 3) * 8, db.at(ks * 2048), id, ks > K0 ? 1 : add);
}

// A position in a ring of N stages: the stage and the parity of its current use.
template <int N> struct Ring {
    uint32_t st = 0, ph = 0;
    __device__ __forceinline__ void next() {
        if (++st == N) {
            st = 0;
            ph ^= 1;
        }
    }
};

// The last loads issued into a ring of `stages` tiles have landed (bounded).  Every loader
// waits for its own before it leaves, also when all went well for it: another role may have
// given up on them, and the CTA's shared memory is the next CTA's once all roles are done.
__device__ __forceinline__ void land(uint64_t *full, int issued, int stages) {
    for (int i = max(0, issued - stages); i < issued; ++i) mbar_wait(&full[i % stages], (i / stages) & 1, kDrainWaitNs);
}
// Likewise the products that this thread has issued: it waits for them before it leaves, so
// that none is running when tensor memory is freed.
__device__ __forceinline__ void finish_mma(uint64_t *done) {
    mma_commit(done);
    mbar_wait(done, 0, kDrainWaitNs);
}

// Rows of a ring's tile that are summed over but belong to something else are set to
// zero by a warp of its own, at the request of the (single) MMA thread, which has seen
// the tile arrive and waits for `clean` before the product that reads it.  job: the
// stage (-1: no more requests), the first row, and the MMA thread's steps so far; one
// request at a time.
__device__ __forceinline__ void request_clear(uint64_t *req, volatile int *job, int stage, int row) {
    job[0] = stage;
    job[1] = row;
    mbar_arrive(req);
}
__device__ __forceinline__ void clear_role(uint8_t *ring, int tile_bytes, int halves, uint64_t *req, uint64_t *clean,
                                           volatile int *job, volatile int *abort, uint64_t limit_ns, int lane) {
    // Requests may be any time apart.  The MMA thread ends with a request or with the abort flag
    // set, and between two of its steps are at most 15 waits of limit_ns: while it makes steps
    // the role stays, and 32 such waits without one are the bound.
    const uint64_t idle_ns = limit_ns < (1ull << 58) ? 32 * limit_ns : 1ull << 63;
    uint64_t t0 = globaltimer();
    int steps = 0;
    for (int n = 0;; ++n) {
        while (!__all_sync(0xffffffffu, mbar_try(req, n & 1))) {
            const int s = job[2];
            if (s != steps) {
                steps = s;
                t0 = globaltimer();
            }
            if (__any_sync(0xffffffffu, *abort != 0 || globaltimer() - t0 > idle_ns)) return;
        }
        const int stage = job[0], row = job[1];
        if (stage < 0) return;
        uint8_t *tile = ring + stage * tile_bytes;
        for (int i = row * 8 + lane; i < 128 * 8; i += 32)
            for (int h = 0; h < halves; ++h)
                *reinterpret_cast<uint4 *>(tile + h * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_lane0(clean, lane);
    }
}

template <int N> __device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ launches (host)
int sm_count();  // of the current device
// bf16, 64-column boxes of `b1` x `b2` rows, 128-byte swizzle: [n2][n1][cols] with
// strides s1 and s2 in elements
bool make_map3(CUtensorMap *m, const void *base, uint64_t cols, uint64_t n1, uint64_t s1, uint64_t n2, uint64_t s2,
               uint32_t b1, uint32_t b2);

}  // namespace dense
}  // namespace hsa
