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
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
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
                report(ds, HSA_ERR_TIMEOUT, kKDense, role, 0);
                return false;
            }
            ok = mbar_try(bar, parity);
            if (__all_sync(0xffffffffu, ok)) break;
        }
    }
    return true;
}

template <int N> __device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ tensor maps (host)
// bf16, 64-column boxes of `b1` x `b2` rows, 128-byte swizzle: [n2][n1][cols] with
// strides s1 and s2 in elements
bool make_map3(CUtensorMap *m, const void *base, uint64_t cols, uint64_t n1, uint64_t s1, uint64_t n2, uint64_t s2,
               uint32_t b1, uint32_t b2);
bool tensor_maps_available();

}  // namespace dense
}  // namespace hsa
