// ptx_serve.cuh -- inline-PTX building blocks of the serving kernels beside those of ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace mha {

// named_bar_and with OR.
__device__ __forceinline__ bool named_bar_or(int id, int nthreads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(nthreads)
        : "memory");
    return r != 0;
}

// (a.x * b.x, a.y * b.y), round to nearest.
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// top * tanh(x), to about 2^-21 of itself for any x: up to |x| = 0.7 x P(x^2) with a minimax P of degree 4 (Remez
// exchange on the relative error: 2^-21.6, coefficients below), beyond it top - 2 top / (1 + e^2x), off by 2^-22 of top.
// The second form alone would be off by that much for small x too: with a cap far above the scores by more than a
// score's own digits (a cap of 10^6: weights off by 15 %).
constexpr float kTanh0 = 0.9999997019767761f, kTanh1 = -0.3333021402359009f, kTanh2 = 0.13281112909317017f,
                kTanh3 = -0.0508362352848053f, kTanh4 = 0.01377371046692133f;
constexpr float kTanhNear = 0.7f;
__device__ __forceinline__ float capped_score(float x, float top) {
    const float y = x * x;
    const float p = fmaf(fmaf(fmaf(fmaf(kTanh4, y, kTanh3), y, kTanh2), y, kTanh1), y, kTanh0);
    const float e = fmaf(-2.0f * top, rcp_approx(1.0f + ex2_approx(x * 2.8853900817779268f)), top);   // 2 log2(e)
    return fabsf(x) <= kTanhNear ? top * (x * p) : e;
}

// 16 bytes to shared memory; not live: zeros, nothing is read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// 4 bytes, the same way.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Loads from the shared memory of a CTA of the cluster (shared::cluster address).
__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

}  // namespace mha
