// attn_span.cuh -- what the two kernels of attention under span masks share: modes of the scores, row
// intervals, work stealing, capped and biased scores.
#pragma once

#include <math_constants.h>

#include <atomic>

#include "launch.h"
#include "mha_internal.h"
#include "ptx_pair.cuh"
#include "ptx_serve.cuh"
#include "serve.h"

namespace mha {

struct SpanMaps {
    CUtensorMap q, k, v, out;   // {64, L, d_k / 64, heads, B}, box {64, 128, d_k / 64, 1, 1}
};
namespace {

constexpr int BN = 128;          // keys of a tile
constexpr uint32_t kHalf = 128 * 128;        // one 128-row x 64-column bf16 half tile = 16 KB
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;    // log2 units that a row's maximum may grow before O and l are rescaled
constexpr int kHeadGroup = 8;                // (batch, head) pairs whose units run together

// How scores become weights:
//   kPlain   scale > 0, no cap, no bias: running maximum of the raw scores, one multiply-add each
//   kCapped  a cap, no bias: scores formed first, relative to the running maximum already. Most tiles cannot raise it, which
//            their largest |q.k| tells, and then their own maximum is not formed (4 x 8192 causal, 8 heads of 128, a cap
//            of 50: 476 us, with the maximum of every tile 501 us). A reference of 0 for all rows, which a small cap allows,
//            would save the agreement too (414 us), but under it a row's weights lie anywhere in e^+-cap, and large or tiny values
//            leave fp32's range in the sums
//   kGeneral anything else: scores formed first, then as kPlain
//   kSingle  as kGeneral, scale / cap outside the range of TanhForm: far scores one by one (an instance of its own: in the
//            others the branch alone cost 2 to 10 %)
enum Mode { kPlain, kCapped, kGeneral, kSingle };

// Coordinates of a (head, sequence) in a map: a broadcast dimension (stride 0) has one entry there.
__device__ __forceinline__ int at_h(const Strided& t, int head) { return t.h != 0 ? head : 0; }
__device__ __forceinline__ int at_b(const Strided& t, int b) { return t.b != 0 ? b : 0; }

__device__ __forceinline__ void tma_load_5d(const CUtensorMap* m, uint64_t* bar, void* dst, int c1, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(0), "r"(c1), "r"(c3), "r"(c4)
        : "memory");
}

// After a give-up: waits, with a limit of its own, until the copy that completes phase `parity` of `bar` has landed, so
// that none is in flight when the CTA's shared memory is released.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    for (uint32_t it = 0; it < (1u << 16) && !mbar_try_wait(a, parity); ++it) {
    }
}
// The last tiles of a ring of kStages into which `issued` were loaded.
template <int kStages>
__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t issued) {
    for (uint32_t i = 1; i <= kStages && i <= issued; ++i)
        drain(&full[(issued - i) % kStages], ((issued - i) / kStages) & 1);
}

// Work stealing: the grid has one CTA a unit; a running CTA asks the hardware to cancel the launch of
// one that has not started and does its unit instead (its set-up is paid once, and no counter in
// memory is needed). After a refusal no further request is made.
__device__ __forceinline__ void steal_request(void* answer, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}
// blockIdx.x of the cancelled CTA, or -1
__device__ __forceinline__ int steal_answer(const void* answer) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 x, y, z, w;\n\t"
        "ld.shared.b128 r, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "mov.b32 x, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {x, y, z, w}, r;\n\t"
        "mov.b32 %0, x;\n\t}"
        : "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return x;
}

// Keys [x, y) of query i: the unit's valid length and prefix, its own span.
__device__ __forceinline__ int2 interval_of(const SpanAttnParams& p, int valid, int seen, int2 span, int i) {
    const int hi = p.causal ? min(valid, max(i + p.q_offset + 1, seen)) : valid;
    return make_int2(max(span.x, 0), min(span.y, hi));
}
__device__ __forceinline__ int2 span_of(const SpanAttnParams& p, int b, int i) {
    if (p.spans == nullptr || i >= p.Lq) return make_int2(0, p.Lk);
    return reinterpret_cast<const int2*>(p.spans)[static_cast<int64_t>(b) * p.Lq + i];
}

template <int kKeys>
__device__ __forceinline__ void scale_scores(uint32_t (&u)[kKeys], float scale) {
#pragma unroll
    for (int c = 0; c < kKeys; c += 2) {
        const float2 r = fmul2(make_float2(__uint_as_float(u[c]), __uint_as_float(u[c + 1])), make_float2(scale, scale));
        u[c] = __float_as_uint(r.x);
        u[c + 1] = __float_as_uint(r.y);
    }
}

// u -> cap log2(e) tanh(u a), a = scale / cap. tanh(x) = x P(x^2) with minimax P (Remez exchange on the relative
// error): degree 2 for |x| <= 0.3, within 2^-19.7 of tanh, degree 4 for |x| <= 0.7, within 2^-21.2 in fp32 arithmetic; beyond,
// 1 - 2 / (1 + e^2x), within 2^-22 of 1 anywhere. Powers of a are folded into the coefficients, so a score costs two and
// a half instructions (packed) in the first range. Which range is decided for 16 scores of a warp at a time, so that near
// scores beside far ones are off by 2^-22 of the cap: 3 10^-4 of a weight at a = 2^-13 (a cap of 724 or 1024), which bf16
// weights hide. kSingle has the other caps, where that would be more than a score's own digits, or powers of a would leave
// fp32's range: it multiplies by a first, and takes far scores one by one (4 x 8192 causal, 8 heads of 128, a cap of 10^4: 567
// us, all scores one by one 866 us).
template <bool kAlone>
struct TanhForm {
    float pre, a, top;    // x = (u pre) a, one of the two is 1
    float near, mid;      // bounds of (u pre)^2
    __device__ __forceinline__ TanhForm(float a_, float top_) : pre(kAlone ? a_ : 1.0f), a(kAlone ? 1.0f : a_), top(top_) {
        near = 0.09f / (a * a);
        mid = 0.49f / (a * a);
    }
};
inline bool tanh_folds(float a) { return fabsf(a) >= 0x1p-13f && fabsf(a) <= 0x1p13f; }

// u becomes the score minus ref; the result is the largest (u pre)^2.
template <bool kAlone, int kKeys>
__device__ __forceinline__ float cap_scores(uint32_t (&u)[kKeys], const TanhForm<kAlone>& f, float ref) {
    if constexpr (kAlone) scale_scores(u, f.pre);
    const float t1 = f.a * f.top, a2 = f.a * f.a;
    const float n0 = 0.9999988675117493f * t1, n1 = -0.33310022950172424f * a2 * t1, n2 = 0.12633946537971497f * a2 * a2 * t1;
    const float2 d0 = make_float2(n0, n0), d1 = make_float2(n1, n1), d2 = make_float2(n2, n2), by = make_float2(-ref, -ref);
    const float end = f.top - ref;
    float farthest = 0.0f;
#pragma unroll
    for (int q = 0; q < kKeys / 16; ++q) {
        float2 y[8];
        float far = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 x = make_float2(__uint_as_float(u[16 * q + 2 * e]), __uint_as_float(u[16 * q + 2 * e + 1]));
            y[e] = fmul2(x, x);
            far = fmax3(far, y[e].x, y[e].y);
        }
        farthest = fmaxf(farthest, far);
        if (!__any_sync(0xffffffffu, far > f.near)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 x = make_float2(__uint_as_float(u[16 * q + 2 * e]), __uint_as_float(u[16 * q + 2 * e + 1]));
                const float2 r = ffma2(ffma2(ffma2(d2, y[e], d1), y[e], d0), x, by);
                u[16 * q + 2 * e] = __float_as_uint(r.x);
                u[16 * q + 2 * e + 1] = __float_as_uint(r.y);
            }
        } else if (!__any_sync(0xffffffffu, far > f.mid)) {
            const float m0 = kTanh0 * t1, m1 = kTanh1 * a2 * t1, m2 = kTanh2 * a2 * a2 * t1, m3 = kTanh3 * a2 * a2 * (a2 * t1),
                        m4 = kTanh4 * a2 * a2 * (a2 * a2 * t1);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 x = make_float2(__uint_as_float(u[16 * q + 2 * e]), __uint_as_float(u[16 * q + 2 * e + 1]));
                float2 r = ffma2(make_float2(m4, m4), y[e], make_float2(m3, m3));
                r = ffma2(r, y[e], make_float2(m2, m2));
                r = ffma2(r, y[e], make_float2(m1, m1));
                r = ffma2(ffma2(r, y[e], make_float2(m0, m0)), x, by);
                u[16 * q + 2 * e] = __float_as_uint(r.x);
                u[16 * q + 2 * e + 1] = __float_as_uint(r.y);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                if constexpr (kAlone) {
                    u[16 * q + e] = __float_as_uint(capped_score(__uint_as_float(u[16 * q + e]), f.top) - ref);
                    continue;
                }
                const float r = rcp_approx(1.0f + ex2_approx(__uint_as_float(u[16 * q + e]) * (f.a * 2.0f * kLog2e)));
                u[16 * q + e] = __float_as_uint(fmaf(-2.0f * f.top, r, end));
            }
        }
    }
    return farthest;
}

// u * scale - slope |i - j|: away = i - (first key of u), scale and slope in log2 units.
template <int kKeys>
__device__ __forceinline__ void bias_scores(uint32_t (&u)[kKeys], float scale, float away, float slope) {
    const bool below = away >= kKeys - 1.0f, above = away <= 0.0f;
    const float2 sc = make_float2(scale, scale);
    if (__all_sync(0xffffffffu, below) || __all_sync(0xffffffffu, above)) {   // |away - c| is linear in c
        const float s = __all_sync(0xffffffffu, below) ? slope : -slope;
        const float2 b = make_float2(-s * away, fmaf(-s, away, s)), step = make_float2(2.0f * s, 2.0f * s);
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c) {
            const float2 r = ffma2(make_float2(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1])), sc,
                                   ffma2(step, make_float2(c, c), b));
            u[2 * c] = __float_as_uint(r.x);
            u[2 * c + 1] = __float_as_uint(r.y);
        }
    } else {
#pragma unroll
        for (int c = 0; c < kKeys; ++c)
            u[c] = __float_as_uint(fmaf(-slope, fabsf(away - static_cast<float>(c)), __uint_as_float(u[c]) * scale));
    }
}

// A unit that the CTAs of a cluster share: each has its piece of the key tiles, and leaves its part in its shared memory:
// maxima of kUnit rows from m_at on, their sums behind them, outputs [row][part_pitch] from o_at on. A CTA joins kUnit /
// kPieces rows, a thread four features of a row of all parts at a time; all its loads are in flight together (one row after
// the other: 15.4 against 14.4 us at 128 x 2048 keys by two, d_k = 128, bf16).
__host__ __device__ constexpr int part_pitch(int d) { return d + 4; }
__device__ __forceinline__ void store4(__nv_bfloat16* y, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}
__device__ __forceinline__ void store4(float* y, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(y) = make_float4(a, b, c, d);
}
template <typename T, int kD, int kUnit, int kThr, int kPieces>
__device__ __forceinline__ void join_by(const SpanAttnParams& p, int b, int head, int q0, int piece, uint32_t m_at, uint32_t o_at) {
    constexpr int kRows = kUnit / kPieces, kCols = kD / 4, kStep = kThr / kCols;      // rows of one pass
    constexpr int kItems = kRows > kStep ? kRows / kStep : 1;
    const int c = threadIdx.x % kCols * 4, r0 = threadIdx.x / kCols;
    float ms[kItems][kPieces], ls[kItems][kPieces];
    float4 os[kItems][kPieces];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int r = piece * kRows + min(r0 + i * kStep, kRows - 1);
#pragma unroll
        for (int s = 0; s < kPieces; ++s) {
            ms[i][s] = ld_cluster(mapa_shared(m_at + r * 4, s));
            ls[i][s] = ld_cluster(mapa_shared(m_at + (kUnit + r) * 4, s));
            os[i][s] = ld_cluster4(mapa_shared(o_at + (r * part_pitch(kD) + c) * 4, s));
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int r = piece * kRows + r0 + i * kStep;
        if (r0 + i * kStep >= kRows || q0 + r >= p.Lq) continue;
        float M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
        for (int s = 0; s < kPieces; ++s) M = fmaxf(M, ms[i][s]);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kPieces; ++s) {
            if (ms[i][s] == -CUDART_INF_F) {   // no key: its output may hold anything; its sum is 0, or NaN if all scores are
                L += ls[i][s];
                continue;
            }
            const float f = ex2_approx(ms[i][s] - M);
            L = fmaf(f, ls[i][s], L);
            a.x = fmaf(f, os[i][s].x, a.x);
            a.y = fmaf(f, os[i][s].y, a.y);
            a.z = fmaf(f, os[i][s].z, a.z);
            a.w = fmaf(f, os[i][s].w, a.w);
        }
        const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);   // no key at all: zeros; NaN stays
        store4(static_cast<T*>(p.out.p) + b * p.out.b + (q0 + r) * p.out.l + head * p.out.h + c, a.x * inv, a.y * inv, a.z * inv,
               a.w * inv);
    }
}
template <typename T, int kD, int kUnit, int kThr>
__device__ __forceinline__ void join_parts(const SpanAttnParams& p, int b, int head, int q0, int pieces, int piece, uint32_t m_at,
                                           uint32_t o_at) {
    if (pieces == 2) join_by<T, kD, kUnit, kThr, 2>(p, b, head, q0, piece, m_at, o_at);
    else if (pieces == 4) join_by<T, kD, kUnit, kThr, 4>(p, b, head, q0, piece, m_at, o_at);
    else join_by<T, kD, kUnit, kThr, 8>(p, b, head, q0, piece, m_at, o_at);
}

// launch_pdl with clusters of `size` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, int size, size_t smem, cudaStream_t s,
                                      Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(size), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// Clusters of a kernel, allowed `smem` bytes by the caller, that the current device runs at once; asked once a device and
// size, for it is a property of the device.
struct ClusterRoom {
    static constexpr int kDevices = 64;
    std::atomic<int> known[kDevices][4] = {};      // by log2(size); 0: not asked, else 1 + the answer
    template <typename Kernel>
    int at_once(Kernel kernel, int threads, size_t smem, int size) {
        const int lg = size == 8 ? 3 : size == 4 ? 2 : 1;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
        if (const int k = known[dev][lg].load(std::memory_order_relaxed)) return k - 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {static_cast<unsigned>(size), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
        known[dev][lg].store(n + 1, std::memory_order_relaxed);
        return n;
    }
};

}  // namespace

cudaError_t launch_span_attn_d64(const SpanAttnParams& p, const SpanMaps& maps, int mode, cudaStream_t s);

}  // namespace mha
