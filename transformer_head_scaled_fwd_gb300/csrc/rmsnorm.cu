// rmsnorm.cu -- RMS norm of rows with the residual's addition before it and, on request, output in
// e4m3 with one scale a row or a group of the row.
//
//   z = x + r;  y = gain * z / sqrt(mean(z^2) + eps);  e4m3: scale = max |y| / 448, y8 = y / scale
// The squares are summed in fp32 from the fp32 z (not from its bf16 rounding, which only the stored
// sum goes through); y is rounded once, to its own type. HBM-bound: x and r read, z and y written. Measured back to back
// in bf16: 32768 x 4096 with residual, e4m3 output with a scale a row, 940 MB: 134 us, 7.0 TB/s (1.03 of measured copy
// bandwidth); 262144 x 512, bf16 output: 153 us (1.03); 32768 x 1001 (an element an access): 51 us (0.75).
#include <cuda_fp8.h>
#include <math_constants.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx_serve.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr float kE4M3Max = 448.0f;

// Two values to two bytes, low first, nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint8_t to_e4m3(float v) { return static_cast<uint8_t>(e4m3x2(v, 0.0f)); }

// The scale of a group whose largest value is `top` (a product: within 2^-23 of the quotient), and y / scale as an IEEE
// division rounds it: a product with an approximate reciprocal, corrected once by its exact remainder. (Divisions cost more
// than the rest of the pass: a group of 128 at d = 4096, 162 us with two divisions a group; the product alone gave the
// neighbouring code for one quotient in a million.) `up` keeps the reciprocal inside fp32's normal range.
struct Quant {
    float scale, up, by, inv;      // by = -scale * up
    __device__ __forceinline__ explicit Quant(float top) {
        up = top < 0x1p-100f ? 0x1p100f : top > 0x1p100f ? 0x1p-100f : 1.0f;
        scale = top * (1.0f / kE4M3Max);
        if (scale == 0.0f) scale = 1.0f;
        by = top < CUDART_INF_F ? -scale * up : 0.0f;    // infinite: inv is 0, and so is every finite quotient
        inv = rcp_approx(scale * up);
    }
    __device__ __forceinline__ float operator()(float y) const {
        const float n = y * up, q = n * inv;
        return fmaf(fmaf(q, by, n), inv, q);
    }
    // Two at a time, packed (32768 x 4096 without residual: 87 us, one at a time 92 us, without the correction 84 us)
    __device__ __forceinline__ void pair(float& a, float& b) const {
        float2 n = make_float2(a, b);
        if (up != 1.0f) n = fmul2(n, make_float2(up, up));
        const float2 q = fmul2(n, make_float2(inv, inv));
        const float2 r = ffma2(ffma2(q, make_float2(by, by), n), make_float2(inv, inv), q);
        a = r.x;
        b = r.y;
    }
};

// Accesses of 16 bytes (Vec) or, for rows of odd length or start, of one element (One).
template <typename T_>
struct One {
    using T = T_;
    using Raw = T_;
    static constexpr int kN = 1;
    static __device__ __forceinline__ Raw zero() { return T(0.0f); }
    static __device__ __forceinline__ void unpack(Raw v, float (&f)[1]) { f[0] = load_f(&v); }
    static __device__ __forceinline__ void store(T* p, const float (&f)[1]) { store_f(p, f[0]); }
};
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    using T = __nv_bfloat16;
    using Raw = uint4;
    static constexpr int kN = 8;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __bfloat1622float2(h[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
        uint4 v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        *reinterpret_cast<uint4*>(p) = v;
    }
};
template <>
struct Vec<float> {
    using T = float;
    using Raw = uint4;
    static constexpr int kN = 4;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};

template <int kN>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[kN]) {
    if constexpr (kN == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16, e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16);
    else if constexpr (kN == 4)
        *reinterpret_cast<uint32_t*>(p) = e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16;
    else
        *p = to_e4m3(f[0]);
}

// Sum (or maximum) over the kThr threads of a row; for more than a warp one barrier of theirs, `part` is used once.
template <int kThr, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* part) {
#pragma unroll
    for (int o = (kThr < 32 ? kThr : 32) / 2; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = kMax ? fmaxf(v, w) : v + w;
    }
    if constexpr (kThr > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x % kThr / 32] = v;
        named_bar_sync(1 + threadIdx.x / kThr, kThr);
        v = part[0];
#pragma unroll
        for (int i = 1; i < kThr / 32; ++i) v = kMax ? fmaxf(v, part[i]) : v + part[i];
    }
    return v;
}

// Rows a CTA takes: as many as fill its 256 threads, because an SM starts CTAs one after the other, each in about 0.2
// us (32768 rows of 501: 39 us with a CTA of 64 threads each, 27 us so; 32768 x 4096 without residual, 128 threads a row:
// 108 us with one row a CTA, 84 us with two).
__host__ __device__ constexpr int rows_of_cta(int thr) { return kThreads / thr; }

// The row stays in registers between the passes: kThr threads a row, kC accesses a thread. Groups need Vec (a group is up to 32 neighbouring lanes of one access;
// rows of fewer lanes hold no wider group than that, or are one group).
template <typename V, int kThr, int kC, bool kQuant>
__global__ void __launch_bounds__(kThr* rows_of_cta(kThr)) rmsnorm_row_kernel(const __grid_constant__ RmsNormParams p) {
    using T = typename V::T;
    using Raw = typename V::Raw;
    constexpr int kN = V::kN;
    constexpr int kRowsCta = rows_of_cta(kThr);
    __shared__ float part[2][kRowsCta][kThr < 32 ? 1 : kThr / 32];
    const int tid = threadIdx.x % kThr, sub = threadIdx.x / kThr;
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * kRowsCta + sub;
    const bool live = mine < p.rows;
    const int64_t row = kThr < 32 ? min(mine, p.rows - 1) : mine;
    pdl_trigger();
    pdl_wait();
    if (kThr >= 32 && !live) return;      // all threads of the row: its barriers are its own
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* r = static_cast<const T*>(p.residual) + row * p.r_stride;
    const T* gain = static_cast<const T*>(p.gain);
    Raw raw[kC], res[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int i = (c * kThr + tid) * kN;
        raw[c] = i < p.d ? *reinterpret_cast<const Raw*>(x + i) : V::zero();
        res[c] = p.residual != nullptr && i < p.d ? *reinterpret_cast<const Raw*>(r + i) : V::zero();
    }
    float z[kC][kN];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        float a[kN], b[kN];
        V::unpack(raw[c], a);
        V::unpack(res[c], b);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            z[c][e] = a[e] + b[e];
            ss = fmaf(z[c][e], z[c][e], ss);
        }
    }
    if (p.sum != nullptr) {
        T* sum = static_cast<T*>(p.sum) + row * p.s_stride;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = (c * kThr + tid) * kN;
            if (live && i < p.d) V::store(sum + i, z[c]);
        }
    }
    const float inv = rsqrtf(row_reduce<kThr, false>(ss, part[0][sub]) / p.d + p.eps);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int i = (c * kThr + tid) * kN;
        float g[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) g[e] = 1.0f;
        if (gain != nullptr && i < p.d) V::unpack(*reinterpret_cast<const Raw*>(gain + i), g);
#pragma unroll
        for (int e = 0; e + 1 < kN; e += 2) {
            const float2 v = fmul2(fmul2(make_float2(z[c][e], z[c][e + 1]), make_float2(inv, inv)), make_float2(g[e], g[e + 1]));
            z[c][e] = v.x;
            z[c][e + 1] = v.y;
        }
        if constexpr (kN == 1) z[c][0] = z[c][0] * inv * g[0];
    }
    if constexpr (!kQuant) {
        T* y = static_cast<T*>(p.y) + row * p.y_stride;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = (c * kThr + tid) * kN;
            if (live && i < p.d) V::store(y + i, z[c]);
        }
    } else {
        uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.y_stride;
        const bool whole = p.group == p.d;
        float top[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            top[c] = 0.0f;
#pragma unroll
            for (int e = 0; e < kN; ++e) top[c] = fmaxf(top[c], fabsf(z[c][e]));
        }
        if (whole) {
#pragma unroll
            for (int c = 1; c < kC; ++c) top[0] = fmaxf(top[0], top[c]);
            top[0] = row_reduce<kThr, true>(top[0], part[1][sub]);
            if (live && tid == 0) p.scales[row] = Quant(top[0]).scale;
#pragma unroll
            for (int c = 1; c < kC; ++c) top[c] = top[0];
        } else {
            // a group is p.group / kN neighbouring lanes (4 to 32) of one chunk
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int i = (c * kThr + tid) * kN;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    if (o * kN < p.group) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], o));
                if (live && i < p.d && (i & (p.group - 1)) == 0)
                    p.scales[row * (p.d >> p.group_log2) + (i >> p.group_log2)] = Quant(top[c]).scale;
            }
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int i = (c * kThr + tid) * kN;
            const Quant quant(top[c]);
            if constexpr (kN > 1) {
#pragma unroll
                for (int e = 0; e < kN; e += 2) quant.pair(z[c][e], z[c][e + 1]);
            } else if (c % 2 == 0) {
                quant.pair(z[c][0], z[c + 1][0]);      // one group a row
            }
            if (live && i < p.d) store_e4m3<kN>(y + i, z[c]);
        }
    }
}

// CTA per row, any d and any alignment: the row is read again from cache for each pass.
template <typename T>
__global__ void __launch_bounds__(kThreads) rmsnorm_any_kernel(const __grid_constant__ RmsNormParams p) {
    __shared__ float part[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.r_stride : nullptr;
    T* sum = p.sum ? static_cast<T*>(p.sum) + row * p.s_stride : nullptr;
    const T* gain = static_cast<const T*>(p.gain);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto z_of = [&](int i) { return load_f(x + i) + (r ? load_f(r + i) : 0.0f); };
    float ss = 0.0f;
    for (int i = threadIdx.x; i < p.d; i += kThreads) {
        const float z = z_of(i);
        ss = fmaf(z, z, ss);
    }
    ss = warp_add(ss);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) ss += part[w];
    const float inv = rsqrtf(ss / p.d + p.eps);
    auto y_of = [&](int i) { return z_of(i) * inv * (gain ? load_f(gain + i) : 1.0f); };
    if (p.scales == nullptr) {
        T* y = static_cast<T*>(p.y) + row * p.y_stride;
        for (int i = threadIdx.x; i < p.d; i += kThreads) {
            const float v = y_of(i);
            if (sum) store_f(sum + i, z_of(i));   // after the last read of x and r at i
            store_f(y + i, v);
        }
        return;
    }
    uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.y_stride;
    const int groups = p.d / p.group;
    // a warp takes whole groups; one group a row is shared by all warps
    const bool whole = groups == 1;
    for (int g = whole ? 0 : warp; g < groups; g += whole ? 1 : kThreads / 32) {
        const int i0 = g * p.group + (whole ? static_cast<int>(threadIdx.x) : lane);
        const int i1 = (g + 1) * p.group, step = whole ? kThreads : 32;
        float top = 0.0f;
        for (int i = i0; i < i1; i += step) top = fmaxf(top, fabsf(y_of(i)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (whole) {
            __syncthreads();
            if (lane == 0) part[warp] = top;
            __syncthreads();
            for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, part[w]);
        }
        const Quant quant(top);
        if (whole ? threadIdx.x == 0 : lane == 0) p.scales[row * groups + g] = quant.scale;
        for (int i = i0; i < i1; i += step) {
            const float v = y_of(i);
            if (sum) store_f(sum + i, z_of(i));
            y[i] = to_e4m3(quant(v));
        }
    }
}

template <typename V, int kThr, int kC>
cudaError_t launch_row(const RmsNormParams& p, cudaStream_t s) {
    constexpr int kRowsCta = rows_of_cta(kThr);
    const dim3 grid(static_cast<unsigned>((p.rows + kRowsCta - 1) / kRowsCta)), block(kThr * kRowsCta);
    return p.scales != nullptr ? launch_pdl(rmsnorm_row_kernel<V, kThr, kC, true>, grid, block, 0, s, p)
                               : launch_pdl(rmsnorm_row_kernel<V, kThr, kC, false>, grid, block, 0, s, p);
}

template <typename T>
cudaError_t launch_t(const RmsNormParams& p, cudaStream_t s) {
    using V = Vec<T>;
    using O = One<T>;
    constexpr int kN = V::kN;
    auto ok = [&](const void* q, int64_t stride) {
        return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && (p.rows == 1 || stride % kN == 0);
    };
    const bool y_ok = p.scales != nullptr ? reinterpret_cast<uintptr_t>(p.y) % kN == 0 && (p.rows == 1 || p.y_stride % kN == 0)
                                          : ok(p.y, p.y_stride);
    if (p.d % kN == 0 && ok(p.x, p.x_stride) && ok(p.residual, p.residual ? p.r_stride : 0) &&
        ok(p.sum, p.sum ? p.s_stride : 0) && ok(p.gain, 0) && y_ok) {
        // Four accesses a thread keep enough bytes in flight (32768 x 4096 without a residual: 84 us, with two 130 us);
        // when there are fewer rows than four for each of 152 SMs, twice the threads finish a row sooner (16 x 1024: 6.7 against
        // 8.2 us with the launch).
        const bool few = p.rows <= 608;
        const int chunks = p.d / kN;
        // Narrow rows (a norm of each head) share a warp, whose instructions then serve several (1310720 x 128: 232 us with a
        // warp a row, 126 us with 16 lanes and one access each, 103 us with 8 and two; x 64: 229, 64 and 53 us; 524288 x 256: 100 us with
        // 32 lanes, 82 us with 16). 64 chunks keep 32 lanes: a group of 128 fp32 elements has as many.
        if (chunks <= 8) return launch_row<V, 4, 2>(p, s);
        if (chunks <= 16) return launch_row<V, 8, 2>(p, s);
        if (chunks <= 32) return launch_row<V, 16, 2>(p, s);
        if (chunks <= 64) return launch_row<V, 32, 2>(p, s);
        if (chunks <= 128) return few ? launch_row<V, 64, 2>(p, s) : launch_row<V, 32, 4>(p, s);
        if (chunks <= 256) return few ? launch_row<V, 128, 2>(p, s) : launch_row<V, 64, 4>(p, s);
        if (chunks <= 512) return few ? launch_row<V, 256, 2>(p, s) : launch_row<V, 128, 4>(p, s);
        if (chunks <= 1024) return launch_row<V, 256, 4>(p, s);
        if (chunks <= 2048) return launch_row<V, 256, 8>(p, s);
    } else if (p.scales == nullptr || p.group == p.d) {
        if (p.d <= 64) return launch_row<O, 16, 4>(p, s);
        if (p.d <= 128) return launch_row<O, 32, 4>(p, s);
        if (p.d <= 256) return launch_row<O, 32, 8>(p, s);
        if (p.d <= 512) return launch_row<O, 32, 16>(p, s);
        if (p.d <= 1024) return launch_row<O, 64, 16>(p, s);
        if (p.d <= 2048) return launch_row<O, 128, 16>(p, s);
        if (p.d <= 4096) return launch_row<O, 256, 16>(p, s);
        if (p.d <= 8192) return launch_row<O, 256, 32>(p, s);
    }
    return launch_pdl(rmsnorm_any_kernel<T>, dim3(static_cast<unsigned>(p.rows)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormParams& p, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace mha
