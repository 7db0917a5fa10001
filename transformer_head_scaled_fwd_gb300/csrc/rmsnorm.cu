// rmsnorm.cu -- RMS norm of rows with the residual's addition before it and, on request, output in
// e4m3 with one scale a row or a group of the row.
//
//   z = x + r;  y = gain * z / sqrt(mean(z^2) + eps);  e4m3: scale = max |y| / 448, y8 = y / scale
// The squares are summed in fp32 from the fp32 z (not from its bf16 rounding, which only the stored
// sum goes through); y is rounded once, to its own type. HBM-bound: x and r read, z and y written.
#include <cuda_fp8.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr float kE4M3Max = 448.0f;

__device__ __forceinline__ uint8_t to_e4m3(float v) {
    return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
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
        const float scale = top == 0.0f ? 1.0f : top / kE4M3Max;
        if (whole ? threadIdx.x == 0 : lane == 0) p.scales[row * groups + g] = scale;
        for (int i = i0; i < i1; i += step) {
            const float v = y_of(i);
            if (sum) store_f(sum + i, z_of(i));
            y[i] = to_e4m3(v / scale);
        }
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormParams& p, bool bf16, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.rows));
    return bf16 ? launch_pdl(rmsnorm_any_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, p)
                : launch_pdl(rmsnorm_any_kernel<float>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace mha
