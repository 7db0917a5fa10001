// paged_attn.cu -- attention of one new token a sequence over a paged key/value cache.
//
//   s_j = cap tanh(scale q.k_j / cap) - slope (n - 1 - j),  o = sum_j softmax_j(s) v_j,  j < n
// in one pass with a running maximum m and sum l (o and l are multiplied by exp(m_old - m_new)
// when m grows). n = 0 gives zeros.
#include <algorithm>

#include <math_constants.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kWarps = 8;

// CTA per (sequence, query head): a warp takes every kWarps-th key, d / 32 features a lane.
template <typename T, int kD>
__global__ void __launch_bounds__(32 * kWarps) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int kPer = kD / 32;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][kD];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y, head = blockIdx.x;
    const int kvh = head / (p.h / p.h_kv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t room = static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d;
    int n = max(p.kv_lens[b], 0);
    if (n > room) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, 0x501);
        n = static_cast<int>(room);
    }
    const float slope = p.slopes != nullptr ? p.slopes[head] : 0.0f;
    float q[kPer], o[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        q[e] = load_f(static_cast<const T*>(p.q) + b * p.q_b + head * p.q_h + lane + 32 * e);
        o[e] = 0.0f;
    }
    float m = -CUDART_INF_F, l = 0.0f;
    for (int j = warp; j < n; j += kWarps) {
        const int pi = p.cache.page.div(j);
        const int page = p.cache.table[b * p.cache.table_stride + pi];
        if (page < 0 || page >= p.cache.n_pages) {
            if (lane == 0) atomicCAS(p.status, 0, 0x501);
            continue;
        }
        const int64_t off = page * p.cache.page_stride + (j - pi * static_cast<int>(p.cache.page.d)) * p.cache.slot_stride +
                            kvh * p.cache.head_stride + lane;
        const T* k = static_cast<const T*>(p.cache.k) + off;
        const T* v = static_cast<const T*>(p.cache.v) + off;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) s = fmaf(q[e], load_f(k + 32 * e), s);
        s = warp_add(s) * p.scale;
        if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
        s -= slope * static_cast<float>(n - 1 - j);
        const float m_new = fmaxf(m, s);
        const float alpha = expf(m - m_new), w = expf(s - m_new);
        l = l * alpha + w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, load_f(v + 32 * e), o[e] * alpha);
        m = m_new;
    }
    if (lane == 0) { sm_m[warp] = m; sm_l[warp] = l; }
#pragma unroll
    for (int e = 0; e < kPer; ++e) sm_o[warp][lane + 32 * e] = o[e];
    __syncthreads();
    if (threadIdx.x < kD) {
        float M = -CUDART_INF_F;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
        float L = 0.0f, a = 0.0f;
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w] == -CUDART_INF_F ? 0.0f : expf(sm_m[w] - M);
            L += sm_l[w] * f;
            a += sm_o[w][threadIdx.x] * f;
        }
        store_f(static_cast<T*>(p.out) + b * p.o_b + head * p.o_h + threadIdx.x, L > 0.0f ? a / L : 0.0f);
    }
}

}  // namespace

size_t paged_attn_workspace(bool, int, int, int, int) { return 256; }

cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, cudaStream_t s) {
    const dim3 grid(p.h, p.B), block(32 * kWarps);
    if (bf16)
        return p.d == 64 ? launch_pdl(paged_attn_kernel<__nv_bfloat16, 64>, grid, block, 0, s, p)
                         : launch_pdl(paged_attn_kernel<__nv_bfloat16, 128>, grid, block, 0, s, p);
    return p.d == 64 ? launch_pdl(paged_attn_kernel<float, 64>, grid, block, 0, s, p)
                     : launch_pdl(paged_attn_kernel<float, 128>, grid, block, 0, s, p);
}

}  // namespace mha
