// rotary.cu -- rotary positions of queries and keys, and the append of new keys and values to
// a paged cache on the same pass.
//
// Pair (x_0, x_1) of a token at position t turns by t * inv_freq[i]. The angle is formed in half
// turns as an unevaluated sum of two floats (error-free product by fused multiply-add, after
// Dekker): t * f in one float is off by up to 2^-25 of its size, 0.03 rad at t = 10^6. Whole turns
// are removed exactly before the sum is rounded, so cos and sin are good to a few 2^-24 anywhere.
//
// HBM-bound: every element is read once and written once (keys twice where k_out is asked for).
#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kThreads = 256;

// (cos, sin) of pos * f
__device__ __forceinline__ float2 turn_of(int pos, float f) {
    constexpr float kInvPi = 0.318309873342514038f;        // 1 / pi rounded to fp32 ...
    constexpr float kInvPiLow = 1.28412766334e-8f;         // ... and the rest
    const float ph = f * kInvPi;
    const float pl = fmaf(f, kInvPiLow, fmaf(f, kInvPi, -ph));
    const float th = static_cast<float>(pos);
    const float tl = static_cast<float>(static_cast<long long>(pos) - static_cast<long long>(th));
    const float ah = th * ph;
    float al = fmaf(th, ph, -ah);
    al = fmaf(th, pl, al);
    al = fmaf(tl, ph, al);
    const float r = (ah - 2.0f * rintf(0.5f * ah)) + al;   // the difference is exact
    float2 cs;
    sincospif(r, &cs.y, &cs.x);
    return cs;
}

// One token per CTA: the token's cos and sin once in shared memory, then its heads, one pair or
// one plain element an item.
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    extern __shared__ float2 turns[];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x / p.T;
    const int t = blockIdx.x - b * p.T;
    if (p.new_lens != nullptr && t >= p.new_lens[b]) return;
    const int at = p.start != nullptr ? p.start[b] + t : t;
    const int pos = p.positions != nullptr ? p.positions[static_cast<int64_t>(b) * p.T + t] : at;
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const float2 cs = turn_of(pos, p.inv_freq[i]);
        turns[i] = make_float2(cs.x * p.scale, cs.y * p.scale);
    }
    T* page_k = nullptr;
    T* page_v = nullptr;
    if (p.cache.k != nullptr) {
        const int n = at >= 0 ? p.cache.page.div(at) : -1;
        int page = -1;
        if (n >= 0 && n < p.cache.max_pages) page = p.cache.table[b * p.cache.table_stride + n];
        if (page >= 0 && page < p.cache.n_pages) {
            const int64_t off = page * p.cache.page_stride + (at - n * static_cast<int>(p.cache.page.d)) * p.cache.slot_stride;
            page_k = static_cast<T*>(p.cache.k) + off;
            page_v = static_cast<T*>(p.cache.v) + off;
        } else if (threadIdx.x == 0) {
            atomicCAS(p.status, 0, 0x501);   // the token has no slot: it is not appended
        }
    }
    __syncthreads();
    const int rest = p.d - p.rot;
    const int items = half + rest;            // per turned head
    const int nq = p.q.p != nullptr ? p.h : 0, nk = p.k.p != nullptr ? p.h_kv : 0;
    for (int i = threadIdx.x; i < (nq + nk) * items; i += kThreads) {
        const int head = i / items;
        const int c = i - head * items;
        const bool is_q = head < nq;
        const int hd = is_q ? head : head - nq;
        const Strided& in = is_q ? p.q : p.k;
        const Strided& out = is_q ? p.q_out : p.k_out;
        const T* x = static_cast<const T*>(in.p) + b * in.b + t * in.l + hd * in.h;
        T* y = out.p != nullptr ? static_cast<T*>(out.p) + b * out.b + t * out.l + hd * out.h : nullptr;
        T* z = !is_q && page_k != nullptr ? page_k + hd * p.cache.head_stride : nullptr;
        if (c < half) {
            const int i0 = p.interleaved ? 2 * c : c, i1 = p.interleaved ? 2 * c + 1 : c + half;
            const float a = load_f(x + i0), e = load_f(x + i1);
            const float2 cs = turns[c];
            const float u = fmaf(a, cs.x, -(e * cs.y)), w = fmaf(e, cs.x, a * cs.y);
            if (y) { store_f(y + i0, u); store_f(y + i1, w); }
            if (z) { store_f(z + i0, u); store_f(z + i1, w); }
        } else {
            const int i0 = p.rot + c - half;
            const T raw = x[i0];
            if (y) y[i0] = raw;
            if (z) z[i0] = raw;
        }
    }
    if (page_v != nullptr) {
        for (int i = threadIdx.x; i < p.h_kv * p.d; i += kThreads) {
            const int hd = i / p.d;
            const int c = i - hd * p.d;
            page_v[hd * p.cache.head_stride + c] =
                static_cast<const T*>(p.v.p)[b * p.v.b + t * p.v.l + hd * p.v.h + c];
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, bool bf16, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.T);
    const size_t smem = sizeof(float2) * (p.rot / 2);
    return bf16 ? launch_pdl(rotary_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), smem, s, p)
                : launch_pdl(rotary_kernel<float>, dim3(grid), dim3(kThreads), smem, s, p);
}

}  // namespace mha
