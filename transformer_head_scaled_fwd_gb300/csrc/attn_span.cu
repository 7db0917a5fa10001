// attn_span.cu -- attention with grouped heads over strided tensors, capped and biased scores,
// and masks that leave each query one interval of keys (document spans, prefix, causal, valid
// length: their intersection is an interval [lo, hi)). An empty interval gives a row of zeros.
#include <algorithm>

#include <math_constants.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kWarps = 4;

// Keys [x, y) of query i of sequence b.
__device__ __forceinline__ int2 interval_of(const SpanAttnParams& p, int b, int i) {
    int lo = 0, hi = p.Lk;
    if (p.valid_lens != nullptr) hi = min(hi, p.valid_lens[b]);
    if (p.causal) {
        int seen = i + p.q_offset + 1;
        if (p.prefix_lens != nullptr) seen = max(seen, p.prefix_lens[b]);
        hi = min(hi, seen);
    }
    if (p.spans != nullptr) {
        const int2 sp = reinterpret_cast<const int2*>(p.spans)[static_cast<int64_t>(b) * p.Lq + i];
        lo = max(lo, sp.x);
        hi = min(hi, sp.y);
    }
    return make_int2(lo, max(hi, lo));
}

// One warp per (query, head, sequence), d / 32 features a lane.
template <int kD>
__global__ void __launch_bounds__(32 * kWarps) span_attn_simple_kernel(const __grid_constant__ SpanAttnParams p) {
    constexpr int kPer = kD / 32;
    using T = __nv_bfloat16;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= p.Lq) return;
    const int head = blockIdx.y % p.h, b = blockIdx.y / p.h;
    const int kvh = head / (p.h / p.h_kv);
    const T* qr = static_cast<const T*>(p.q.p) + b * p.q.b + i * p.q.l + head * p.q.h + lane;
    const T* K = static_cast<const T*>(p.k.p) + b * p.k.b + kvh * p.k.h + lane;
    const T* V = static_cast<const T*>(p.v.p) + b * p.v.b + kvh * p.v.h + lane;
    float q[kPer], o[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        q[e] = load_f(qr + 32 * e);
        o[e] = 0.0f;
    }
    const float slope = p.slopes != nullptr ? p.slopes[head] : 0.0f;
    const int2 range = interval_of(p, b, i);
    float m = -CUDART_INF_F, l = 0.0f;
    for (int j = range.x; j < range.y; ++j) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) s = fmaf(q[e], load_f(K + j * p.k.l + 32 * e), s);
        s = warp_add(s) * p.scale;
        if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
        s -= slope * fabsf(static_cast<float>(i + p.q_offset - j));
        const float m_new = fmaxf(m, s);
        const float alpha = expf(m - m_new), w = expf(s - m_new);
        l = l * alpha + w;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, load_f(V + j * p.v.l + 32 * e), o[e] * alpha);
        m = m_new;
    }
    T* y = static_cast<T*>(p.out.p) + b * p.out.b + i * p.out.l + head * p.out.h + lane;
#pragma unroll
    for (int e = 0; e < kPer; ++e) store_f(y + 32 * e, range.y > range.x ? o[e] / l : 0.0f);
}

// spans[b, i]: the run of equal ids around i. One CTA per sequence; each thread finds the bounds of
// its positions from the nearest changes before and after them.
constexpr int kSpanThreads = 1024;
__global__ void __launch_bounds__(kSpanThreads) document_spans_kernel(const int32_t* ids, int L, int32_t* spans) {
    __shared__ int edge[kSpanThreads];
    pdl_trigger();
    pdl_wait();
    const int32_t* x = ids + static_cast<int64_t>(blockIdx.x) * L;
    int2* out = reinterpret_cast<int2*>(spans) + static_cast<int64_t>(blockIdx.x) * L;
    const int tid = threadIdx.x;
    // thread t owns positions [t per, (t + 1) per)
    const int per = (L + kSpanThreads - 1) / kSpanThreads;
    const int i0 = min(tid * per, L), i1 = min(i0 + per, L);
    // starts: the last change at or before a position
    int last = -1;
    for (int i = i0; i < i1; ++i)
        if (i == 0 || x[i] != x[i - 1]) last = i;
    edge[tid] = last;
    __syncthreads();
    for (int o = 1; o < kSpanThreads; o <<= 1) {
        const int other = tid >= o ? edge[tid - o] : -1;
        __syncthreads();
        edge[tid] = max(edge[tid], other);
        __syncthreads();
    }
    int start = tid > 0 ? edge[tid - 1] : 0;
    __syncthreads();
    for (int i = i0; i < i1; ++i) {
        if (i == 0 || x[i] != x[i - 1]) start = i;
        out[i].x = x[i] < 0 ? 0 : start;
    }
    // ends: the first change after a position
    int first = L;
    for (int i = i1 - 1; i >= i0; --i)
        if (i + 1 == L || x[i] != x[i + 1]) first = i + 1;
    edge[tid] = first;
    __syncthreads();
    for (int o = 1; o < kSpanThreads; o <<= 1) {
        const int other = tid + o < kSpanThreads ? edge[tid + o] : L;
        __syncthreads();
        edge[tid] = min(edge[tid], other);
        __syncthreads();
    }
    int end = tid + 1 < kSpanThreads ? edge[tid + 1] : L;
    for (int i = i1 - 1; i >= i0; --i) {
        if (i + 1 == L || x[i] != x[i + 1]) end = i + 1;
        out[i].y = x[i] < 0 ? 0 : end;
    }
}

}  // namespace

cudaError_t launch_document_spans(const int32_t* ids, int B, int L, int32_t* spans, cudaStream_t s) {
    return launch_pdl(document_spans_kernel, dim3(B), dim3(kSpanThreads), 0, s, ids, L, spans);
}

cudaError_t launch_span_attn(const SpanAttnParams& p, cudaStream_t s) {
    const dim3 grid((p.Lq + kWarps - 1) / kWarps, p.B * p.h), block(32 * kWarps);
    return p.d == 64 ? launch_pdl(span_attn_simple_kernel<64>, grid, block, 0, s, p)
                     : launch_pdl(span_attn_simple_kernel<128>, grid, block, 0, s, p);
}

}  // namespace mha
