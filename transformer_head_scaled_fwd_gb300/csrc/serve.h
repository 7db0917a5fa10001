// serve.h -- parameter blocks and launchers of the serving operators (rotary positions and
// the paged append, paged attention, attention under span masks, RMS norm); not part of the
// public C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/mha.h"

namespace mha {

// From mha_api.cu: the device status word of the current device (nullptr on failure), and a
// bf16 tiled tensor map with zero fill (false: the driver refused it).
int* device_status();
bool encode_bf16_tiled(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                       const uint32_t* box, bool swizzle);

// n / d for 0 <= n < 2^31 by a multiplication: with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (umulhi(n, m) + n) >> s (round-up method of Granlund and Montgomery; the sum stays below
// 2^32 for n < 2^31).
struct FastDiv {
    uint32_t d, m, s;
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int n) const {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
    }
#endif
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.s = 0;
    while ((uint64_t(1) << f.s) < d) ++f.s;
    f.m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.s) - d)) / d + 1);
    return f;
}

struct PagedView {
    void* k;
    void* v;
    int64_t page_stride, slot_stride, head_stride;   // elements
    const int32_t* table;
    int64_t table_stride;
    int n_pages, max_pages;
    FastDiv page;            // page size
};

struct Strided {
    void* p;
    int64_t b, l, h;         // elements
};

// ------------------------------------------------------------ rotary positions, paged append
struct RotaryParams {
    Strided q, q_out, k, k_out, v;    // q.p, k.p, k_out.p may be nullptr
    PagedView cache;                  // cache.k nullptr: no append
    const int32_t* positions;         // [B, T] or nullptr: start[b] + t (start nullptr: t)
    const int32_t* start;             // [B] or nullptr
    const int32_t* new_lens;          // [B] or nullptr
    const float* inv_freq;            // [rot / 2]
    int rot, interleaved;             // rot 0: nothing is turned
    float scale;
    int B, T, h, h_kv, d;
    int* status;
    FastDiv by_t;            // set by the launcher
};
cudaError_t launch_rotary(const RotaryParams& p, bool bf16, cudaStream_t s);

// ------------------------------------------------------------ attention over the paged cache
struct PagedAttnParams {
    const void* q;
    int64_t q_b, q_h;
    void* out;
    int64_t o_b, o_h;
    PagedView cache;
    const int32_t* kv_lens;
    const float* slopes;     // [h] or nullptr
    float scale, cap;
    int B, h, h_kv, d;
    float* partial;          // workspace
    int* status;
    const float* k_scales;   // a cache in 8 bits: [n_pages, page_scales]; page_scales = blocks of a page * h_kv
    const float* v_scales;
    FastDiv scale_block;     // tokens a scale covers
    int64_t page_scales;
    FastDiv side;            // set by the launcher: neighbouring units that as many CTAs take side by side
    int whole;               // ... no unit is split
    int direct;              // ... and each has a CTA of its own
};
size_t paged_attn_workspace(bool bf16, int B, int h, int h_kv, int d);
cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, cudaStream_t s);

// ------------------------------------------------------------ a cache in 8 bits
size_t coded_attn_workspace(int d);
cudaError_t launch_coded_attn(const PagedAttnParams& p, bool bf16, bool int8, cudaStream_t s);
cudaError_t launch_coded_attn_f32(const PagedAttnParams& p, bool int8, cudaStream_t s);

struct CodedAppendParams {
    Strided q, q_out, k, k_out, v;    // q.p, k_out.p may be nullptr
    PagedView cache;                  // strides in bytes
    float* k_scales;                  // [n_pages, page_scales]
    float* v_scales;
    int64_t page_scales;              // blocks of a page * h_kv
    FastDiv block;                    // tokens a scale covers
    const int32_t* start;             // [B]
    const int32_t* new_lens;          // [B] or nullptr
    const float* inv_freq;            // [rot / 2]
    int rot, interleaved;             // rot 0: nothing is turned
    float scale;
    int B, T, h, h_kv, d, int8;
    int* status;
};
cudaError_t launch_coded_append(const CodedAppendParams& p, bool bf16, cudaStream_t s);
cudaError_t launch_coded_append_f32(const CodedAppendParams& p, cudaStream_t s);

// ------------------------------------------------------------ pages granted and returned
struct ResizeParams {
    const int32_t* held;     // [B]
    const int32_t* want;     // [B]
    int32_t* table;
    int64_t table_stride;
    int max_pages;
    int32_t* free_pages;     // [n_pages], the first *free_count are free
    int32_t* free_count;
    int n_pages;
    int32_t* lens;           // [B]
    int32_t* new_lens;       // [B] or nullptr
    int64_t* slots;          // [B, T] or nullptr
    int B, T;
    FastDiv page, by_t;
    int* status;
    bool slots_after;        // set by the launcher: by a kernel of their own
};
cudaError_t launch_resize(const ResizeParams& p, cudaStream_t s);

// ------------------------------------------------------------ attention under span masks
struct SpanAttnParams {
    Strided q, k, v, out;
    const int32_t* valid_lens;
    const int32_t* prefix_lens;
    const int32_t* spans;    // [B, Lq, 2] or nullptr
    const float* slopes;
    float scale, cap;
    int causal, q_offset;
    int B, Lq, Lk, h, h_kv, d;
    int* status;
    int pieces;              // set by the launcher: CTAs that share a unit
};
inline void set_mask(const mha_span_mask_t& m, SpanAttnParams* p) {
    p->causal = m.causal != 0;
    p->q_offset = m.q_offset;
    p->valid_lens = m.key_valid_lens;
    p->prefix_lens = m.causal != 0 ? m.prefix_lens : nullptr;   // not read otherwise
    p->spans = m.doc_spans;
}
cudaError_t launch_span_attn(const SpanAttnParams& p, cudaStream_t s);        // bf16
cudaError_t launch_span_attn_f32(const SpanAttnParams& p, cudaStream_t s);
cudaError_t launch_document_spans(const int32_t* ids, int B, int L, int32_t* spans, cudaStream_t s);

// ------------------------------------------------------------ RMS norm
struct RmsNormParams {
    const void* x;
    const void* residual;    // or nullptr
    void* sum;               // or nullptr
    const void* gain;        // or nullptr
    void* y;
    float* scales;           // or nullptr: y in the input's type
    int64_t x_stride, r_stride, s_stride, y_stride;
    int64_t rows;
    int d, group;            // group: elements a scale covers (d: the row; else 2^group_log2)
    int group_log2;
    float eps;
};
cudaError_t launch_rmsnorm(const RmsNormParams& p, bool bf16, cudaStream_t s);

}  // namespace mha
