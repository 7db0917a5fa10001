// serve_api.cu -- C ABI of the serving operators declared in include/mha.h: argument checks,
// parameter blocks and launches. Every check runs before anything is enqueued.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/mha.h"
#include "mha_internal.h"
#include "serve.h"

namespace {

mha_status_t fail(mha_status_t st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    mha::set_last_error(buf);
    return st;
}

mha_status_t launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return MHA_OK;
    return fail(MHA_ERR_CUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem(mha_dtype_t dt) { return dt == MHA_BF16 ? 2 : 4; }

mha_status_t check_dtype(mha_dtype_t dt) {
    if (dt != MHA_F32 && dt != MHA_BF16) return fail(MHA_ERR_INVALID_ARG, "dtype %d is not MHA_F32 or MHA_BF16", dt);
    return MHA_OK;
}

mha_status_t check_heads(int h, int h_kv) {
    if (h <= 0 || h_kv <= 0) return fail(MHA_ERR_INVALID_ARG, "heads must be positive (h=%d h_kv=%d)", h, h_kv);
    if (h % h_kv != 0) return fail(MHA_ERR_INVALID_ARG, "h %% h_kv != 0 (h=%d, h_kv=%d)", h, h_kv);
    return MHA_OK;
}

// Tensor [B, L, H, d] with its strides; `what` names it in messages.
mha_status_t view(const void* p, const mha_strides_t* st, size_t es, const char* what, mha::Strided* out) {
    if (p == nullptr || st == nullptr) return fail(MHA_ERR_INVALID_ARG, "%s and its strides must not be NULL", what);
    if (!aligned(p, es)) return fail(MHA_ERR_INVALID_ARG, "%s is not aligned to its element type", what);
    if (st->b < 0 || st->l < 0 || st->h < 0) return fail(MHA_ERR_INVALID_ARG, "%s has a negative stride", what);
    out->p = const_cast<void*>(p);
    out->b = st->b;
    out->l = st->l;
    out->h = st->h;
    return MHA_OK;
}

mha_status_t check_rotary(const mha_rotary_t* r, int d_k) {
    if (r->inv_freq == nullptr) return fail(MHA_ERR_INVALID_ARG, "inv_freq must not be NULL");
    if (r->rot_dim < 2 || r->rot_dim % 2 != 0 || r->rot_dim > d_k)
        return fail(MHA_ERR_INVALID_ARG, "rot_dim must be even and in 2 .. d_k (rot_dim=%d, d_k=%d)", r->rot_dim, d_k);
    if (r->interleaved != 0 && r->interleaved != 1)
        return fail(MHA_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", r->interleaved);
    if (!std::isfinite(r->scale)) return fail(MHA_ERR_INVALID_ARG, "the rotary scale must be finite");
    return MHA_OK;
}

void set_rotary(const mha_rotary_t* r, mha::RotaryParams* p) {
    if (r == nullptr) return;
    p->inv_freq = r->inv_freq;
    p->rot = r->rot_dim;
    p->interleaved = r->interleaved;
    p->scale = r->scale;
}

mha_status_t check_cache(const mha_paged_cache_t* c, mha_dtype_t dt, mha::PagedView* out) {
    if (c == nullptr || c->k_pages == nullptr || c->v_pages == nullptr || c->block_table == nullptr)
        return fail(MHA_ERR_INVALID_ARG, "the cache, its pages and its block table must not be NULL");
    if (c->n_pages <= 0 || c->page_size <= 0 || c->max_pages <= 0)
        return fail(MHA_ERR_INVALID_ARG, "cache sizes must be positive (n_pages=%d page_size=%d max_pages=%d)",
                    c->n_pages, c->page_size, c->max_pages);
    if (c->table_stride < 0 || c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0)
        return fail(MHA_ERR_INVALID_ARG, "the cache has a negative stride");
    if (!aligned(c->k_pages, elem(dt)) || !aligned(c->v_pages, elem(dt)))
        return fail(MHA_ERR_INVALID_ARG, "the pages are not aligned to their element type");
    out->k = c->k_pages;
    out->v = c->v_pages;
    out->page_stride = c->page_stride;
    out->slot_stride = c->slot_stride;
    out->head_stride = c->head_stride;
    out->table = c->block_table;
    out->table_stride = c->table_stride;
    out->n_pages = c->n_pages;
    out->max_pages = c->max_pages;
    out->page = mha::fast_div(static_cast<uint32_t>(c->page_size));
    return MHA_OK;
}

// scores NULL: the plain scaled scores
mha_status_t check_scores(const mha_scores_t* s, int d_k, float* scale, float* cap, const float** slopes) {
    *scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d_k)));
    *cap = 0.0f;
    *slopes = nullptr;
    if (s == nullptr) return MHA_OK;
    if (!std::isfinite(s->scale) || !std::isfinite(s->cap) || s->cap < 0.0f)
        return fail(MHA_ERR_INVALID_ARG, "scale must be finite and cap finite and >= 0 (got %g, %g)", s->scale, s->cap);
    if (s->scale != 0.0f) *scale = s->scale;
    if (s->cap > 0.0f) {
        // The kernels form scale / cap and cap log2(e), so the cap is kept where both are normal numbers. Under a smaller one
        // scores are within 2^-100 of 0; a larger one changes scores below 2^85 (products below 2^95) by less than 2^-30 of
        // themselves.
        const float most = std::fmin(0x1p100f, std::fabs(*scale) < 0x1p-10f ? std::fabs(*scale) * 0x1p110f : 0x1p100f);
        *cap = std::fmax(std::fmin(s->cap, most), 0x1p-100f);
        if (!std::isfinite(*scale / *cap))
            return fail(MHA_ERR_INVALID_ARG, "scale / cap must be finite (got %g / %g)", *scale, s->cap);
    }
    *slopes = s->slopes;
    return MHA_OK;
}

// heads of all tokens that one launch turns or copies (32-bit CTA numbers)
constexpr int64_t kMostRows = int64_t(1) << 30;

mha_status_t check_bt(int B, int T, int d_k) {
    if (B <= 0 || T <= 0 || d_k <= 0)
        return fail(MHA_ERR_INVALID_ARG, "sizes must be positive (B=%d T=%d d_k=%d)", B, T, d_k);
    if (d_k > 512) return fail(MHA_ERR_UNSUPPORTED, "d_k <= 512 is implemented (d_k = %d)", d_k);
    if (static_cast<int64_t>(B) * T > 0x7fffffffll) return fail(MHA_ERR_UNSUPPORTED, "B * T must stay below 2^31");
    return MHA_OK;
}

}  // namespace

extern "C" {

mha_status_t mha_rotary_frequencies(float* inv_freq, float* scale, int rot_dim, double base,
                                    mha_rope_scaling_t scaling, double factor, double original_length, double low,
                                    double high) {
    if (inv_freq == nullptr || scale == nullptr) return fail(MHA_ERR_INVALID_ARG, "inv_freq and scale must not be NULL");
    if (rot_dim < 2 || rot_dim % 2 != 0) return fail(MHA_ERR_INVALID_ARG, "rot_dim must be even and >= 2 (got %d)", rot_dim);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(MHA_ERR_INVALID_ARG, "base must be finite and above 1");
    if (scaling < MHA_ROPE_PLAIN || scaling > MHA_ROPE_RAMP) return fail(MHA_ERR_INVALID_ARG, "unknown scaling %d", scaling);
    if (scaling != MHA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(MHA_ERR_INVALID_ARG, "factor must be finite and >= 1 (got %g)", factor);
    if (scaling == MHA_ROPE_BASE && rot_dim == 2)
        return fail(MHA_ERR_INVALID_ARG, "stretching the base needs rot_dim > 2");
    const bool banded = scaling == MHA_ROPE_BANDED || scaling == MHA_ROPE_RAMP;
    if (banded && (!(original_length > 0.0) || !std::isfinite(original_length) || !(low > 0.0) || !(high > low) ||
                   !std::isfinite(high)))
        return fail(MHA_ERR_INVALID_ARG, "original_length must be positive and 0 < low < high");
    const double two_pi = 6.283185307179586476925;
    const int half = rot_dim / 2;
    if (scaling == MHA_ROPE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    // MHA_ROPE_RAMP: index of the pair that turns n times over original_length. The table ends at half - 1, the ramp may end
    // beyond it.
    auto pair_of = [&](double n) {
        return rot_dim * std::log(original_length / (n * two_pi)) / (2.0 * std::log(base));
    };
    const double first = banded ? std::fmax(std::floor(pair_of(high)), 0.0) : 0.0;
    const double last = banded ? std::fmin(std::ceil(pair_of(low)), rot_dim - 1.0) : 0.0;
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == MHA_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == MHA_ROPE_BANDED) {
            const double turns = original_length * f / two_pi;   // original_length / wavelength
            const double keep = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
            f = keep * f + (1.0 - keep) * f / factor;
        } else if (scaling == MHA_ROPE_RAMP) {
            const double width = std::fmax(last - first, 1e-3);
            const double keep = 1.0 - std::fmin(std::fmax((i - first) / width, 0.0), 1.0);
            f = keep * f + (1.0 - keep) * f / factor;
        }
        inv_freq[i] = static_cast<float>(f);
    }
    *scale = scaling == MHA_ROPE_RAMP ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return MHA_OK;
}

mha_status_t mha_rotary(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides, void* q_out,
                        const mha_strides_t* q_out_strides, const void* k, const mha_strides_t* k_strides, void* k_out,
                        const mha_strides_t* k_out_strides, int B, int T, int h, int h_kv, int d_k,
                        const int32_t* positions, const mha_rotary_t* rotary, void* stream) {
    mha_status_t st;
    if ((st = check_dtype(dt)) != MHA_OK || (st = check_bt(B, T, d_k)) != MHA_OK) return st;
    if (h <= 0 || (k != nullptr && h_kv <= 0))
        return fail(MHA_ERR_INVALID_ARG, "heads must be positive (h=%d h_kv=%d)", h, h_kv);
    if (static_cast<int64_t>(B) * T * (static_cast<int64_t>(h) + (k != nullptr ? h_kv : 0)) > kMostRows)
        return fail(MHA_ERR_UNSUPPORTED, "B * T * (h + h_kv) must stay below 2^30");
    if (rotary == nullptr) return fail(MHA_ERR_INVALID_ARG, "rotary must not be NULL");
    if ((st = check_rotary(rotary, d_k)) != MHA_OK) return st;
    mha::RotaryParams p{};
    const size_t es = elem(dt);
    if ((st = view(q, q_strides, es, "q", &p.q)) != MHA_OK) return st;
    if ((st = view(q_out, q_out_strides, es, "q_out", &p.q_out)) != MHA_OK) return st;
    if (k != nullptr) {
        if ((st = view(k, k_strides, es, "k", &p.k)) != MHA_OK) return st;
        if ((st = view(k_out, k_out_strides, es, "k_out", &p.k_out)) != MHA_OK) return st;
    }
    set_rotary(rotary, &p);
    p.positions = positions;
    p.B = B; p.T = T; p.h = h; p.h_kv = k != nullptr ? h_kv : 0; p.d = d_k;
    return launched(mha::launch_rotary(p, dt == MHA_BF16, as_stream(stream)), "rotary");
}

mha_status_t mha_paged_append(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides, void* q_out,
                              const mha_strides_t* q_out_strides, const void* k, const mha_strides_t* k_strides,
                              void* k_out, const mha_strides_t* k_out_strides, const void* v,
                              const mha_strides_t* v_strides, int B, int T, int h, int h_kv, int d_k,
                              const int32_t* start, const int32_t* new_lens, const mha_rotary_t* rotary,
                              const mha_paged_cache_t* cache, void* stream) {
    mha_status_t st;
    if ((st = check_dtype(dt)) != MHA_OK || (st = check_bt(B, T, d_k)) != MHA_OK) return st;
    if (h_kv <= 0 || (q != nullptr && h <= 0))
        return fail(MHA_ERR_INVALID_ARG, "heads must be positive (h=%d h_kv=%d)", h, h_kv);
    if (static_cast<int64_t>(B) * T * ((q != nullptr ? static_cast<int64_t>(h) : 0) + 2 * static_cast<int64_t>(h_kv)) > kMostRows)
        return fail(MHA_ERR_UNSUPPORTED, "B * T * (h + 2 h_kv) must stay below 2^30");
    if (start == nullptr) return fail(MHA_ERR_INVALID_ARG, "start must not be NULL");
    if (rotary != nullptr && (st = check_rotary(rotary, d_k)) != MHA_OK) return st;
    mha::RotaryParams p{};
    const size_t es = elem(dt);
    if ((st = check_cache(cache, dt, &p.cache)) != MHA_OK) return st;
    if ((st = view(k, k_strides, es, "k", &p.k)) != MHA_OK) return st;
    if ((st = view(v, v_strides, es, "v", &p.v)) != MHA_OK) return st;
    if (k_out != nullptr && (st = view(k_out, k_out_strides, es, "k_out", &p.k_out)) != MHA_OK) return st;
    if (q != nullptr) {
        if ((st = view(q, q_strides, es, "q", &p.q)) != MHA_OK) return st;
        if ((st = view(q_out, q_out_strides, es, "q_out", &p.q_out)) != MHA_OK) return st;
    }
    set_rotary(rotary, &p);
    p.start = start;
    p.new_lens = new_lens;
    p.B = B; p.T = T; p.h = q != nullptr ? h : 0; p.h_kv = h_kv; p.d = d_k;
    p.status = mha::device_status();
    if (p.status == nullptr) return fail(MHA_ERR_CUDA, "device status word unavailable");
    return launched(mha::launch_rotary(p, dt == MHA_BF16, as_stream(stream)), "paged append");
}

size_t mha_paged_attention_workspace_size(mha_dtype_t dt, int B, int h, int h_kv, int d_k) {
    if ((dt != MHA_F32 && dt != MHA_BF16) || B <= 0 || h <= 0 || h_kv <= 0 || h % h_kv != 0 || (d_k != 64 && d_k != 128))
        return 0;
    return mha::paged_attn_workspace(dt == MHA_BF16, B, h, h_kv, d_k);
}

mha_status_t mha_paged_attention(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides, void* out,
                                 const mha_strides_t* out_strides, int B, int h, int h_kv, int d_k,
                                 const int32_t* kv_lens, const mha_scores_t* scores, const mha_paged_cache_t* cache,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    mha_status_t st;
    if ((st = check_dtype(dt)) != MHA_OK) return st;
    if (B <= 0) return fail(MHA_ERR_INVALID_ARG, "B must be positive (got %d)", B);
    if ((st = check_heads(h, h_kv)) != MHA_OK) return st;
    if (d_k != 64 && d_k != 128)
        return fail(MHA_ERR_UNSUPPORTED, "paged attention is implemented for d_k = 64 and 128 (d_k = %d)", d_k);
    if (B > 65535 || h > 65535) return fail(MHA_ERR_UNSUPPORTED, "B and h up to 65535 (got %d, %d)", B, h);
    if (kv_lens == nullptr) return fail(MHA_ERR_INVALID_ARG, "kv_lens must not be NULL");
    mha::PagedAttnParams p{};
    if ((st = check_cache(cache, dt, &p.cache)) != MHA_OK) return st;
    if ((st = check_scores(scores, d_k, &p.scale, &p.cap, &p.slopes)) != MHA_OK) return st;
    mha::Strided qv, ov;
    if ((st = view(q, q_strides, elem(dt), "q", &qv)) != MHA_OK) return st;
    if ((st = view(out, out_strides, elem(dt), "out", &ov)) != MHA_OK) return st;
    const int64_t chunk = 16 / static_cast<int64_t>(elem(dt));
    if (!aligned(cache->k_pages, 16) || !aligned(cache->v_pages, 16) || cache->page_stride % chunk != 0 ||
        cache->slot_stride % chunk != 0 || cache->head_stride % chunk != 0)
        return fail(MHA_ERR_INVALID_ARG, "the pages and their strides must be aligned to 16 bytes");
    const size_t need = mha_paged_attention_workspace_size(dt, B, h, h_kv, d_k);
    if (workspace == nullptr || !aligned(workspace, 256))
        return fail(MHA_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
    if (workspace_bytes < need) return fail(MHA_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes, need);
    p.q = qv.p; p.q_b = qv.b; p.q_h = qv.h;
    p.out = ov.p; p.o_b = ov.b; p.o_h = ov.h;
    p.kv_lens = kv_lens;
    p.B = B; p.h = h; p.h_kv = h_kv; p.d = d_k;
    p.partial = static_cast<float*>(workspace);
    p.status = mha::device_status();
    if (p.status == nullptr) return fail(MHA_ERR_CUDA, "device status word unavailable");
    return launched(mha::launch_paged_attn(p, dt == MHA_BF16, as_stream(stream)), "paged attention");
}

mha_status_t mha_document_spans(const int32_t* doc_ids, int B, int L, int32_t* spans, void* stream) {
    if (doc_ids == nullptr || spans == nullptr) return fail(MHA_ERR_INVALID_ARG, "doc_ids and spans must not be NULL");
    if (B <= 0 || L <= 0) return fail(MHA_ERR_INVALID_ARG, "sizes must be positive (B=%d L=%d)", B, L);
    if (B > 65535 || L > 0x7ffffbff) return fail(MHA_ERR_UNSUPPORTED, "B up to 65535, L below 2^31 - 1024 (got %d, %d)", B, L);
    if (!aligned(doc_ids, 4) || !aligned(spans, 8))
        return fail(MHA_ERR_INVALID_ARG, "doc_ids must be aligned to 4 bytes and spans to 8");
    return launched(mha::launch_document_spans(doc_ids, B, L, spans, as_stream(stream)), "document spans");
}

mha_status_t mha_attention(mha_dtype_t dt, const void* q, const mha_strides_t* q_strides, const void* k,
                           const mha_strides_t* k_strides, const void* v, const mha_strides_t* v_strides, void* out,
                           const mha_strides_t* out_strides, int B, int L_q, int L_k, int h, int h_kv, int d_k,
                           const mha_scores_t* scores, const mha_span_mask_t* mask, void* stream) {
    mha_status_t st;
    if ((st = check_dtype(dt)) != MHA_OK) return st;
    if (B <= 0 || L_q <= 0 || L_k <= 0)
        return fail(MHA_ERR_INVALID_ARG, "sizes must be positive (B=%d L_q=%d L_k=%d)", B, L_q, L_k);
    if (L_q > 0x7fffff00 || L_k > 0x7fffff00)
        return fail(MHA_ERR_UNSUPPORTED, "L_q and L_k must stay below 2^31 - 255 (got %d, %d)", L_q, L_k);
    if ((st = check_heads(h, h_kv)) != MHA_OK) return st;
    if (d_k != 64 && d_k != 128)
        return fail(MHA_ERR_UNSUPPORTED, "attention under span masks is implemented for d_k = 64 and 128 (d_k = %d)", d_k);
    mha::SpanAttnParams p{};
    if ((st = check_scores(scores, d_k, &p.scale, &p.cap, &p.slopes)) != MHA_OK) return st;
    const void* ptrs[4] = {q, k, v, out};
    const mha_strides_t* strides[4] = {q_strides, k_strides, v_strides, out_strides};
    mha::Strided* views[4] = {&p.q, &p.k, &p.v, &p.out};
    const char* names[4] = {"q", "k", "v", "out"};
    const int64_t chunk = 16 / static_cast<int64_t>(elem(dt));
    for (int i = 0; i < 4; ++i) {
        const int L = i == 0 || i == 3 ? L_q : L_k, H = i == 0 || i == 3 ? h : h_kv;
        if ((st = view(ptrs[i], strides[i], elem(dt), names[i], views[i])) != MHA_OK) return st;
        // a dimension of one element has no stride to speak of
        if (B == 1) views[i]->b = chunk;
        if (L == 1) views[i]->l = chunk;
        if (H == 1) views[i]->h = chunk;
        if (!aligned(ptrs[i], 16) || views[i]->b % chunk != 0 || views[i]->l % chunk != 0 || views[i]->h % chunk != 0)
            return fail(MHA_ERR_INVALID_ARG, "%s and its strides must be aligned to 16 bytes", names[i]);
        if (views[i]->l == 0 || (i == 3 && (views[i]->b == 0 || views[i]->h == 0)))
            return fail(MHA_ERR_INVALID_ARG, "%s: only the batch and head strides of an input may be 0", names[i]);
        if (views[i]->b >= (int64_t(1) << 39) || views[i]->l >= (int64_t(1) << 39) || views[i]->h >= (int64_t(1) << 39))
            return fail(MHA_ERR_UNSUPPORTED, "%s: strides must stay below 2^40 bytes", names[i]);
    }
    if (mask != nullptr) {
        if (mask->q_offset < 0 || mask->q_offset > 0x7fffffff - L_q)
            return fail(MHA_ERR_INVALID_ARG, "q_offset must be >= 0 and q_offset + L_q below 2^31 (got %d)", mask->q_offset);
        if (!aligned(mask->doc_spans, 8)) return fail(MHA_ERR_INVALID_ARG, "doc_spans must be aligned to 8 bytes");
        mha::set_mask(*mask, &p);
    }
    if (static_cast<int64_t>(B) * h > (int64_t(1) << 30) ||
        static_cast<int64_t>(B) * h * ((L_q + 63) / 64) > 0x7fffffffll)
        return fail(MHA_ERR_UNSUPPORTED, "B * h * ceil(L_q / 64) must stay below 2^31");
    p.B = B; p.Lq = L_q; p.Lk = L_k; p.h = h; p.h_kv = h_kv; p.d = d_k;
    p.status = mha::device_status();
    if (p.status == nullptr) return fail(MHA_ERR_CUDA, "device status word unavailable");
    return launched(dt == MHA_BF16 ? mha::launch_span_attn(p, as_stream(stream)) : mha::launch_span_attn_f32(p, as_stream(stream)),
                    "attention");
}

mha_status_t mha_rmsnorm(mha_dtype_t dt, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                         void* sum, int64_t sum_stride, const void* gain, float eps, int64_t rows, int d, void* y,
                         int64_t y_stride, float* scales, int group, void* stream) {
    mha_status_t st;
    if ((st = check_dtype(dt)) != MHA_OK) return st;
    if (rows < 0 || d <= 0) return fail(MHA_ERR_INVALID_ARG, "rows must be >= 0 and d positive (rows=%lld d=%d)",
                                        static_cast<long long>(rows), d);
    if (rows > 0x7fffffffll || d > (1 << 30))
        return fail(MHA_ERR_UNSUPPORTED, "rows must stay below 2^31 and d up to 2^30 (got d=%d)", d);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MHA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (scales != nullptr && group != 0 && group != 32 && group != 64 && group != 128)
        return fail(MHA_ERR_INVALID_ARG, "group must be 0, 32, 64 or 128 (got %d)", group);
    if (scales != nullptr && group != 0 && d % group != 0)
        return fail(MHA_ERR_INVALID_ARG, "group must divide d (group=%d, d=%d)", group, d);
    if (rows == 0) return MHA_OK;
    if (x == nullptr || y == nullptr) return fail(MHA_ERR_INVALID_ARG, "x and y must not be NULL");
    if (residual == nullptr) {
        residual_stride = sum_stride = 0;
        sum = nullptr;
    }
    const size_t es = elem(dt);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(sum, es) || !aligned(gain, es) ||
        !aligned(y, scales ? 1 : es) || !aligned(scales, 4))
        return fail(MHA_ERR_INVALID_ARG, "a tensor is not aligned to its element type");
    if (x_stride < 0 || residual_stride < 0 || sum_stride < 0 || y_stride < 0)
        return fail(MHA_ERR_INVALID_ARG, "row strides must be >= 0");
    if (rows > 1 && (y_stride < d || (sum != nullptr && sum_stride < d)))
        return fail(MHA_ERR_INVALID_ARG, "rows of y and sum must not overlap (strides below d=%d)", d);
    mha::RmsNormParams p{};
    p.x = x; p.residual = residual; p.sum = sum; p.gain = gain; p.y = y;
    p.scales = scales;
    p.x_stride = x_stride; p.r_stride = residual_stride; p.s_stride = sum_stride; p.y_stride = y_stride;
    p.rows = rows; p.d = d; p.group = group == 0 ? d : group; p.eps = eps;
    p.group_log2 = group == 128 ? 7 : group == 64 ? 6 : 5;
    return launched(mha::launch_rmsnorm(p, dt == MHA_BF16, as_stream(stream)), "RMS norm");
}

}  // extern "C"
