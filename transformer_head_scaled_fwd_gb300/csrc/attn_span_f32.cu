// attn_span_f32.cu -- attention under span masks in fp32: fp32 products and sums on the CUDA cores (no TF32), the same
// masks and scores as the bf16 kernels.
//
//   m, l, O: running maximum (log2 units), sum and output of a row over the key tiles seen so far; a tile's weights
//   are exp2(s - m), O and l are rescaled when m grows.
//
// Bound by fp32 multiply-adds: 4 d_k flop a (query, key) pair. Unit of work: 64 query rows of one head, a CTA of 128
// threads, two (d_k = 128) or three CTAs an SM, which cover one another's waits (two of d_k = 64: 61 against 53 us on
// documents of 200). A thread forms 8 x 4 scores (rows 8 r .. 8 r + 7, keys c + 16 n) and 8 x d_k / 16 outputs of the same
// rows, so the 16 lanes that share rows exchange maxima by shuffles and the weights through 16 KB of shared memory that
// no other warp reads. The values of a tile arrive during its scores, the next keys during its products with the values.
// Multiply-adds are packed in pairs, along d_k for the scores and along the outputs for the product (2 x 4096 causal, 8
// heads of 128: 1364 us; single ones in the product 1448 us, in both 1562 us).
// Measured, 2 x 4096, 8 heads of 128: all keys 2792 us, 49 TFLOP/s (0.66 of 128 multiply-adds a clock and SM); causal
// 1364 us; of 64: 1628 and 782 us.
#include <algorithm>

#include "attn_span.cuh"

namespace mha {
namespace {

constexpr int BM = 64, BK = 64;          // queries of a unit, keys of a tile
constexpr int kThreads = 128;
constexpr int kRows = 8, kKeysT = 4;     // rows and keys of a thread
constexpr int kLanes = BK / kKeysT;      // lanes that share rows

template <int kD>
struct Geo {
    static constexpr int kTile = 64 * kD;                          // floats
    static constexpr int kCtas = kD == 128 ? 2 : 3;                // of an SM
    static constexpr int kBytes = (3 * kTile + BM * BK) * 4 + BM * 8;
};

// 64 rows of kD floats; a row's 16-byte chunk c lies at c ^ twist(row), so that 8 neighbouring rows, and rows 8 apart,
// have theirs in different banks.
__device__ __forceinline__ int twist(int row) { return (row & 7) ^ ((row >> 3) & 1); }

template <int kD, bool kTwist>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t stride, int row0, int rows) {
    constexpr int kChunks = kD / 4, kStep = kThreads / kChunks;
    const int c = threadIdx.x % kChunks;
#pragma unroll
    for (int i = 0; i < 64 / kStep; ++i) {
        const int r = i * kStep + threadIdx.x / kChunks;
        const bool live = row0 + r < rows;
        cp_async16(smem_u32(dst + r * kD + (kTwist ? c ^ twist(r) : c) * 4), src + (live ? (row0 + r) * stride : 0) + c * 4, live);
    }
}

template <int kD, bool kSplit>
__global__ void __launch_bounds__(kThreads, Geo<kD>::kCtas) span_attn_f32_kernel(const __grid_constant__ SpanAttnParams p) {
    constexpr int kTile = Geo<kD>::kTile, kV4 = kD / 64;      // float4 of the output a row and thread
    extern __shared__ __align__(16) float sm[];
    float *qs = sm, *ks = sm + kTile, *vs = sm + 2 * kTile, *ps = sm + 3 * kTile;
    int2* ivs = reinterpret_cast<int2*>(ps + BM * BK);
    const int pieces = kSplit ? p.pieces : 1, piece = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
    pdl_trigger();
    pdl_wait();   // the tensors and the mask parts come from earlier kernels

    // units with the last queries first: the longest under a causal mask
    const int planes = p.B * p.h, tiles = (p.Lq + BM - 1) / BM;
    const int unit = blockIdx.x / pieces, back = unit / planes, plane = unit - back * planes;
    const int q0 = (tiles - 1 - back) * BM, b = plane / p.h, head = plane - b * p.h, kvh = head / (p.h / p.h_kv);
    const int lane = threadIdx.x & 31;
    const int valid = p.valid_lens != nullptr ? min(max(p.valid_lens[b], 0), p.Lk) : p.Lk;
    const int seen = p.prefix_lens != nullptr ? p.prefix_lens[b] : 0;
    // every warp finds the unit's keys: some row sees [lo_min, hi_max), all rows [lo_max, hi_min)
    int lo_min = p.Lk, lo_max = 0, hi_min = p.Lk, hi_max = 0;
#pragma unroll
    for (int r = 0; r < BM; r += 32) {
        const int i = q0 + r + lane;
        int2 iv = make_int2(0, 0);
        if (i < p.Lq) {
            iv = interval_of(p, valid, seen, span_of(p, b, i), i);
            lo_max = max(lo_max, iv.x);
            hi_min = min(hi_min, iv.y);
            if (iv.y > iv.x) {
                lo_min = min(lo_min, iv.x);
                hi_max = max(hi_max, iv.y);
            }
        }
        if (threadIdx.x < 32) ivs[r + lane] = iv;
    }
    lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    hi_max = __reduce_max_sync(0xffffffffu, hi_max);
    int j0 = lo_min / BK, j1 = hi_max > lo_min ? (hi_max + BK - 1) / BK : j0;
    if constexpr (kSplit) {
        const int64_t n = j1 - j0;
        j1 = j0 + static_cast<int>(n * (piece + 1) / pieces);
        j0 += static_cast<int>(n * piece / pieces);
    }

    const float* q = static_cast<const float*>(p.q.p) + b * p.q.b + head * p.q.h;
    const float* k = static_cast<const float*>(p.k.p) + b * p.k.b + kvh * p.k.h;
    const float* v = static_cast<const float*>(p.v.p) + b * p.v.b + kvh * p.v.h;
    if (j0 < j1) {
        load_tile<kD, true>(qs, q, p.q.l, q0, p.Lq);
        load_tile<kD, true>(ks, k, p.k.l, j0 * BK, valid);   // keys and values behind the valid length: zeros
        cp_commit();
    }

    const int rg = threadIdx.x / kLanes, kg = threadIdx.x % kLanes;
    const float slope = p.slopes != nullptr ? p.slopes[head] * kLog2e : 0.0f;
    const float in = p.cap > 0.0f ? p.scale / p.cap : p.scale * kLog2e, top = p.cap * kLog2e;
    // chunk c of row 8 rg + i: c ^ i ^ (rg & 1)
    const float* const qr[2] = {qs + rg * kRows * kD + (rg & 1) * 4, qs + rg * kRows * kD + ((rg & 1) ^ 1) * 4};
    const float* const kr = ks + kg * kD;
    const int kt = twist(kg);
    // the weights of row 8 rg + i: key n at n ^ 16 (rg & 1)
    float* const pr = ps + rg * kRows * BK;
    const int pt = (rg & 1) * 16;
    float m[kRows], l[kRows];
    float4 o[kRows][kV4];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < kV4; ++e) o[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int j = j0; j < j1; ++j) {
        cp_wait<0>();
        __syncthreads();   // the tile's keys are here, and the last values have been read
        load_tile<kD, false>(vs, v, p.v.l, j * BK, valid);
        cp_commit();
        float2 s2[kRows][kKeysT];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int n = 0; n < kKeysT; ++n) s2[i][n] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c8 = 0; c8 < kD; c8 += 32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float4 a[kRows], w[kKeysT];
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    a[i] = *reinterpret_cast<const float4*>(qr[(e ^ i) & 1] + i * kD + c8 + ((e ^ i) & 6) * 4);
#pragma unroll
                for (int n = 0; n < kKeysT; ++n)
                    w[n] = *reinterpret_cast<const float4*>(kr + n * kLanes * kD + c8 + (e ^ kt) * 4);
#pragma unroll
                for (int i = 0; i < kRows; ++i)
#pragma unroll
                    for (int n = 0; n < kKeysT; ++n) {
                        s2[i][n] = ffma2(make_float2(a[i].x, a[i].y), make_float2(w[n].x, w[n].y), s2[i][n]);
                        s2[i][n] = ffma2(make_float2(a[i].z, a[i].w), make_float2(w[n].z, w[n].w), s2[i][n]);
                    }
            }
        }
        const int k0 = j * BK + kg;
        const bool edge = j * BK < lo_max || (j + 1) * BK > hi_min;
        bool grow = false;
        float alpha[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float x[kKeysT];
            float tile_top = -CUDART_INF_F;
            const int row = rg * kRows + i;
            int2 iv = make_int2(0, 0);
            if (edge) iv = ivs[row];
#pragma unroll
            for (int n = 0; n < kKeysT; ++n) {
                const int key = k0 + n * kLanes;
                const float dot = s2[i][n].x + s2[i][n].y;
                x[n] = p.cap > 0.0f ? top * tanhf(dot * in) : dot * in;
                if (slope != 0.0f) x[n] = fmaf(-slope, fabsf(static_cast<float>(q0 + row + p.q_offset - key)), x[n]);
                if (edge && (key < iv.x || key >= iv.y)) x[n] = -CUDART_INF_F;
                tile_top = fmaxf(tile_top, x[n]);
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) tile_top = fmaxf(tile_top, __shfl_xor_sync(0xffffffffu, tile_top, d));
            const float next = fmaxf(m[i], tile_top);
            grow |= next != m[i];
            alpha[i] = next == m[i] ? 1.0f : ex2_approx(m[i] - next);   // 0 for the first keys
            m[i] = next;
            // with no key of the row yet (m = -inf) every weight is exp2(-inf) = 0
            const float ref = next == -CUDART_INF_F ? 0.0f : next;
            l[i] *= alpha[i];
#pragma unroll
            for (int n = 0; n < kKeysT; ++n) {
                const float w = ex2_approx(x[n] - ref);
                l[i] += w;
                pr[i * BK + ((kg + n * kLanes) ^ pt)] = w;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int e = 0; e < kV4; ++e) {
                    o[i][e].x *= alpha[i];
                    o[i][e].y *= alpha[i];
                    o[i][e].z *= alpha[i];
                    o[i][e].w *= alpha[i];
                }
        }
        cp_wait<0>();
        __syncthreads();   // the tile's values are here, and its keys have been read
        if (j + 1 < j1) {
            load_tile<kD, true>(ks, k, p.k.l, (j + 1) * BK, valid);
            cp_commit();
        }
#pragma unroll 2
        for (int c = 0; c < BK; c += 4) {
            float4 w[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) w[i] = *reinterpret_cast<const float4*>(pr + i * BK + (c ^ pt));
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < kV4; ++e) {
                    const float4 x = *reinterpret_cast<const float4*>(vs + (c + n) * kD + e * 64 + kg * 4);
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        const float a = n == 0 ? w[i].x : n == 1 ? w[i].y : n == 2 ? w[i].z : w[i].w;
                        const float2 lo = ffma2(make_float2(a, a), make_float2(x.x, x.y), make_float2(o[i][e].x, o[i][e].y));
                        const float2 hi = ffma2(make_float2(a, a), make_float2(x.z, x.w), make_float2(o[i][e].z, o[i][e].w));
                        o[i][e] = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    if constexpr (kSplit) {
        // the part in place of the key and value tiles, its statistics in place of the weights
        float* const part = ks;
        static_assert(BM * part_pitch(kD) <= 2 * kTile, "a part fits the tiles");
        __syncthreads();   // the last values and weights have been read
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int row = rg * kRows + i;
            if (kg == 0) {
                ps[row] = m[i];
                ps[BM + row] = l[i];
            }
#pragma unroll
            for (int e = 0; e < kV4; ++e) *reinterpret_cast<float4*>(part + row * part_pitch(kD) + e * 64 + kg * 4) = o[i][e];
        }
        __syncwarp();
        cluster_sync_all();
        join_parts<float, kD, BM, kThreads>(p, b, head, q0, pieces, piece, smem_u32(ps), smem_u32(part));
        __syncwarp();
        cluster_sync_all();   // the others have read this CTA's part
        return;
    }
    float* out = static_cast<float*>(p.out.p) + b * p.out.b + head * p.out.h;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = q0 + rg * kRows + i;
        const float L = l[i];
        const bool none = L == 0.0f;              // no key: a row of zeros, o may hold 0 * NaN from the tile's other rows' keys
        const float inv = L > 0.0f ? 1.0f / L : L;   // NaN stays
        if (row >= p.Lq) continue;
#pragma unroll
        for (int e = 0; e < kV4; ++e)
            *reinterpret_cast<float4*>(out + row * p.out.l + e * 64 + kg * 4) =
                none ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(o[i][e].x * inv, o[i][e].y * inv, o[i][e].z * inv, o[i][e].w * inv);
    }
}

template <int kD>
cudaError_t launch_d(SpanAttnParams p, cudaStream_t s) {
    constexpr int kBytes = Geo<kD>::kBytes;
    static_assert(Geo<kD>::kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory budget");
    const int64_t units = static_cast<int64_t>(p.B) * p.h * ((p.Lq + BM - 1) / BM);
    // As in bf16: as many CTAs a unit as let all units run at once; a tile takes longer here, so fewer keys pay for it. Where
    // clusters of eight fit with a CTA an SM they ask for more shared memory than half an SM has, because side by side
    // they take twice as long (one query over 4096 keys, 8 heads of 64 (128), us by one CTA 344 (499), side by side 77
    // (111), an SM each 43 (70)); more units share SMs (200 queries over 2000 keys, 20 heads: 350 -> 94 (413 -> 219)).
    constexpr int kAlone = 120 * 1024;
    static_assert(kBytes <= kAlone, "room for the tiles");
    auto kernel = span_attn_f32_kernel<kD, true>;
    static ClusterRoom alone, shared;
    const int64_t reach = p.causal && p.prefix_lens == nullptr ? std::min<int64_t>(p.Lk, static_cast<int64_t>(p.q_offset) + p.Lq) : p.Lk;
    int bytes = kAlone;
    p.pieces = 1;
    if (reach >= 256 && units <= 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAlone);
        if (e != cudaSuccess) return e;
        if (units <= alone.at_once(kernel, kThreads, kAlone, 8)) {
            p.pieces = 8;
        } else {
            bytes = kBytes;
            for (int size = 8; size > 1 && p.pieces == 1; size /= 2)
                if (units <= shared.at_once(kernel, kThreads, kBytes, size)) p.pieces = size;
        }
    }
    if (p.pieces > 1)
        return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(units * p.pieces)), dim3(kThreads), p.pieces, bytes, s, p);
    cudaError_t e = cudaFuncSetAttribute(span_attn_f32_kernel<kD, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(span_attn_f32_kernel<kD, false>, dim3(static_cast<unsigned>(units)), dim3(kThreads), kBytes, s, p);
}

}  // namespace

cudaError_t launch_span_attn_f32(const SpanAttnParams& p, cudaStream_t s) {
    return p.d == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace mha
