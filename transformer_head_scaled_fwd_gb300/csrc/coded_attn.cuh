// coded_attn.cuh -- attention of one new token a sequence over a paged cache in 8 bits (e4m3 or int8 codes, a scale for each
// block of tokens and key head).
//
//   s_j = cap tanh(scale ks_j q.ck_j / cap) - slope (n - 1 - j),  o = sum_j softmax_j(s) vs_j cv_j,  j < n
// with codes c and the scales ks, vs of their blocks; one pass with a running maximum m and sum l. n = 0 gives zeros.
//
// HBM-bound: 2 d_k bytes a position and key head, half of a bf16 cache, so the same loads feed twice the keys and the
// instructions a key count twice as much. Codes become fp16 in registers, which is exact (e4m3 is a subset of fp16, int8 is
// below 2^8), and the products are fp16 matrix instructions on them. A query row is scaled by a power of two to below 2^15 and
// enters as one fp16 number an element (bf16: exact down to 2^-29 of the row's largest) or as two (fp32: to 2^-22).
//
// Scales: ks multiplies a score after its product. vs belongs to a weight, p_j vs_j, whose size is not bounded by that of p_j, and fp16 has no
// range to spare: the weights have a running maximum of their own, over s_j + log2 of vs_j's power of two, so that the largest that a warp has
// met lies in 2^10 .. 2^15 for scales from 2^-106 on. (p_j is fp32 relative to the largest: below 2^-126 of that it is 0, here and in the
// joins, and its value counts for nothing whatever its scale.) They are rounded to fp16: to 2^-11 of themselves (against 2^-8 of a bf16
// result), or, where fp16 ends, to 2^-25, that is 2^-35 of the largest. A second term would take that to what an fp32 result has, for 1 to 7 %
// of the time (16 x 8192 50.8 -> 52.3 us, 48 ragged capped 135.7 -> 145.6), and bring the error of a bf16 result against 64 bits to that of
// rounding it, which it is within 0.6 % of (12 x 9000 int8, capped, 1.650e-3 of the norm for 1.641e-3; 16 x 8192 1.627e-3 for 1.623e-3): for
// that it is not taken. For an fp32 result there are two: the second is the first one's rest times 2^12, whose products have sums of their
// own, so a weight is good to 2^-22 of itself or to 2^-37, 2^-47 of the largest. (With the rest on the first one's scale, and the largest from
// 2^6 on, a key of 99 % of the weight and no value left the other 32768 keys seven bits each: 2e-4 of the result's norm.) p_j itself is summed
// in fp32.
//
// Work split, loads and join: paged_line.cuh; a step is 32 keys.
//
// Measured: 16 sequences of 8192, 16 heads of 64, e4m3, 268 MB: 52 us, 5.2 TB/s (0.77 of measured copy bandwidth; a bf16 cache takes 89); 24 of 15000,
// 32 / 8 heads of 128, 737 MB: 120 us (0.92); 48 ragged ones up to 15000, int8, capped, 790 MB: 142 us (0.83); one of 131071, 16 / 2 heads: 22 us,
// of which 10 are its traffic; fp32 queries 16 x 8192 55 us (int8 59), 9 ragged up to 5000, 24 / 8 heads of 128 20 us. A step costs a warp 2700 cycles, 1000 of them to issue its copies and 1400 to compute; at eight warps
// an SM that is what HBM delivers, so long streams run at its rate and the rest is what any call has: the look-ups 1.7 + 3 us, the queries 1, a
// unit's end 1.7, the second launch and the join 3.7.
#pragma once

#include "paged_line.cuh"

namespace mha {
namespace {

constexpr float kBase = 10.0f;      // log2 of the least the largest weight is taken to

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(x));
    return f;
}

// Four codes to fp16: bytes 0, 1 and 2, 3 (kCross: 0, 2 and 1, 3).
template <bool kInt8, bool kCross>
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t& a, uint32_t& b) {
    if constexpr (kInt8) {
        // the byte c + 128 under the exponent of 1024 is 1024 + 128 + c
        const uint32_t u = x ^ 0x80808080u;
        a = __byte_perm(u, 0x64646464u, kCross ? 0x4240 : 0x4140);
        b = __byte_perm(u, 0x64646464u, kCross ? 0x4341 : 0x4342);
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(b) : "r"(0x64806480u));
    } else {
        const uint32_t u = kCross ? __byte_perm(x, 0u, 0x3120) : x;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(u));
    }
}

// Exponent of a scale, at least kLeastExponent: what then takes a weight of 2^kGrow to the weights' maximum stays in fp32.
constexpr int kLeastExponent = -106;
static_assert(kGrow - kLeastExponent + kBase < 127.0f, "2^127 is fp32's largest power of two");
__device__ __forceinline__ float exponent_of(float s) {
    return static_cast<float>(max(static_cast<int>((__float_as_uint(s) >> 23) & 0xffu) - 127, kLeastExponent));
}
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

// As in paged_attn.cu, both products are taken transposed: S^T = K q^T (16 keys x d_k times d_k x 8 heads) and
// o^T = V^T P^T (16 features x 16 keys times 16 keys x 8 heads). An operand's 16-bit elements are made from bytes that lie
// side by side, so the feature that a row or column of a product stands for is not its number: for K, the k of lane t of
// four are features 4 t .. 4 t + 3 (q is loaded to match); for V, loaded transposed in units of two bytes, rows g and
// g + 8 are features 2 g and 2 g + 1.
//
// A row of 128 bytes is a key of d_k = 128, or (kHeads = 2) the same position of two neighbouring key heads of 64, whose query heads
// are the unit's two tiles or, up to four each, the two halves of one (kNT = 0: every column meets both heads'
// codes, in sums of their own, and what is not of its head is left): lines of memory are 128 bytes, and with a head of 64 bytes a unit each line came from HBM twice
// (16 x 8192, 16 heads of 64: 537 MB read for 268).
// kNT tiles of 8 query heads a key head, 0: one for both
// CTAs an SM: one of eight warps, two of four, seven (six) of one
enum Shape { kOne, kTwo, kMany };
constexpr int kShort = 512;       // positions that one warp takes, at most
template <typename T_, int kD, int kHeads, int kNT, bool kInt8, int kShape = kOne>
struct WarpCoded {
    using T = T_;
    static constexpr int kRow = kD * kHeads;
    static constexpr bool kShared = kNT == 0;       // columns 0 - 3 are of the first key head, 4 - 7 of the second
    static constexpr int kTiles = kShared ? 1 : kNT * kHeads;
    static constexpr int kOfChunk = kShared ? 1 : kNT;          // tiles that a chunk of features takes part in
    static constexpr int kOfKey = kShared ? 1 : kHeads;         // key heads that a lane has scores of
    static_assert(kHeads == 1 ? kNT >= 1 : kNT <= 1, "at most a tile for each of two key heads");
    static constexpr int kRows = 8 * kTiles;
    static_assert(kShape != kTwo || (kTiles == 1 && kRow == 128), "what shared memory takes twice");
    using Step = StepOf<kRow, 1, 32, kRow == 128 ? 3 : 6, kHeads, kShape == kOne ? 8 : kShape == kTwo ? 4 : 1, 2,
                        kShape == kOne ? 1 : kShape == kTwo ? 2 : (kTiles * kD > 128) ? 6 : 7, kShape == kOne ? 4 : kShape == kTwo ? 8 : kShort / 32>;
    static constexpr int kBufs = kShape == kMany ? 1 : kShape == kTwo || kTiles * kD > 128 ? 2 : 4;      // of the join, in what shared memory the stages leave
    static constexpr int kQFloats = 0;
    static constexpr bool kSplits = kShape != kMany;     // units among CTAs
    static constexpr int kKT = Step::kKeys / 16;
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int kQT = kWide ? 2 : 1;       // fp16 terms of q
    static constexpr int kPT = kWide ? 2 : 1;       // and of a weight
    static constexpr float kMost = 32768.0f;        // largest weight: it may grow 2^4 beyond the power of two that it was taken to
    static constexpr float kRest = 4096.0f;         // factor of a weight's second term: that of 2^15 is up to 2^3 and has to stay below 2^16
    uint32_t q[kQT][kD / 16][kTiles][2];
    float o[kPT][kRow / 16][kOfChunk][4];     // of a weight's terms; features 2 (lane / 4) (+ 1), heads 2 (lane % 4) + {0, 1}
    // of those two heads: maximum of the scores, and of score + scale's exponent; 2^(m - mo + kBase); this lane's share of the
    // sum; the bias' slope; what takes a product to a score (capped: to q.k)
    float m[kTiles][2], mo[kTiles][2], u[kTiles][2], l[kTiles][2], slope[kTiles][2], in[kTiles][2];
    bool biased;
    int each;                       // query heads of a key head, kHeads = 2

    static __device__ __forceinline__ int swizzle(int row) { return kRow == 128 ? row & 7 : (row >> 1) & 3; }
    // the unit's row of column `col` of a tile, and whether it is one
    __device__ __forceinline__ int row_of(int nt, int col) const {
        return kShared ? (col >> 2) * each + (col & 3) : kHeads == 2 ? nt * each + col : nt * 8 + col;
    }
    __device__ __forceinline__ bool is_row(int nt, int col, int rows) const {
        return kShared ? (col & 3) < each : kHeads == 2 ? col < each : nt * 8 + col < rows;
    }
    static __device__ __forceinline__ bool second(int lane) { return kShared && (lane & 2); }     // its columns are of the second key head

    // the lane's elements of its query rows, as they lie in memory
    struct alignas(4 * sizeof(T)) Four {
        T e[4];
    };
    __device__ __forceinline__ void start(const PagedAttnParams& p, float*, int b, int head0, int rows, int lane) {
        each = rows / 2;
        biased = p.slopes != nullptr;
        const T* base = static_cast<const T*>(p.q) + b * p.q_b + head0 * p.q_h;
        const bool wide = reinterpret_cast<uintptr_t>(base) % sizeof(Four) == 0 && p.q_h % 4 == 0;
        Four raw[kTiles][kD / 16];
        const T* x[kTiles];      // operand column: head lane / 4; a column without a head reads another's, for nothing
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
            x[nt] = base + (is_row(nt, lane >> 2, rows) ? row_of(nt, lane >> 2) : 0) * p.q_h + 4 * (lane & 3);
        if (wide) {
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) raw[nt][k] = *reinterpret_cast<const Four*>(x[nt] + 16 * k);
        } else {
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                for (int k = 0; k < kD / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) raw[nt][k].e[e] = x[nt][16 * k + e];
        }
        const float form_in = p.cap > 0.0f ? 1.0f : p.scale * kLog2e;        // capped: below, so that scale / cap meets a whole score
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
            float f[kD / 16][4];
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < kD / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[k][e] = is_row(nt, lane >> 2, rows) ? load_f(&raw[nt][k].e[e]) : 0.0f;
                    top = fmaxf(top, fabsf(f[k][e]));
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int x0 = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            // not finite, or nothing but zeros (and NaN): as it is
            const int shift = x0 == 128 || top == 0.0f ? 0 : 14 - max(x0, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
            for (int k = 0; k < kD / 16; ++k)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float r0 = f[k][2 * hf] * up, r1 = f[k][2 * hf + 1] * up;
#pragma unroll
                    for (int t = 0; t < kQT; ++t) {
                        q[t][k][nt][hf] = pack_f16x2(r0, r1);
                        const float2 got = unpack_f16x2(q[t][k][nt][hf]);
                        r0 -= got.x;
                        r1 -= got.y;
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = 2 * (lane & 3) + e;
                const int of_head = __shfl_sync(0xffffffffu, shift, 4 * col);
                in[nt][e] = form_in * __uint_as_float(static_cast<uint32_t>(127 - of_head) << 23);
                slope[nt][e] = biased && is_row(nt, col, rows) ? p.slopes[head0 + row_of(nt, col)] * kLog2e : 0.0f;
                m[nt][e] = mo[nt][e] = -CUDART_INF_F;
                u[nt][e] = l[nt][e] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kRow / 16; ++i)
#pragma unroll
            for (int nt = 0; nt < kOfChunk; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int x = 0; x < kPT; ++x) o[x][i][nt][e] = 0.0f;
    }

    // keys key0 .. key0 + 31 in shared memory at k, v, their scales behind v; live: bit i: key0 + i counts
    __device__ __forceinline__ void step(uint32_t k, uint32_t v, int key0, uint32_t live, int n, const ScoreForm& form,
                                         int rows, int lane) {
        const int r8 = lane & 7, mi = lane >> 3, g = lane >> 2;
        const uint32_t row = (mi & 1) * 8 + r8;
        const uint32_t c0 = static_cast<uint32_t>(((mi >> 1) ^ swizzle(r8)) << 4);
        // key 16 t + 8 hf + g of the lane
        float ks[kOfKey][kKT][2], vs[kOfKey][kKT][2];
#pragma unroll
        for (int i = 0; i < kOfKey; ++i) {
            const uint32_t a = v + Step::kBytes + 128 * (second(lane) ? 1 : i) + 16 * g;
            const float4 x = lds4(a), y = lds4(a + 128 * kHeads);
            ks[i][0][0] = x.x; ks[i][0][1] = x.y; ks[i][1][0] = x.z; ks[i][1][1] = x.w;
            vs[i][0][0] = y.x; vs[i][0][1] = y.y; vs[i][1][0] = y.z; vs[i][1][1] = y.w;
        }
        float s[kKT][kTiles][4], other[kShared ? kKT : 1][4];      // shared: the columns' products with the second key head's codes
#pragma unroll
        for (int t = 0; t < kKT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt) s[t][nt][e] = 0.0f;
                if (kShared) other[t][e] = 0.0f;
            }
        // the two tiles of keys in turn: their sums are two chains
#pragma unroll
        for (int kk = 0; kk < kRow / 32; ++kk) {
            uint32_t f[kKT][4];
#pragma unroll
            for (int t = 0; t < kKT; ++t) ldsm4(f[t], k + (t * 16 + row) * kRow + (c0 ^ (kk << 5)));
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {       // the two chunks of 16 features
                const int i = (2 * kk + hf) % (kD / 16), head = (2 * kk + hf) / (kD / 16);
#pragma unroll
                for (int t = 0; t < kKT; ++t) {
                    uint32_t a[4];
                    codes_f16<kInt8, false>(f[t][2 * hf], a[0], a[2]);
                    codes_f16<kInt8, false>(f[t][2 * hf + 1], a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < kOfChunk; ++n) {
                        const int nt = kShared ? 0 : head * kOfChunk + n;
#pragma unroll
                        for (int x = kQT - 1; x >= 0; --x)
                            mma_f16(kShared && head == 1 ? other[kShared ? t : 0] : s[t][nt], a, q[x][i][nt][0], q[x][i][nt][1]);
                    }
                }
            }
        }
        if (second(lane)) {
#pragma unroll
            for (int t = 0; t < kKT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][0][e] = other[kShared ? t : 0][e];
        }
#pragma unroll
        for (int t = 0; t < kKT; ++t)
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][nt][e] *= ks[nt / kOfChunk][t][e >> 1] * in[nt][e & 1];
        if (form.capped) {
#pragma unroll
            for (int t = 0; t < kKT; ++t)
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[t][nt][e] = kWide ? form.top * tanhf(s[t][nt][e] * form.in) : capped_score(s[t][nt][e] * form.in, form.top);
        }
        if (biased) {
#pragma unroll
            for (int t = 0; t < kKT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float away = static_cast<float>(n - 1 - key0 - t * 16 - 8 * (e >> 1) - g);
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt) s[t][nt][e] = fmaf(-slope[nt][e & 1], away, s[t][nt][e]);
                }
        }
        if (live != 0xffffffffu) {
#pragma unroll
            for (int t = 0; t < kKT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!((live >> (t * 16 + 8 * (e >> 1) + g)) & 1u)) {
#pragma unroll
                        for (int nt = 0; nt < kTiles; ++nt) s[t][nt][e] = -CUDART_INF_F;
                    }
        }
        float w[kKT][kTiles][4], sum[kTiles][2];
        auto weigh = [&](float& most_p, float& most_w) {
            most_p = most_w = 0.0f;
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) {
                sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
                for (int t = 0; t < kKT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float p0 = ex2_approx(s[t][nt][e] - m[nt][0]), p1 = ex2_approx(s[t][nt][e + 1] - m[nt][1]);
                        const float scale = vs[nt / kOfChunk][t][e >> 1];
                        sum[nt][0] += p0;
                        sum[nt][1] += p1;
                        w[t][nt][e] = p0 * u[nt][0] * scale;           // u * scale may be beyond fp32 where p is 0
                        w[t][nt][e + 1] = p1 * u[nt][1] * scale;
                        most_p = fmax3(most_p, p0, p1);
                        most_w = fmax3(most_w, w[t][nt][e], w[t][nt][e + 1]);
                    }
            }
        };
        // The maxima move only when a weight passes what they allow by 2^kGrow (the first keys always do that: theirs are infinite);
        // nothing is rescaled in between.
        float most_p, most_w;
        weigh(most_p, most_w);
        if (__any_sync(0xffffffffu, most_p > 256.0f || most_w > kMost)) {
            static_assert(kGrow == 8.0f && kBase == 10.0f, "the bounds above");
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = m[nt][e], most = mo[nt][e];
#pragma unroll
                    for (int t = 0; t < kKT; ++t) {
                        top = fmax3(top, s[t][nt][e], s[t][nt][e + 2]);
                        most = fmax3(most, s[t][nt][e] + exponent_of(vs[nt / kOfChunk][t][0]), s[t][nt][e + 2] + exponent_of(vs[nt / kOfChunk][t][1]));
                    }
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
                    }
                    const bool first = m[nt][e] == -CUDART_INF_F;
                    l[nt][e] *= first ? 0.0f : ex2_approx(m[nt][e] - top);
                    const float alpha = first ? 0.0f : ex2_approx(mo[nt][e] - most);
                    m[nt][e] = top;
                    mo[nt][e] = most;
                    u[nt][e] = top == -CUDART_INF_F ? 0.0f : ex2_approx(top - most + kBase);
                    // the tile's accumulators
#pragma unroll
                    for (int i = 0; i < kRow / 16 / (kTiles / kOfChunk); ++i)
#pragma unroll
                        for (int x = 0; x < kPT; ++x) {
                            o[x][nt / kOfChunk * (kD / 16) + i][nt % kOfChunk][e] *= alpha;
                            o[x][nt / kOfChunk * (kD / 16) + i][nt % kOfChunk][e + 2] *= alpha;
                        }
                }
            weigh(most_p, most_w);
        }
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
            l[nt][0] += sum[nt][0];
            l[nt][1] += sum[nt][1];
        }
#pragma unroll
        for (int t = 0; t < kKT; ++t) {
            uint32_t pt[kPT][kTiles][2];
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float w0 = w[t][nt][2 * hf], w1 = w[t][nt][2 * hf + 1];
#pragma unroll
                    for (int x = 0; x < kPT; ++x) {
                        uint32_t h = pack_f16x2(w0, w1);
                        if (x + 1 < kPT) {
                            const float2 got = unpack_f16x2(h);
                            w0 = (w0 - got.x) * kRest;
                            w1 = (w1 - got.y) * kRest;
                        }
                        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pt[x][nt][hf]) : "r"(h));
                    }
                }
            const uint32_t at = v + (t * 16 + row) * kRow;
#pragma unroll
            for (int i = 0; i < kRow / 32; ++i) {
                uint32_t f[4];
                ldsm4t(f, at + (c0 ^ (i << 5)));
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t a[4];
                    codes_f16<kInt8, true>(f[2 * hf], a[0], a[1]);
                    codes_f16<kInt8, true>(f[2 * hf + 1], a[2], a[3]);
                    const int head = kShared ? 0 : (2 * i + hf) / (kD / 16);
#pragma unroll
                    for (int nt = 0; nt < kOfChunk; ++nt)
#pragma unroll
                        for (int x = 0; x < kPT; ++x)
                            mma_f16(o[x][2 * i + hf][nt], a, pt[x][head * kOfChunk + nt][0], pt[x][head * kOfChunk + nt][1]);
                }
            }
        }
    }

    // the maxima and sums of the heads to shared memory
    __device__ __forceinline__ void put_stats(float* sm_m, float* sm_l, int lane) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                const int col = 2 * lane + e;
                if (lane < 4 && is_row(nt, col, kRows)) {
                    sm_m[row_of(nt, col)] = m[nt][e];
                    sm_l[row_of(nt, col)] = sum;
                }
            }
    }
    // o, taken back to the scores' maximum and scaled by f[head], written or added (add = true) to rows of kD floats
    __device__ __forceinline__ void put(float* buf, const float* f, bool add, int rows, int lane) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = 2 * (lane & 3) + e, hd = row_of(nt, col);
                if (!is_row(nt, col, rows)) continue;
                const float fr = f[hd], up = m[nt][e] == -CUDART_INF_F ? 0.0f : ex2_approx(mo[nt][e] - m[nt][e] - kBase);
#pragma unroll
                for (int i = 0; i < kD / 16; ++i)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float* y = buf + hd * kD + 16 * i + 2 * (lane >> 2) + hf;
                        auto sum = [&](int chunk) {
                            const float first = o[0][chunk][nt % kOfChunk][e + 2 * hf];
                            return kPT == 1 ? first : fmaf(o[kPT - 1][chunk][nt % kOfChunk][e + 2 * hf], 1.0f / kRest, first);
                        };
                        const float mine = second(lane) ? sum((kHeads - 1) * (kD / 16) + i) : sum(nt / kOfChunk * (kD / 16) + i);
                        const float x = mine * up * fr;
                        *y = add ? *y + x : x;
                    }
            }
    }
};

// Many units: two CTAs of four warps an SM, of which one computes and loads while the other ends a unit and begins the next. (8 key
// heads of 128, four query heads each, lengths up to: 32 x 1000 21.5 -> 17.3 us, 256 x 1000 98 -> 78, 128 x 4000 125 -> 117, 128 x 8000 214 -> 207;
// 64 x 8000 107 both; but 48 x 15000 143 -> 144, and where units are fewer than SMs, so that each is split: one of 131071 with 2 key heads
// 22.1 -> 24.6, 4 x 333 with 4 of 64 6.3 -> 7.1.)
//
// Many units of a table with room for little (the host does not know the lengths: the same units behind a wide table take the forms above, 200 x 20 25 us for 12.5): a warp a unit, seven CTAs of one an SM, which the hardware hands out. What such calls wait for is latency (queries, first keys, the
// unit's end), and that of seven units runs side by side. (Shapes above -> this: 8 key heads of 128, four query heads each, room for 32: 41 x 20 10.0 -> 7.0,
// 200 x 20 22.7 -> 13.0; room for 128, full: 54 10.9 both, 200 28.7 -> 23.0; for 256, full: 54 14.1 -> 15.9, 200 36.2 -> 32.6; 64 x 500, 16 heads 34.6 -> 27.7; but 41 x 500 19.7 -> 25.3, 30 x 20
// 5.5 -> 6.9. What has no two CTAs an SM: pairs of heads of 64, eight query heads each, 49 x 20, 4 pairs 12.4 -> 9.5, full in 128 12.5 -> 12.8, in 256 13.3 -> 17.2. fp32: 64 x 240,
// 16 heads 28.0 -> 20.9; 30 x 240, 8 heads of twelve query heads, two tiles each, 16.4 -> 20.9.)
template <typename T, int kD, int kHeads, int kNT, bool kInt8>
cudaError_t launch_w(const PagedAttnParams& p, cudaStream_t s) {
    int sms = 0;
    if (const cudaError_t e = sm_count(&sms); e != cudaSuccess) return e;
    using One = WarpCoded<T, kD, kHeads, kNT, kInt8>;
    constexpr bool kHalves = One::kTiles == 1 && One::kRow == 128;
    const int64_t units = static_cast<int64_t>(p.B) * p.h_kv * ((p.h / p.h_kv + One::kRows - 1) / One::kRows);
    const int64_t room = static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d;
    if ((room <= 128 && units > (kHalves ? 2 : 1) * sms) || (room <= 256 && units >= 3 * sms) || (room <= kShort && units >= 6 * sms))
        return launch_rows<WarpCoded<T, kD, kHeads, kNT, kInt8, kMany>, kD>(p, s);
    if constexpr (kHalves)
        if (units >= sms && (room <= 8192 || units >= 3 * sms)) return launch_rows<WarpCoded<T, kD, kHeads, kNT, kInt8, kTwo>, kD>(p, s);
    return launch_rows<One, kD>(p, s);
}

template <typename T, bool kInt8>
cudaError_t launch_t(PagedAttnParams p, cudaStream_t s) {
    const int group = p.h / p.h_kv;
    constexpr bool kBf16 = sizeof(T) == 2;
    if (p.d == 128) {
        if constexpr (kBf16)
            if (group > 8) return launch_w<T, 128, 1, 2, kInt8>(p, s);
        return launch_w<T, 128, 1, 1, kInt8>(p, s);
    }
    // heads of 64 go two at a time
    if (group <= 8 && p.h_kv % 2 == 0) {
        p.h_kv /= 2;
        p.cache.head_stride *= 2;
        return group <= 4 ? launch_w<T, 64, 2, 0, kInt8>(p, s) : launch_w<T, 64, 2, 1, kInt8>(p, s);
    }
    if constexpr (kBf16)
        if (group > 8) return launch_w<T, 64, 1, 2, kInt8>(p, s);
    return launch_w<T, 64, 1, 1, kInt8>(p, s);
}

}  // namespace
}  // namespace mha
