// paged_attn.cu -- attention of one new token a sequence over a paged key/value cache.
//
//   s_j = cap tanh(scale q.k_j / cap) - slope (n - 1 - j),  o = sum_j softmax_j(s) v_j,  j < n
// in one pass with a running maximum m and sum l. n = 0 gives zeros.
//
// HBM-bound: K and V of every cached position are read once, 4 d_k bytes a position and key head in
// bf16, for 4 d_k flop a query head. The heads that share a key head are the rows of one matrix
// product (mma.sync in bf16: CUDA cores could not keep up from 4 heads on), so the cache is read once for up to 16 of them (8
// in fp32); further ones are another unit, which reads it again.
//
// Work split, loads and join: paged_line.cuh.
//
// Measured (bf16): 16 sequences of 8192, 16 heads of 64, 537 MB: 89-97 us by box, 5.5-6.0 TB/s (0.81-0.89 of measured copy
// bandwidth); 48 ragged ones up to 15000, 32 / 8 heads of 128, capped, 1.5 GB: 237 us, 6.4 TB/s (0.94); one of 131071, 16 / 2 heads: 30.5 us, of which
// 20 us are its traffic: the two launches, the look-ups (length, page, key: three dependent loads) and the join are the
// rest, 11 us at any length, and 7.2 TB/s is what each further key costs.

#include "paged_line.cuh"

namespace mha {
namespace {

// 4 KB of keys, 4 KB of values a step
template <typename T, int kD>
using Halves = StepOf<kD * static_cast<int>(sizeof(T)), static_cast<int>(sizeof(T)), 4096 / (kD * static_cast<int>(sizeof(T))), 3, 0, 8, 0, 1, 4>;

// ------------------------------------------------------------ a warp's heads: bf16, matrix instructions
// Both products are taken transposed, so that the long sides are the matrix instruction's 16 rows and the
// query heads its 8 columns: S^T = K q^T (16 keys x d_k times d_k x 8 heads) and o^T = V^T P^T (16 features x
// 16 keys times 16 keys x 8 heads). With the heads as the 16 rows, up to 8 heads fill half of every
// instruction and of the accumulators. P^T turns from result to operand layout by a register transpose.
template <int kD, int kNT>          // kNT tiles of 8 heads
struct WarpBf16 {
    using T = __nv_bfloat16;
    using Step = Halves<T, kD>;
    static constexpr int kRows = 8 * kNT, kBufs = 4;
    static constexpr int kQFloats = 0;      // shared memory for the query rows (they stay in registers)
    static constexpr bool kSplits = true;   // units among CTAs
    static constexpr int kKeys = Step::kKeys;
    static constexpr int kKT = kKeys / 16;
    uint32_t q[kD / 16][kNT][2];
    float o[kD / 16][kNT][4];       // features lane / 4 (+ 8), heads 2 (lane % 4) + {0, 1}
    float m[kNT][2], l[kNT][2], slope[kNT][2];     // of those two heads; l is this lane's share

    static __device__ __forceinline__ int swizzle(int row) { return row & 7; }

    __device__ __forceinline__ void start(const PagedAttnParams& p, float*, int b, int head0, int rows, int lane) {
        const T* base = static_cast<const T*>(p.q) + b * p.q_b + head0 * p.q_h;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int row = nt * 8 + (lane >> 2);      // operand column: head lane / 4
            const T* x = base + row * p.q_h + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    __nv_bfloat162 v = __floats2bfloat162_rn(0.0f, 0.0f);
                    if (row < rows) {
                        v.x = x[16 * k + 8 * hf];
                        v.y = x[16 * k + 8 * hf + 1];
                    }
                    q[k][nt][hf] = *reinterpret_cast<uint32_t*>(&v);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k][nt][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hd = nt * 8 + 2 * (lane & 3) + e;
                slope[nt][e] = p.slopes != nullptr && hd < rows ? p.slopes[head0 + hd] * kLog2e : 0.0f;
                m[nt][e] = -CUDART_INF_F;
                l[nt][e] = 0.0f;
            }
        }
    }

    // keys key0 .. key0 + kKeys - 1 in shared memory at k, v; live: bit i: key0 + i counts
    __device__ __forceinline__ void step(uint32_t k, uint32_t v, int key0, uint32_t live, int n, const ScoreForm& form,
                                         int rows, int lane) {
        constexpr int kRow = Step::kRow;
        const int r8 = lane & 7, mi = lane >> 3;
        float s[kKT][kNT][4];
#pragma unroll
        for (int t = 0; t < kKT; ++t) {
            const uint32_t row = k + (t * 16 + (mi & 1) * 8 + r8) * kRow;
            const uint32_t c0 = static_cast<uint32_t>(((mi >> 1) ^ r8) << 4);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][nt][e] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
                uint32_t f[4];
                ldsm4(f, row + (c0 ^ (kk << 5)));
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) mma16816(s[t][nt], f, q[kk][nt][0], q[kk][nt][1]);
            }
        }
        bool more = false;
#pragma unroll
        for (int t = 0; t < kKT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = t * 16 + (lane >> 2) + 8 * (e >> 1);
                const bool ok = (live >> i) & 1u;
                const float away = static_cast<float>(n - 1 - key0 - i);
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    s[t][nt][e] = ok ? form.of<false>(s[t][nt][e], slope[nt][e & 1], away) : -CUDART_INF_F;
                    more |= s[t][nt][e] > m[nt][e & 1] + kGrow;
                }
            }
        // The maximum moves only when a score passes it by kGrow (the first keys always do); until then
        // the weights stay below 2^kGrow and nothing is rescaled.
        if (__any_sync(0xffffffffu, more)) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = m[nt][e];
#pragma unroll
                    for (int t = 0; t < kKT; ++t) top = fmax3(top, s[t][nt][e], s[t][nt][e + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float alpha = m[nt][e] == -CUDART_INF_F ? 0.0f : ex2_approx(m[nt][e] - top);
                    m[nt][e] = top;
                    l[nt][e] *= alpha;
#pragma unroll
                    for (int i = 0; i < kD / 16; ++i) {
                        o[i][nt][e] *= alpha;
                        o[i][nt][e + 2] *= alpha;
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < kKT; ++t) {
            // A weight goes into the product as two bf16 numbers, its rounding and the rest: the values' own rounding is
            // then the only one. The second product costs no time (the loads bound the kernel); with one the result
            // was off by 2.4e-3 where rounding the exact result to bf16 gives 1.7e-3.
            uint32_t pt[kNT][2], rest[kNT][2];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const float r0 = m[nt][0] == -CUDART_INF_F ? 0.0f : m[nt][0], r1 = m[nt][1] == -CUDART_INF_F ? 0.0f : m[nt][1];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float p0 = ex2_approx(s[t][nt][2 * hf] - r0), p1 = ex2_approx(s[t][nt][2 * hf + 1] - r1);
                    l[nt][0] += p0;
                    l[nt][1] += p1;
                    const uint32_t hi = pack_bf16x2(p0, p1);
                    const uint32_t lo = pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pt[nt][hf]) : "r"(hi));
                    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(rest[nt][hf]) : "r"(lo));
                }
            }
            const uint32_t row = v + (t * 16 + (mi >> 1) * 8 + r8) * kRow;
            const uint32_t c0 = static_cast<uint32_t>(((mi & 1) ^ r8) << 4);
#pragma unroll
            for (int i = 0; i < kD / 16; ++i) {
                uint32_t f[4];
                ldsm4t(f, row + (c0 ^ (i << 5)));
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    mma16816(o[i][nt], f, pt[nt][0], pt[nt][1]);
                    mma16816(o[i][nt], f, rest[nt][0], rest[nt][1]);
                }
            }
        }
    }

    // the maxima and sums of the heads to shared memory
    __device__ __forceinline__ void put_stats(float* sm_m, float* sm_l, int lane) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                if (lane < 4) {
                    sm_m[nt * 8 + 2 * lane + e] = m[nt][e];
                    sm_l[nt * 8 + 2 * lane + e] = sum;
                }
            }
    }
    // o scaled by f[head], written or added (add = true) to rows of kD floats
    __device__ __forceinline__ void put(float* buf, const float* f, bool add, int rows, int lane) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int hd = nt * 8 + 2 * (lane & 3) + e;
                if (hd >= rows) continue;
                const float fr = f[hd];
#pragma unroll
                for (int i = 0; i < kD / 16; ++i)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float* y = buf + hd * kD + 16 * i + 8 * hf + (lane >> 2);
                        const float x = o[i][nt][e + 2 * hf] * fr;
                        *y = add ? *y + x : x;
                    }
            }
    }
};

// ------------------------------------------------------------ a warp's rows: fp32, CUDA cores
template <int kD, int kR>
struct WarpF32 {
    using T = float;
    using Step = Halves<T, kD>;
    static constexpr int kRows = kR, kBufs = 4;
    static constexpr int kQFloats = kR * kD;
    static constexpr bool kSplits = true;
    static constexpr int kKeys = Step::kKeys;      // 8 or 16
    static constexpr int kLanes = 32 / kKeys;             // lanes that share a key's dot product: 4 or 2
    static constexpr int kDims = kD / kLanes;             // features a lane multiplies: 32
    static constexpr int kOwn = kD / 32;                  // features of o a lane keeps
    float o[kR][kOwn];
    float m[kR], l[kR];                                   // l is this lane's share
    uint32_t q;                                           // the unit's query rows in shared memory
    float slope[kR];

    // two (or four) keys of a quarter-warp's 16-byte reads land in different 64-byte (32-byte) parts
    static __device__ __forceinline__ int swizzle(int row) { return kLanes == 4 ? (row & 1) << 2 : (row & 3) << 1; }

    __device__ __forceinline__ void start(const PagedAttnParams& p, float* shared_q, int b, int head0, int rows, int) {
        const float* x = static_cast<const float*>(p.q) + b * p.q_b + head0 * p.q_h;
        for (int i = threadIdx.x; i < kR * kD; i += Step::kThreads)
            shared_q[i] = i < rows * kD ? x[(i / kD) * p.q_h + i % kD] : 0.0f;
        __syncthreads();      // the last unit's readers are behind the barriers of its end
        q = smem_u32(shared_q);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            slope[r] = p.slopes != nullptr && r < rows ? p.slopes[head0 + r] * kLog2e : 0.0f;
            m[r] = -CUDART_INF_F;
            l[r] = 0.0f;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) o[r][e] = 0.0f;
        }
    }

    // All kR rows are computed, whether the unit has them or not: their chains then run side by side (with a test a
    // row, 16 x 8192 at 4 heads a key head took 125 us).
    __device__ __forceinline__ void step(uint32_t k, uint32_t v, int key0, uint32_t live, int n, const ScoreForm& form,
                                         int rows, int lane) {
        constexpr int kRow = Step::kRow;
        const int key = lane / kLanes, part = lane % kLanes;   // chunks part, part + kLanes, ... of the key
        float4 kv[kDims / 4];
#pragma unroll
        for (int i = 0; i < kDims / 4; ++i)
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(kv[i].x), "=f"(kv[i].y), "=f"(kv[i].z), "=f"(kv[i].w)
                         : "r"(k + key * kRow + (((i * kLanes + part) ^ swizzle(key)) << 4)));
        float vv[kKeys][kOwn];
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            const int byte = lane * kOwn * 4;
            const uint32_t a = v + j * kRow + (((byte >> 4) ^ swizzle(j)) << 4) + (byte & 15);
            if constexpr (kOwn == 4)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(vv[j][0]), "=f"(vv[j][1]), "=f"(vv[j][2]), "=f"(vv[j][3]) : "r"(a));
            else
                asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(vv[j][0]), "=f"(vv[j][1]) : "r"(a));
        }
        const bool ok = (live >> key) & 1u;
        const float away = static_cast<float>(n - 1 - key0 - key);
        float s[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
            for (int i = 0; i < kDims / 4; ++i) {
                float4 x;
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(q + (r * kD + (i * kLanes + part) * 4) * 4));
                d0 = fmaf(kv[i].x, x.x, d0);
                d1 = fmaf(kv[i].y, x.y, d1);
                d0 = fmaf(kv[i].z, x.z, d0);
                d1 = fmaf(kv[i].w, x.w, d1);
            }
            s[r] = d0 + d1;
        }
        bool more = false;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
            for (int w = 1; w < kLanes; w <<= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], w);
            s[r] = ok ? form.of<true>(s[r], slope[r], away) : -CUDART_INF_F;
            more |= s[r] > m[r];
        }
        if (__any_sync(0xffffffffu, more)) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                float top = fmaxf(s[r], m[r]);
#pragma unroll
                for (int w = kLanes; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float alpha = m[r] == -CUDART_INF_F ? 0.0f : ex2_approx(m[r] - top);   // 1 where it stays
                l[r] *= alpha;
#pragma unroll
                for (int e = 0; e < kOwn; ++e) o[r][e] *= alpha;
                m[r] = top;
            }
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const float w = ex2_approx(s[r] - (m[r] == -CUDART_INF_F ? 0.0f : m[r]));
            if (part == 0) l[r] += w;
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j * kLanes);
#pragma unroll
                for (int e = 0; e < kOwn; ++e) o[r][e] = fmaf(wj, vv[j][e], o[r][e]);
            }
        }
    }

    __device__ __forceinline__ void put_stats(float* sm_m, float* sm_l, int lane) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const float sum = warp_add(l[r]);
            if (lane == 0) {
                sm_m[r] = m[r];
                sm_l[r] = sum;
            }
        }
    }
    __device__ __forceinline__ void put(float* buf, const float* f, bool add, int rows, int lane) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (r >= rows) break;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                float* y = buf + r * kD + lane * kOwn + e;
                const float x = o[r][e] * f[r];
                *y = add ? *y + x : x;
            }
        }
    }
};
template <int kD>
cudaError_t launch_d(const PagedAttnParams& p, bool bf16, cudaStream_t s) {
    const int group = p.h / p.h_kv;
    if (bf16) return group <= 8 ? launch_rows<WarpBf16<kD, 1>, kD>(p, s) : launch_rows<WarpBf16<kD, 2>, kD>(p, s);
    if (group == 1) return launch_rows<WarpF32<kD, 1>, kD>(p, s);
    if (group == 2) return launch_rows<WarpF32<kD, 2>, kD>(p, s);
    if (group <= 4) return launch_rows<WarpF32<kD, 4>, kD>(p, s);
    return launch_rows<WarpF32<kD, 8>, kD>(p, s);
}

}  // namespace

size_t paged_attn_workspace(bool, int, int, int, int d) {
    return line_workspace(d, 1);
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, cudaStream_t s) {
    return p.d == 64 ? launch_d<64>(p, bf16, s) : launch_d<128>(p, bf16, s);
}

}  // namespace mha
