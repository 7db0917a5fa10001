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
// Work split: a unit is (sequence, key head, tile of query heads). All units' keys, in blocks of
// kWarps steps, form one line that is cut into equal pieces, one CTA a piece, whatever the lengths
// are: one long sequence fills the GPU as well as many ragged ones. A piece that covers part of a unit
// leaves (m, l, o) in the workspace, in a slot given by its CTA; a second kernel joins them in the order of
// the CTAs, so the result does not depend on timing. There are at most (CTAs - 1) units to join.
//
// Inside a CTA the warps are independent: each loads its own steps (4 KB of keys, 4 KB of values) with
// cp.async into kStages private stages that run ahead across units, so 128 KB an SM are in flight
// and no barrier stands in the loop; at the end of a unit the warps' sums are joined through
// shared memory. Keys behind the end of a sequence, and pages outside the pool, arrive as zeros and get
// no weight: what lies there is never touched.
//
// Measured (bf16): 16 sequences of 8192, 16 heads of 64, 537 MB: 89-97 us by box, 5.5-6.0 TB/s (0.81-0.89 of measured copy
// bandwidth); 48 ragged ones up to 15000, 32 / 8 heads of 128, capped, 1.5 GB: 237 us, 6.4 TB/s (0.94); one of 131071, 16 / 2 heads: 30.5 us, of which
// 20 us are its traffic: the two launches, the look-ups (length, page, key: three dependent loads) and the join are the
// rest, 11 us at any length, and 7.2 TB/s is what each further key costs.
#include <algorithm>

#include <math_constants.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx_serve.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kStepBytes = 4096;        // of keys, and of values, in one step of a warp
constexpr int kMaxCtas = 192;           // slots of the workspace
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWholeBlocks = 4;
constexpr float kGrow = 8.0f;           // log2 units the maximum may grow before o and l are rescaled

template <typename T, int kD>
struct Step {
    static constexpr int kRow = kD * static_cast<int>(sizeof(T));   // bytes of a key
    static constexpr int kKeys = kStepBytes / kRow;
    static constexpr int kChunks = kRow / 16;
};
constexpr int kMaxRows = 16;

struct JoinDesc {
    int c0, c1;         // CTAs whose pieces make up the unit; c1 < c0: nothing to join
    int b, unit;
    int first_slot;     // slot of c0's piece (every later CTA's is 0)
};

// One piece in the workspace: m[16], l[16], o[16][kD]
template <int kD>
__host__ __device__ constexpr int slot_floats() { return 2 * kMaxRows + kMaxRows * kD; }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A score in log2 units from q.k: capped, minus the distance bias. fp32 takes the library's tanh: 2^-21 of a
// score of 50 would be an error of 2 10^-5 in a weight, which bf16 values hide and fp32 ones do not.
struct ScoreForm {
    float in, top;     // capped: s = top * tanh(dot * in), else dot * in
    bool capped;
    template <bool kExact>
    __device__ __forceinline__ float of(float dot, float slope, float away) const {
        const float s = !capped ? dot * in : kExact ? top * tanhf(dot * in) : capped_score(dot * in, top);
        return fmaf(-slope, away, s);
    }
};

// ------------------------------------------------------------ a warp's heads: bf16, matrix instructions
// Both products are taken transposed, so that the long sides are the matrix instruction's 16 rows and the
// query heads its 8 columns: S^T = K q^T (16 keys x d_k times d_k x 8 heads) and o^T = V^T P^T (16 features x
// 16 keys times 16 keys x 8 heads). With the heads as the 16 rows, up to 8 heads fill half of every
// instruction and of the accumulators. P^T turns from result to operand layout by a register transpose.
template <int kD, int kNT>          // kNT tiles of 8 heads
struct WarpBf16 {
    using T = __nv_bfloat16;
    static constexpr int kRows = 8 * kNT;
    static constexpr int kQFloats = 0;      // shared memory for the query rows (they stay in registers)
    static constexpr int kKeys = Step<T, kD>::kKeys;
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
        constexpr int kRow = Step<T, kD>::kRow;
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
    static constexpr int kRows = kR;
    static constexpr int kQFloats = kR * kD;
    static constexpr int kKeys = Step<T, kD>::kKeys;      // 8 or 16
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
        for (int i = threadIdx.x; i < kR * kD; i += kThreads)
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
        constexpr int kRow = Step<T, kD>::kRow;
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

// ------------------------------------------------------------ the line of blocks
struct Cursor {
    int b, unit;        // unit of the sequence: key head * head tiles + head tile
    int blk, nblk;
    int n;              // the sequence's length
};

struct Lens {
    const int32_t* kv_lens;
    int64_t room;
    int block;          // keys of a block
    __device__ __forceinline__ int len(int b) const {
        const int n = max(kv_lens[b], 0);
        return static_cast<int>(min(static_cast<int64_t>(n), room));
    }
    __device__ __forceinline__ int blocks(int n) const { return n / block + (n % block != 0); }
};

struct Found {
    long long before;    // blocks before sequence b
    int b;
};

struct Shared {
    float m[kWarps][kMaxRows], l[kWarps][kMaxRows], f[kWarps][kMaxRows];
    long long scan[kWarps];
    Found found[2];
};

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Inclusive scan over the warp.
__device__ __forceinline__ long long warp_scan64(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long other = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += other;
    }
    return v;
}

template <typename W, int kD>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    using T = typename W::T;
    using S = Step<T, kD>;
    constexpr int kKeys = S::kKeys;
    constexpr int kSlot = slot_floats<kD>();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.h / p.h_kv;
    const int head_tiles = (group + W::kRows - 1) / W::kRows;
    const int units = p.h_kv * head_tiles;
    // positions stay below 2^31 with a block to spare
    const int64_t room = min(static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d, static_cast<int64_t>(0x7ffff000));
    const Lens lens{p.kv_lens, room, kKeys * kWarps};
    JoinDesc* join = reinterpret_cast<JoinDesc*>(p.partial + static_cast<int64_t>(kMaxCtas) * 2 * kSlot);
    pdl_trigger();
    pdl_wait();

    const int c = blockIdx.x;
    Cursor at;               // the block that is computed
    long long t0, t1;        // the CTA's blocks of the line
    int early = -1;          // page of the warp's first key `lane`
    if (p.direct) {
        // a CTA a unit: the first pages are looked up beside the length
        at.b = c / units;
        at.unit = c - at.b * units;
        at.blk = 0;
        const int key = warp * kKeys + lane, held = p.kv_lens[at.b];
        if (lane < kKeys && key < room) early = p.cache.table[at.b * p.cache.table_stride + p.cache.page.div(key)];
        at.n = static_cast<int>(min(static_cast<int64_t>(max(held, 0)), room));
        at.nblk = lens.blocks(at.n);
        t0 = 0;
        t1 = at.nblk;
        if (held > room && threadIdx.x == 0) atomicCAS(p.status, 0, 0x501);
        if (at.n == 0) {
            const int kh = at.unit / head_tiles, ht = at.unit - kh * head_tiles;
            const int many = min(group - ht * W::kRows, W::kRows), first = kh * group + ht * W::kRows;
            for (int i = threadIdx.x; i < many * kD; i += kThreads)
                store_f(static_cast<T*>(p.out) + at.b * p.o_b + (first + i / kD) * p.o_h + i % kD, 0.0f);
            return;
        }
    } else {
        // ---- total number of blocks, and the sequences that have none. Up to 32 sequences are summed by every warp for
        // itself, without a barrier before the first loads.
        const bool few = p.B <= 32;
        long long total = 0, inc = 0, v = 0;     // few: blocks (of one unit) up to and of sequence `lane`
        if (few) {
            if (lane < p.B) {
                v = lens.blocks(lens.len(lane));
                if (p.kv_lens[lane] > room) atomicCAS(p.status, 0, 0x501);
            }
            inc = warp_scan64(v, lane);
            total = __shfl_sync(0xffffffffu, inc, 31);
        } else {
            for (int b = threadIdx.x; b < p.B; b += kThreads) {
                if (p.kv_lens[b] > room) atomicCAS(p.status, 0, 0x501);
                v += lens.blocks(lens.len(b));
            }
            v = warp_sum64(v);
            if (lane == 0) sh.scan[warp] = v;
            __syncthreads();
            for (int w = 0; w < kWarps; ++w) total += sh.scan[w];
        }
        total *= units;
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (lens.len(b) > 0) continue;
            for (int i = threadIdx.x; i < p.h * kD; i += kThreads)
                store_f(static_cast<T*>(p.out) + b * p.o_b + (i / kD) * p.o_h + i % kD, 0.0f);
        }
        const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
        if (c >= ctas) {
            if (threadIdx.x == 0 && !p.whole) join[c] = JoinDesc{0, -1, 0, 0, 0};
            return;
        }
        // CTA c takes blocks [c total / ctas, (c + 1) total / ctas); block t belongs to the last CTA that starts at or before it
        const bool small = total < (1 << 24);       // kMaxCtas * total fits 32 bits: divisions a quarter as long
        auto start_of = [&](long long i) -> long long {
            return small ? static_cast<uint32_t>(i * total) / static_cast<uint32_t>(ctas) : i * total / ctas;
        };
        t0 = start_of(c);
        t1 = start_of(c + 1);
        auto owner = [&](long long t) { return static_cast<int>(((t + 1) * ctas + total - 1) / total - 1); };

        // ---- the sequences that t0 and t1 fall into (t1 may be the end of the line)
        Found found[2] = {};
        if (few) {
            const long long lo = (inc - v) * units, hi = inc * units;
            const int b0 = __ffs(__ballot_sync(0xffffffffu, t0 >= lo && t0 < hi)) - 1;
            const int b1 = max(__ffs(__ballot_sync(0xffffffffu, t1 >= lo && t1 < hi)) - 1, 0);
            found[0] = Found{__shfl_sync(0xffffffffu, lo, b0), b0};
            found[1] = Found{__shfl_sync(0xffffffffu, lo, b1), b1};
        } else {
            long long acc = 0;   // blocks (of one unit) before sequence b0
            for (int b0 = 0; b0 < p.B; b0 += kThreads) {
                const int b = b0 + threadIdx.x;
                v = b < p.B ? lens.blocks(lens.len(b)) : 0;
                inc = warp_scan64(v, lane);
                __syncthreads();
                if (lane == 31) sh.scan[warp] = inc;
                __syncthreads();
                long long all = 0;
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) inc += sh.scan[w];
                    all += sh.scan[w];
                }
                const long long lo = (acc + inc - v) * units, hi = (acc + inc) * units;
                if (t0 >= lo && t0 < hi) sh.found[0] = Found{lo, b};
                if (t1 >= lo && t1 < hi) sh.found[1] = Found{lo, b};
                acc += all;
                if (t1 < acc * units) break;
            }
            __syncthreads();
            found[0] = sh.found[0];
            found[1] = sh.found[1];
        }
        auto cursor_at = [&](long long t, const Found& f) {
            Cursor x;
            x.b = f.b;
            x.n = lens.len(x.b);
            x.nblk = lens.blocks(x.n);
            const long long rem = t - f.before;
            x.unit = small ? static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(x.nblk)) : static_cast<int>(rem / x.nblk);
            x.blk = static_cast<int>(rem - static_cast<long long>(x.unit) * x.nblk);
            return x;
        };
        at = cursor_at(t0, found[0]);
        if (p.whole) {
            // units are not split: a CTA takes those that start in its piece of the line
            if (t1 < total) {
                const Cursor e = cursor_at(t1, found[1]);
                if (e.blk > 0) t1 += e.nblk - e.blk;
            }
        } else if (threadIdx.x == 0) {
            JoinDesc d{0, -1, 0, 0, 0};
            const long long u0 = t0 - at.blk;       // first block of the unit
            if (at.blk > 0 && owner(u0) == c - 1) {  // the first of the CTAs that continue it describes the join
                d.c0 = c - 1;
                d.c1 = owner(u0 + at.nblk - 1);
                d.b = at.b;
                d.unit = at.unit;
                d.first_slot = start_of(c - 1) == u0 ? 0 : 1;
            }
            join[c] = d;
        }
    }
    auto advance = [&](Cursor& x) {
        if (++x.blk < x.nblk) return;
        x.blk = 0;
        if (++x.unit < units) return;
        x.unit = 0;
        do {
            if (++x.b >= p.B) { x.b = p.B; return; }   // past the last block: never followed
            x.n = lens.len(x.b);
            x.nblk = lens.blocks(x.n);
        } while (x.n == 0);
    };

    if (p.whole && at.blk > 0) {      // never where a CTA has a unit of its own
        t0 += at.nblk - at.blk;
        at.blk = at.nblk - 1;
        advance(at);
    }

    // ---- loads: lane i looks up the page of key i of the step one step ahead of its loads
    Cursor ahead = at;
    long long t_ahead = t0;
    int page = -1, slot = 0, kvh = 0;
    bool inside = false;
    const uint32_t stage0 = smem_u32(smem) + warp * (kStages * 2 * kStepBytes);
    const char* k_lane = static_cast<const char*>(p.cache.k) + (lane % S::kChunks) * 16;
    const long long v_minus_k = static_cast<const char*>(p.cache.v) - static_cast<const char*>(p.cache.k);
    auto look_up = [&](bool first = false) {
        inside = false;
        if (t_ahead < t1) {
            const int key = (ahead.blk * kWarps + warp) * kKeys + lane;
            kvh = ahead.unit / head_tiles;
            if (lane < kKeys && key < ahead.n) {
                const int i = p.cache.page.div(key);
                slot = key - i * static_cast<int>(p.cache.page.d);
                page = first && p.direct ? early : p.cache.table[ahead.b * p.cache.table_stride + i];
                inside = true;
            }
            advance(ahead);
        }
        ++t_ahead;
    };
    auto issue = [&](int stage) -> uint32_t {
        const bool ok = inside && page >= 0 && page < p.cache.n_pages;
        if (inside && !ok) atomicCAS(p.status, 0, 0x501);
        const long long off = ok ? (page * p.cache.page_stride + slot * p.cache.slot_stride + kvh * p.cache.head_stride) *
                                       static_cast<int>(sizeof(T)) : 0;
        const uint32_t live = __ballot_sync(0xffffffffu, ok);
        if (live != 0) {
            constexpr int kRowsPer = 32 / S::kChunks > 0 ? 32 / S::kChunks : 1;   // rows an instruction of the warp covers
            const int row0 = lane / S::kChunks, col = lane % S::kChunks;
            const uint32_t k = stage0 + stage * (2 * kStepBytes) + row0 * S::kRow;
#pragma unroll
            for (int i = 0; i < kStepBytes / 512; ++i) {
                const int row = i * kRowsPer + row0;
                const char* src = k_lane + __shfl_sync(0xffffffffu, off, row);
                const bool on = (live >> row) & 1u;
                const uint32_t dst = k + i * (kRowsPer * S::kRow) + ((col ^ W::swizzle(row)) << 4);
                cp_async16(dst, src, on);
                cp_async16(dst + kStepBytes, src + v_minus_k, on);
            }
        }
        cp_commit();
        return live;
    };
    uint32_t live[kStages];
    look_up(true);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        live[s] = issue(s);
        look_up();
    }

    const ScoreForm form{p.cap > 0.0f ? p.scale / p.cap : p.scale * kLog2e, p.cap * kLog2e, p.cap > 0.0f};
    float* buf = reinterpret_cast<float*>(smem + kWarps * kStages * 2 * kStepBytes);   // 4 x [rows][kD], then the query rows (fp32)
    W w;
    bool fresh = true, first_piece = true;
    int piece_blk = at.blk, stage = 0, rows = 0, head0 = 0;
    for (long long t = t0; t < t1; ++t) {
        if (fresh) {
            const int kh = at.unit / head_tiles, ht = at.unit - kh * head_tiles;
            rows = min(group - ht * W::kRows, W::kRows);
            head0 = kh * group + ht * W::kRows;
            w.start(p, buf + 4 * W::kRows * kD, at.b, head0, rows, lane);
            piece_blk = at.blk;
            fresh = false;
        }
        cp_wait<kStages - 2>();
        __syncwarp();
        const int next = stage + kStages - 1 >= kStages ? stage - 1 : stage + kStages - 1;
        live[kStages - 1] = issue(next);
        look_up();
        if (live[0] != 0) {
            const uint32_t k = stage0 + stage * (2 * kStepBytes);
            w.step(k, k + kStepBytes, (at.blk * kWarps + warp) * kKeys, live[0], at.n, form, rows, lane);
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s + 1 < kStages; ++s) live[s] = live[s + 1];
        stage = stage + 1 == kStages ? 0 : stage + 1;

        const bool unit_done = at.blk + 1 == at.nblk;
        if (unit_done || t + 1 == t1) {
            // ---- join the warps: scaled sums of warps 4-7 in four buffers, warps 0-3 add theirs, all sum the four
            w.put_stats(sh.m[warp], sh.l[warp], lane);
            __syncthreads();
            if (lane < W::kRows) {
                float M = -CUDART_INF_F;
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sh.m[i][lane]);
                const float mw = sh.m[warp][lane];
                sh.f[warp][lane] = mw == -CUDART_INF_F ? 0.0f : ex2_approx(mw - M);
            }
            __syncwarp();
            float* own = buf + (warp & 3) * (W::kRows * kD);
            if (warp >= 4) w.put(own, sh.f[warp], false, rows, lane);
            __syncthreads();
            if (warp < 4) w.put(own, sh.f[warp], true, rows, lane);
            __syncthreads();
            const bool whole = unit_done && piece_blk == 0;
            float* slot_m = p.partial + (static_cast<int64_t>(c) * 2 + (first_piece ? 0 : 1)) * kSlot;
            for (int i = threadIdx.x; i < rows * kD; i += kThreads) {
                const int row = i / kD;
                float a = 0.0f;
#pragma unroll
                for (int s = 0; s < 4; ++s) a += buf[s * (W::kRows * kD) + i];
                if (whole) {
                    float L = 0.0f;
                    for (int s = 0; s < kWarps; ++s) L += sh.l[s][row] * sh.f[s][row];
                    store_f(static_cast<T*>(p.out) + at.b * p.o_b + (head0 + row) * p.o_h + i % kD,
                            L > 0.0f ? a / L : (L == 0.0f ? 0.0f : L));   // no key at all (bad pages): zeros; NaN stays
                } else {
                    slot_m[2 * kMaxRows + i] = a;
                }
            }
            if (!whole && threadIdx.x < rows) {
                float M = -CUDART_INF_F, L = 0.0f;
                for (int s = 0; s < kWarps; ++s) {
                    M = fmaxf(M, sh.m[s][threadIdx.x]);
                    L += sh.l[s][threadIdx.x] * sh.f[s][threadIdx.x];
                }
                slot_m[threadIdx.x] = M;
                slot_m[kMaxRows + threadIdx.x] = L;
            }
            __syncthreads();   // the statistics are read before the next unit's overwrite them
            fresh = true;
            first_piece = false;
        }
        advance(at);
    }
    cp_wait<0>();
}

// Joins the pieces of a unit that several CTAs share: block (c, row). Thread i weighs piece i (there are
// at most kMaxCtas), then groups of kD / 4 threads sum every kGroups-th piece, 16 bytes a thread.
constexpr int kJoinThreads = 256;
constexpr int kEarly = 8;        // loads of a thread that do not wait for the weights (one of 131071: 31.8 -> 30.5 us, of 16000: 12.9 -> 12.1)
template <typename T, int kD>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int rows_tile) {
    constexpr int kSlot = slot_floats<kD>();
    constexpr int kCols = kD / 4;
    constexpr int kGroups = kJoinThreads / kCols;
    static_assert(kMaxCtas <= kJoinThreads, "one thread a piece");
    __shared__ float sh_f[kJoinThreads], sh_x[2][kJoinThreads / 32];
    __shared__ float4 sh_o[kGroups][kCols];
    pdl_trigger();
    pdl_wait();
    const JoinDesc d = reinterpret_cast<const JoinDesc*>(p.partial + static_cast<int64_t>(kMaxCtas) * 2 * kSlot)[blockIdx.x];
    if (d.c1 < d.c0) return;
    const int group = p.h / p.h_kv;
    const int head_tiles = (group + rows_tile - 1) / rows_tile;
    const int kh = d.unit / head_tiles, ht = d.unit - kh * head_tiles;
    const int row = blockIdx.y;
    if (row >= min(group - ht * rows_tile, rows_tile)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pieces = d.c1 - d.c0 + 1;
    const float* slots = p.partial + static_cast<int64_t>(d.c0) * 2 * kSlot;   // piece i at 2 i kSlot, piece 0 at first_slot
    const float* mine = slots + (tid == 0 ? d.first_slot : 2 * tid) * kSlot;
    const int g = tid / kCols, x = tid % kCols;
    auto at = [&](int i) {
        return reinterpret_cast<const float4*>(slots + (i == 0 ? d.first_slot : 2 * i) * kSlot + 2 * kMaxRows + row * kD)[x];
    };
    float4 early[kEarly];      // on their way while the weights are found
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
        if (g + i * kGroups < pieces) early[i] = at(g + i * kGroups);
    const float mi = tid < pieces ? mine[row] : -CUDART_INF_F;
    const float li = tid < pieces ? mine[kMaxRows + row] : 0.0f;
    float M = mi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) sh_x[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) M = fmaxf(M, sh_x[0][i]);
    const float f = mi == -CUDART_INF_F ? 0.0f : ex2_approx(mi - M);
    sh_f[tid] = f;
    const float sum = warp_add(li * f);
    if (lane == 0) sh_x[1][warp] = sum;
    __syncthreads();
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](int i, const float4& v) {
        const float w = sh_f[i];
        a.x = fmaf(v.x, w, a.x);
        a.y = fmaf(v.y, w, a.y);
        a.z = fmaf(v.z, w, a.z);
        a.w = fmaf(v.w, w, a.w);
    };
#pragma unroll
    for (int i = 0; i < kEarly; ++i)
        if (g + i * kGroups < pieces) add(g + i * kGroups, early[i]);
#pragma unroll 4
    for (int i = g + kEarly * kGroups; i < pieces; i += kGroups) add(i, at(i));
    sh_o[g][x] = a;
    __syncthreads();
    if (tid < kD) {
        float L = 0.0f, v = 0.0f;
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) L += sh_x[1][i];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) v += reinterpret_cast<const float*>(sh_o[i])[tid];
        store_f(static_cast<T*>(p.out) + d.b * p.o_b + (kh * group + ht * rows_tile + row) * p.o_h + tid,
                L > 0.0f ? v / L : (L == 0.0f ? 0.0f : L));
    }
}

template <typename W, int kD>
cudaError_t launch_rows(PagedAttnParams p, cudaStream_t s) {
    constexpr int kSmem = kWarps * kStages * 2 * kStepBytes + (4 * W::kRows * kD + W::kQFloats) * static_cast<int>(sizeof(float));
    static_assert(kSmem + sizeof(Shared) <= 232448, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<W, kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(sms, kMaxCtas);
    // Sequences of kWholeBlocks blocks at most are not worth the second kernel: a CTA takes longer over a unit by less
    // than the join costs (64 x 300, 32 / 8 heads of 128: 31 against 34 us; one of 500, 16 / 4 heads of 64: 10.8
    // against 13.0 us with the launches). The lengths are on the device, so the host goes by what the table has room for:
    // the same sequences behind a wider table take the two launches.
    constexpr int kBlock = Step<typename W::T, kD>::kKeys * kWarps;
    p.whole = static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d <= kWholeBlocks * kBlock;
    const int64_t units = static_cast<int64_t>(p.B) * p.h_kv * ((p.h / p.h_kv + W::kRows - 1) / W::kRows);
    p.direct = p.whole && units <= ctas;
    if (p.whole) {
        return launch_pdl(paged_attn_kernel<W, kD>, dim3(static_cast<unsigned>(std::min<int64_t>(units, ctas))), dim3(kThreads),
                          kSmem, s, p);
    }
    if ((e = launch_pdl(paged_attn_kernel<W, kD>, dim3(ctas), dim3(kThreads), kSmem, s, p)) != cudaSuccess) return e;
    const int rows = std::min(p.h / p.h_kv, W::kRows);
    return launch_pdl(paged_join_kernel<typename W::T, kD>, dim3(ctas, rows), dim3(kJoinThreads), 0, s, p, static_cast<int>(W::kRows));
}

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
    const size_t slot = (2 * kMaxRows + kMaxRows * static_cast<size_t>(d)) * sizeof(float);
    return (kMaxCtas * 2 * slot + kMaxCtas * sizeof(JoinDesc) + 255) / 256 * 256;
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, bool bf16, cudaStream_t s) {
    return p.d == 64 ? launch_d<64>(p, bf16, s) : launch_d<128>(p, bf16, s);
}

}  // namespace mha
