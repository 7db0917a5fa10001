// paged_attn.cu -- attention of one new token a sequence over a paged key/value cache.
//
//   s_j = cap tanh(scale q.k_j / cap) - slope (n - 1 - j),  o = sum_j softmax_j(s) v_j,  j < n
// in one pass with a running maximum m and sum l. n = 0 gives zeros.
//
// HBM-bound: K and V of every cached position are read once, 4 d_k bytes a position and key head in
// bf16, for 4 d_k flop a query head. The heads that share a key head are the rows of one matrix
// product (16 rows in bf16, mma.sync: the product takes a sixth of the load's time at 8 heads, and
// CUDA cores could not keep up from 4 heads on), so the cache is read once for all of them.
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
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kStepBytes = 4096;        // of keys, and of values, in one step of a warp
constexpr int kMaxCtas = 192;           // slots of the workspace
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;           // log2 units the maximum may grow before o and l are rescaled

template <typename T, int kD>
struct Step {
    static constexpr int kRow = kD * static_cast<int>(sizeof(T));   // bytes of a key
    static constexpr int kKeys = kStepBytes / kRow;
    static constexpr int kChunks = kRow / 16;
};
constexpr int kRowsBf16 = 16;
constexpr int kMaxRows = 16;

struct JoinDesc {
    int c0, c1;         // CTAs whose pieces make up the unit; c1 < c0: nothing to join
    int b, unit;
    int first_slot;     // slot of c0's piece (every later CTA's is 0)
};

// One piece in the workspace: m[16], l[16], o[16][kD]
template <int kD>
__host__ __device__ constexpr int slot_floats() { return 2 * kMaxRows + kMaxRows * kD; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    // src-size 0 writes zeros and reads nothing
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
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

// cap log2(e) tanh(x): 1 - 2 / (1 + e^2x), good to 2^-22 of the cap
__device__ __forceinline__ float cap_log2(float x, float top) {
    return fmaf(-2.0f * top, rcp_approx(1.0f + ex2_approx(x * (2.0f * kLog2e))), top);
}

// A score in log2 units from q.k: capped, minus the distance bias.
struct ScoreForm {
    float in, top;     // capped: s = cap_log2(dot * in, top), else dot * in
    bool capped;
    __device__ __forceinline__ float operator()(float dot, float slope, float away) const {
        const float s = capped ? cap_log2(dot * in, top) : dot * in;
        return fmaf(-slope, away, s);
    }
};

// ------------------------------------------------------------ a warp's rows: bf16, matrix instructions
template <int kD>
struct WarpBf16 {
    using T = __nv_bfloat16;
    static constexpr int kRows = kRowsBf16;
    static constexpr int kKeys = Step<T, kD>::kKeys;
    uint32_t q[kD / 16][4];
    float o[kD / 8][4];
    float m[2], l[2], slope[2];     // rows lane / 4 and lane / 4 + 8; l is this lane's share

    static __device__ __forceinline__ int swizzle(int row) { return row & 7; }

    __device__ __forceinline__ void start(const PagedAttnParams& p, int b, int head0, int rows, int lane) {
        const T* base = static_cast<const T*>(p.q) + b * p.q_b + head0 * p.q_h;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
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
                    q[k][2 * hf + r] = *reinterpret_cast<uint32_t*>(&v);
                }
            }
            slope[r] = p.slopes != nullptr && row < rows ? p.slopes[head0 + row] * kLog2e : 0.0f;
            m[r] = -CUDART_INF_F;
            l[r] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kD / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    }

    // keys key0 .. key0 + kKeys - 1 in shared memory at k, v; live: bit i: key0 + i counts
    __device__ __forceinline__ void step(uint32_t k, uint32_t v, int key0, uint32_t live, int n, const ScoreForm& form,
                                         int rows, int lane) {
        constexpr int kRow = Step<T, kD>::kRow;
        float s[kKeys / 8][4];
        const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
        for (int t = 0; t < kKeys / 8; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = 0.0f;
        }
#pragma unroll
        for (int kp = 0; kp < kD / 32; ++kp) {
#pragma unroll
            for (int t = 0; t < kKeys / 8; ++t) {
                uint32_t f[4];
                ldsm4(f, k + (t * 8 + r8) * kRow + (((kp * 4 + mi) ^ r8) << 4));
                mma16816(s[t], q[2 * kp], f[0], f[1]);
                mma16816(s[t], q[2 * kp + 1], f[2], f[3]);
            }
        }
        const bool both = rows > 8;
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int t = 0; t < kKeys / 8; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = t * 8 + 2 * (lane & 3) + e;
                const bool ok = (live >> i) & 1u;
                const float away = static_cast<float>(n - 1 - key0 - i);
                s[t][e] = ok ? form(s[t][e], slope[0], away) : -CUDART_INF_F;
                top[0] = fmaxf(top[0], s[t][e]);
                if (both) {
                    s[t][2 + e] = ok ? form(s[t][2 + e], slope[1], away) : -CUDART_INF_F;
                    top[1] = fmaxf(top[1], s[t][2 + e]);
                }
            }
        }
        float alpha[2] = {1.0f, 1.0f}, ref[2];
        bool grew = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            if (top[r] > m[r] + kGrow || m[r] == -CUDART_INF_F) {   // the first keys set the maximum
                const float to = fmaxf(top[r], m[r]);
                if (m[r] != -CUDART_INF_F) {
                    alpha[r] = ex2_approx(m[r] - to);
                    l[r] *= alpha[r];
                    grew = true;
                }
                m[r] = to;
            }
            ref[r] = m[r] == -CUDART_INF_F ? 0.0f : m[r];
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int i = 0; i < kD / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];
        }
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks) {
            uint32_t a[4];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float* c = s[2 * ks + hf];
                const float p0 = ex2_approx(c[0] - ref[0]), p1 = ex2_approx(c[1] - ref[0]);
                l[0] += p0 + p1;
                a[2 * hf] = pack_bf16x2(p0, p1);      // weights rounded to the values' type; l takes them unrounded
                a[2 * hf + 1] = 0u;
                if (both) {
                    const float p2 = ex2_approx(c[2] - ref[1]), p3 = ex2_approx(c[3] - ref[1]);
                    l[1] += p2 + p3;
                    a[2 * hf + 1] = pack_bf16x2(p2, p3);
                }
            }
#pragma unroll
            for (int np = 0; np < kD / 16; ++np) {
                uint32_t f[4];
                ldsm4t(f, v + (ks * 16 + (mi & 1) * 8 + r8) * kRow + (((np * 2 + (mi >> 1)) ^ r8) << 4));
                mma16816(o[2 * np], a, f[0], f[1]);
                mma16816(o[2 * np + 1], a, f[2], f[3]);
            }
        }
    }

    // the row maxima and sums to shared memory
    __device__ __forceinline__ void put_stats(float* sm_m, float* sm_l, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if ((lane & 3) == 0) {
                sm_m[(lane >> 2) + 8 * r] = m[r];
                sm_l[(lane >> 2) + 8 * r] = l[r];
            }
        }
    }
    // o scaled by f[row] (put) or added onto what is there (add = true), rows of kD floats
    __device__ __forceinline__ void put(float* buf, const float* f, bool add, int rows, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
            if (row >= rows) continue;
            const float fr = f[row];
#pragma unroll
            for (int i = 0; i < kD / 8; ++i) {
                float2* y = reinterpret_cast<float2*>(buf + row * kD + 8 * i + 2 * (lane & 3));
                float2 x = make_float2(o[i][2 * r] * fr, o[i][2 * r + 1] * fr);
                if (add) {
                    const float2 z = *y;
                    x.x += z.x;
                    x.y += z.y;
                }
                *y = x;
            }
        }
    }
};

// ------------------------------------------------------------ a warp's rows: fp32, CUDA cores
template <int kD, int kR>
struct WarpF32 {
    using T = float;
    static constexpr int kRows = kR;
    static constexpr int kKeys = Step<T, kD>::kKeys;      // 8 or 16
    static constexpr int kLanes = 32 / kKeys;             // lanes that share a key's dot product: 4 or 2
    static constexpr int kDims = kD / kLanes;             // features a lane multiplies: 32
    static constexpr int kOwn = kD / 32;                  // features of o a lane keeps
    float o[kR][kOwn];
    float m[kR], l[kR];                                   // l is this lane's share
    const float* q;                                       // the unit's query rows, or zeros
    int64_t q_h;
    const float* slopes;
    int rows_;

    // two (or four) keys of a quarter-warp's 16-byte reads land in different 64-byte (32-byte) parts
    static __device__ __forceinline__ int swizzle(int row) { return kLanes == 4 ? (row & 1) << 2 : (row & 3) << 1; }

    __device__ __forceinline__ void start(const PagedAttnParams& p, int b, int head0, int rows, int) {
        q = static_cast<const float*>(p.q) + b * p.q_b + head0 * p.q_h;
        q_h = p.q_h;
        slopes = p.slopes != nullptr ? p.slopes + head0 : nullptr;
        rows_ = rows;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            m[r] = -CUDART_INF_F;
            l[r] = 0.0f;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) o[r][e] = 0.0f;
        }
    }

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
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (r >= rows) break;
            const float* x = q + r * q_h + part * 4;
            float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
            for (int i = 0; i < kDims / 4; ++i) {
                const float* xi = x + i * kLanes * 4;      // the same few lines for every key: L1
                d0 = fmaf(kv[i].x, xi[0], d0);
                d1 = fmaf(kv[i].y, xi[1], d1);
                d0 = fmaf(kv[i].z, xi[2], d0);
                d1 = fmaf(kv[i].w, xi[3], d1);
            }
            float s = d0 + d1;
#pragma unroll
            for (int w = 1; w < kLanes; w <<= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
            s = ok ? form(s, slopes != nullptr ? slopes[r] * kLog2e : 0.0f, away) : -CUDART_INF_F;
            float top = s;
#pragma unroll
            for (int w = kLanes; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float to = fmaxf(top, m[r]);
            if (to > m[r]) {      // the same in every lane
                const float alpha = m[r] == -CUDART_INF_F ? 0.0f : ex2_approx(m[r] - to);
                l[r] *= alpha;
#pragma unroll
                for (int e = 0; e < kOwn; ++e) o[r][e] *= alpha;
                m[r] = to;
            }
            const float w = ex2_approx(s - (m[r] == -CUDART_INF_F ? 0.0f : m[r]));
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

struct Shared {
    float m[kWarps][kMaxRows], l[kWarps][kMaxRows], f[kWarps][kMaxRows];
    long long scan[kWarps];
    long long before;
    int found_b;
};

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

    // ---- total number of blocks, and the sequences that have none
    long long mine = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int n = lens.len(b);
        if (p.kv_lens[b] > room) atomicCAS(p.status, 0, 0x501);
        mine += lens.blocks(n);
    }
    mine = warp_sum64(mine);
    if (lane == 0) sh.scan[warp] = mine;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) total += sh.scan[w];
    total *= units;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (lens.len(b) > 0) continue;
        for (int i = threadIdx.x; i < p.h * kD; i += kThreads)
            store_f(static_cast<T*>(p.out) + b * p.o_b + (i / kD) * p.o_h + i % kD, 0.0f);
    }
    const int c = blockIdx.x;
    const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    if (c >= ctas) {
        if (threadIdx.x == 0) join[c].c1 = -1, join[c].c0 = 0;
        return;
    }
    // CTA c takes blocks [c total / ctas, (c + 1) total / ctas); block t belongs to the last CTA that starts at or before it
    const long long t0 = c * total / ctas, t1 = (c + 1) * total / ctas;
    auto owner = [&](long long t) { return static_cast<int>(((t + 1) * ctas + total - 1) / total - 1); };

    // ---- the sequence that t0 falls into
    long long acc = 0;   // blocks (of one unit) before sequence b0
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const long long v = b < p.B ? lens.blocks(lens.len(b)) : 0;
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long other = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += other;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) inc += sh.scan[w];
            all += sh.scan[w];
        }
        const long long lo = (acc + inc - v) * units, hi = (acc + inc) * units;
        if (t0 >= lo && t0 < hi) {
            sh.found_b = b;
            sh.before = lo;
        }
        acc += all;
        if (t0 < acc * units) break;
    }
    __syncthreads();
    Cursor at;      // the block that is computed
    at.b = sh.found_b;
    at.n = lens.len(at.b);
    at.nblk = lens.blocks(at.n);
    const long long rem = t0 - sh.before;
    at.unit = static_cast<int>(rem / at.nblk);
    at.blk = static_cast<int>(rem - static_cast<long long>(at.unit) * at.nblk);
    if (threadIdx.x == 0) {
        JoinDesc d{0, -1, 0, 0, 0};
        const long long u0 = t0 - at.blk;       // first block of the unit
        if (at.blk > 0 && owner(u0) == c - 1) {  // the first of the CTAs that continue it describes the join
            d.c0 = c - 1;
            d.c1 = owner(u0 + at.nblk - 1);
            d.b = at.b;
            d.unit = at.unit;
            d.first_slot = (c - 1) * total / ctas == u0 ? 0 : 1;
        }
        join[c] = d;
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

    // ---- loads: lane i looks up the page of key i of the step one step ahead of its loads
    Cursor ahead = at;
    long long t_ahead = t0;
    int page = -1, slot = 0, kvh = 0;
    bool inside = false;
    const uint32_t stage0 = smem_u32(smem) + warp * (kStages * 2 * kStepBytes);
    auto look_up = [&]() {
        inside = false;
        if (t_ahead < t1) {
            const int key = (ahead.blk * kWarps + warp) * kKeys + lane;
            kvh = ahead.unit / head_tiles;
            if (lane < kKeys && key < ahead.n) {
                const int i = p.cache.page.div(key);
                slot = key - i * static_cast<int>(p.cache.page.d);
                page = p.cache.table[ahead.b * p.cache.table_stride + i];
                inside = true;
            }
            advance(ahead);
        }
        ++t_ahead;
    };
    auto issue = [&](int stage) -> uint32_t {
        const bool ok = inside && page >= 0 && page < p.cache.n_pages;
        if (inside && !ok) atomicCAS(p.status, 0, 0x501);
        const long long off =
            ok ? page * p.cache.page_stride + slot * p.cache.slot_stride + kvh * p.cache.head_stride : 0;
        const uint32_t live = __ballot_sync(0xffffffffu, ok);
        if (live != 0) {
            const uint32_t k = stage0 + stage * (2 * kStepBytes);
#pragma unroll
            for (int i = 0; i < kStepBytes / 512; ++i) {
                const int id = i * 32 + lane;
                const int row = id / S::kChunks, col = id % S::kChunks;
                const long long ro = __shfl_sync(0xffffffffu, off, row);
                const bool on = (live >> row) & 1u;
                const uint32_t dst = k + row * S::kRow + ((col ^ W::swizzle(row)) << 4);
                const long long e = ro + col * (16 / static_cast<int>(sizeof(T)));
                cp_async16(dst, static_cast<const T*>(p.cache.k) + e, on);
                cp_async16(dst + kStepBytes, static_cast<const T*>(p.cache.v) + e, on);
            }
        }
        cp_commit();
        return live;
    };
    uint32_t live[kStages];
    look_up();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        live[s] = issue(s);
        look_up();
    }

    const ScoreForm form{p.cap > 0.0f ? p.scale / p.cap : p.scale * kLog2e, p.cap * kLog2e, p.cap > 0.0f};
    float* buf = reinterpret_cast<float*>(smem + kWarps * kStages * 2 * kStepBytes);   // 4 x [rows][kD]
    W w;
    bool fresh = true, first_piece = true;
    int piece_blk = at.blk, stage = 0, rows = 0, head0 = 0;
    for (long long t = t0; t < t1; ++t) {
        if (fresh) {
            const int kh = at.unit / head_tiles, ht = at.unit - kh * head_tiles;
            rows = min(group - ht * W::kRows, W::kRows);
            head0 = kh * group + ht * W::kRows;
            w.start(p, at.b, head0, rows, lane);
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

// Joins the pieces of a unit that several CTAs share: block (c, row), threads (group, feature).
template <typename T, int kD>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int rows_tile) {
    constexpr int kSlot = slot_floats<kD>();
    constexpr int kGroups = 256 / kD;
    __shared__ float sh_m[8], sh_o[kGroups][kD], sh_l[kGroups];
    pdl_trigger();
    pdl_wait();
    const JoinDesc d = reinterpret_cast<const JoinDesc*>(p.partial + static_cast<int64_t>(kMaxCtas) * 2 * kSlot)[blockIdx.x];
    if (d.c1 < d.c0) return;
    const int group = p.h / p.h_kv;
    const int head_tiles = (group + rows_tile - 1) / rows_tile;
    const int kh = d.unit / head_tiles, ht = d.unit - kh * head_tiles;
    const int row = blockIdx.y;
    if (row >= min(group - ht * rows_tile, rows_tile)) return;
    auto slot = [&](int c) { return p.partial + (static_cast<int64_t>(c) * 2 + (c == d.c0 ? d.first_slot : 0)) * kSlot; };
    float M = -CUDART_INF_F;
    for (int c = d.c0 + threadIdx.x; c <= d.c1; c += 256) M = fmaxf(M, slot(c)[row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if ((threadIdx.x & 31) == 0) sh_m[threadIdx.x >> 5] = M;
    __syncthreads();
    for (int i = 0; i < 8; ++i) M = fmaxf(M, sh_m[i]);
    const int g = threadIdx.x / kD, x = threadIdx.x % kD;
    float L = 0.0f, a = 0.0f;
#pragma unroll 8
    for (int c = d.c0 + g; c <= d.c1; c += kGroups) {
        const float* s = slot(c);
        const float mc = s[row];
        const float f = mc == -CUDART_INF_F ? 0.0f : ex2_approx(mc - M);
        L = fmaf(s[kMaxRows + row], f, L);
        a = fmaf(s[2 * kMaxRows + row * kD + x], f, a);
    }
    sh_o[g][x] = a;
    if (x == 0) sh_l[g] = L;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < kGroups; ++i) {
            a += sh_o[i][x];
            L += sh_l[i];
        }
        store_f(static_cast<T*>(p.out) + d.b * p.o_b + (kh * group + ht * rows_tile + row) * p.o_h + x,
                L > 0.0f ? a / L : (L == 0.0f ? 0.0f : L));
    }
}

template <typename W, int kD>
cudaError_t launch_rows(const PagedAttnParams& p, cudaStream_t s) {
    constexpr int kSmem = kWarps * kStages * 2 * kStepBytes + 4 * W::kRows * kD * static_cast<int>(sizeof(float));
    static_assert(kSmem + sizeof(Shared) <= 232448, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<W, kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(sms, kMaxCtas);
    if ((e = launch_pdl(paged_attn_kernel<W, kD>, dim3(ctas), dim3(kThreads), kSmem, s, p)) != cudaSuccess) return e;
    const int rows = std::min(p.h / p.h_kv, W::kRows);
    return launch_pdl(paged_join_kernel<typename W::T, kD>, dim3(ctas, rows), dim3(256), 0, s, p, static_cast<int>(W::kRows));
}

template <int kD>
cudaError_t launch_d(const PagedAttnParams& p, bool bf16, cudaStream_t s) {
    if (bf16) return launch_rows<WarpBf16<kD>, kD>(p, s);
    const int group = p.h / p.h_kv;
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
