// rotary.cu -- rotary positions of queries and keys, and the append of new keys and values to
// a paged cache on the same pass.
//
// Pair (x_0, x_1) of a token at position t turns by t * inv_freq[i]. The angle is formed in half
// turns as an unevaluated sum of two floats (error-free product by fused multiply-add, after
// Dekker): t * f in one float is off by up to 2^-25 of its size, 0.03 rad at t = 10^6. Whole turns
// are removed exactly before the sum is rounded, so cos and sin are good to 2^-22 up to positions of 2^24; beyond,
// the low part's own roundings (2^-46 of the angle) show: 2^-21 at 2^26, 2^-17.5 at 2^29.
//
// HBM-bound: every element is read once and written once (keys twice where k_out is asked for). Measured, 4 x 8192
// tokens appended in bf16: 32 + 8 heads of 128, half of each turned, 872 MB: 134 us, 6.5 TB/s (0.96 of measured copy
// bandwidth); 16 + 16 heads of 64: 76 us (0.91); 3 x 2501 tokens of 16 + 16 fp32 heads of 64, no cache: 22.7 us (0.80,
// start and end included).
#include <algorithm>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx_serve.cuh"
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

// kN elements of a head in one access of kN * sizeof(T) bytes.
template <int kBytes>
struct RawOf;
template <>
struct RawOf<2> { using Type = uint16_t; };
template <>
struct RawOf<4> { using Type = uint32_t; };
template <>
struct RawOf<8> { using Type = uint2; };
template <>
struct RawOf<16> { using Type = uint4; };
template <typename T, int kN>
union Chunk {
    typename RawOf<kN * sizeof(T)>::Type raw;
    T e[kN];
    __device__ __forceinline__ Chunk() {}
};

// A row is one head of one token. Its items, one a thread, are the pairs of chunks that turn together (half
// layout: chunk c and the one rot / 2 further; interleaved: two neighbours), then pairs of neighbouring chunks that
// pass unchanged. A thread has the same item in kRows rows, so what depends on the item is computed once; the rows'
// chunks are loaded before the tokens' cos and sin are computed and the pages looked up, so all three latencies
// overlap. A CTA takes rows of queries, of keys or of values only. (With a CTA a token the time went to starting
// CTAs: 96 us for 40 us of traffic at 32768 tokens of 16 + 16 heads of 64; with one list of items for all of a
// token's heads it went to index arithmetic.)
constexpr int kRows = 4;

struct TokenInfo {
    int b, t;           // t < 0: the token does not exist
    int pos, at;        // for the angles, in the cache
    int64_t slot;       // elements, or -1
};

// kStaged: the half layout where no wide chunk's partner is a chunk (rot / 2 odd, say). A thread moves one chunk of a row,
// and the pairs turn in shared memory, one a thread at a time (6 x 585 tokens of 40 + 5 bf16 heads of 64, 14 features turned:
// 27.6 us with an element an access, 16.6 us so; 4 x 8192 of 32 + 8 heads of 128, 126 turned: 447 and 224 us). Chunks of four
// bf16 elements that pair up are as fast as that or faster.
struct RowPlan {
    FastDiv q, k;           // heads
    FastDiv half;           // kStaged: rot / 2
    int items, turn;        // of a row; of those, the ones that turn
    int rows;               // rows of the CTA at a time: threads / items
    int per_cta;            // rows of a CTA: up to kRows * rows
    int tokens;             // most tokens that such rows touch
    int stage_at;           // kStaged: offset of the rows in shared memory
    int ctas_q, ctas_k;     // then the values'
    int64_t total;          // B * T
};

template <typename T, int kN, bool kStaged>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p, const RowPlan plan) {
    using C = Chunk<T, kN>;
    using Raw = decltype(C::raw);
    extern __shared__ __align__(16) uint8_t smem[];
    const int half = p.rot / 2;
    TokenInfo* info = reinterpret_cast<TokenInfo*>(smem);
    float2* turns = reinterpret_cast<float2*>(info + plan.tokens);     // [tokens][half]
    T* stage = reinterpret_cast<T*>(smem + plan.stage_at);              // kStaged: [rows][d]
    pdl_trigger();
    pdl_wait();
    const int job = static_cast<int>(blockIdx.x) < plan.ctas_q ? 0 : static_cast<int>(blockIdx.x) < plan.ctas_q + plan.ctas_k ? 1 : 2;
    const int block = blockIdx.x - (job == 0 ? 0 : job == 1 ? plan.ctas_q : plan.ctas_q + plan.ctas_k);
    const FastDiv heads = job == 0 ? plan.q : plan.k;
    const Strided in = job == 0 ? p.q : job == 1 ? p.k : p.v;
    const Strided out = job == 0 ? p.q_out : p.k_out;
    const int64_t row0 = static_cast<int64_t>(block) * plan.per_cta;
    const int64_t token0 = row0 / heads.d;
    const int skip = static_cast<int>(row0 - token0 * heads.d);       // rows of token0 that an earlier CTA takes
    const int rows = static_cast<int>(min(static_cast<int64_t>(plan.per_cta), plan.total * heads.d - row0));
    const int here = heads.div(skip + rows - 1) + 1;                   // tokens
    for (int i = threadIdx.x; i < here; i += kThreads) {
        const int n = static_cast<int>(token0) + i;
        TokenInfo x;
        x.b = p.by_t.div(n);
        x.t = n - x.b * p.T;
        x.at = (p.start != nullptr ? p.start[x.b] : 0) + x.t;
        x.pos = p.positions != nullptr ? p.positions[n] : x.at;
        if (p.new_lens != nullptr && x.t >= p.new_lens[x.b]) x.t = -1;
        x.slot = -1;
        info[i] = x;
    }
    __syncthreads();

    const int r = threadIdx.x / plan.items, c = threadIdx.x - r * plan.items;
    int c0, c1;     // the item's elements
    bool turns_here = job != 2 && c < plan.turn;
    if (kStaged) {
        c0 = c * kN;
        c1 = p.d;
    } else if (job == 2) {
        c0 = c * 2 * kN;
        c1 = c0 + kN;
    } else if (c >= plan.turn) {
        c0 = p.rot + (c - plan.turn) * 2 * kN;
        c1 = c0 + kN;
    } else {
        c0 = p.interleaved ? c * 2 * kN : c * kN;
        c1 = c0 + (p.interleaved ? kN : half);
    }
    const bool one = c0 < p.d, two = c1 < p.d;
    C x0[kRows], x1[kRows];
    int tok[kRows], head[kRows];
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const int i = n * plan.rows + r;
        tok[n] = -1;
        if (r >= plan.rows || i >= rows || !one) continue;
        const int tk = heads.div(skip + i);
        const TokenInfo& x = info[tk];
        if (x.t < 0) continue;
        tok[n] = tk;
        head[n] = skip + i - tk * static_cast<int>(heads.d);
        const T* src = static_cast<const T*>(in.p) + x.b * in.b + x.t * in.l + head[n] * in.h;
        x0[n].raw = *reinterpret_cast<const Raw*>(src + c0);
        if (two) x1[n].raw = *reinterpret_cast<const Raw*>(src + c1);
    }
    if constexpr (kStaged) {
#pragma unroll
        for (int n = 0; n < kRows; ++n)
            if (tok[n] >= 0 && turns_here) *reinterpret_cast<Raw*>(stage + (n * plan.rows + r) * p.d + c0) = x0[n].raw;
    }
    if (job != 2) {
        for (int i = threadIdx.x; i < here * half; i += kThreads) {
            const int tk = i / half;
            if (info[tk].t < 0) continue;
            const float2 cs = turn_of(info[tk].pos, p.inv_freq[i - tk * half]);
            turns[i] = make_float2(cs.x * p.scale, cs.y * p.scale);
        }
    }
    T* const pages = static_cast<T*>(job == 0 ? nullptr : job == 1 ? p.cache.k : p.cache.v);
    if (pages != nullptr) {
        for (int i = threadIdx.x; i < here; i += kThreads) {
            if (info[i].t < 0) continue;
            const int at = info[i].at;
            const int n = at >= 0 ? p.cache.page.div(at) : -1;
            int page = -1;
            if (n >= 0 && n < p.cache.max_pages) page = p.cache.table[info[i].b * p.cache.table_stride + n];
            if (page >= 0 && page < p.cache.n_pages)
                info[i].slot = page * p.cache.page_stride + (at - n * static_cast<int>(p.cache.page.d)) * p.cache.slot_stride;
            else
                atomicCAS(p.status, 0, 0x501);   // the token has no slot: it is not appended
        }
    }
    __syncthreads();
    if (kStaged && job != 2) {
        for (int i = threadIdx.x; i < rows * half; i += kThreads) {
            const int row = plan.half.div(i), e = i - row * half, tk = heads.div(skip + row);
            if (info[tk].t < 0) continue;
            T* x = stage + row * p.d + e;
            const float2 a = turns[tk * half + e];
            const float u = load_f(x), v = load_f(x + half);
            store_f(x, fmaf(u, a.x, -(v * a.y)));
            store_f(x + half, fmaf(v, a.x, u * a.y));
        }
        __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        if (tok[n] < 0) continue;
        const TokenInfo& x = info[tok[n]];
        if (turns_here) {
            const float2* cs = turns + tok[n] * half;
            if constexpr (kStaged) {
                x0[n].raw = *reinterpret_cast<const Raw*>(stage + (n * plan.rows + r) * p.d + c0);
            } else if (kN > 1 && p.interleaved) {
#pragma unroll
                for (int j = 0; j < 2 * kN; j += 2) {
                    C& y = j < kN ? x0[n] : x1[n];
                    if (c0 + j >= p.rot) break;
                    const float2 a = cs[(c0 + j) / 2];
                    const float u = load_f(&y.e[j % kN]), v = load_f(&y.e[j % kN + 1]);
                    store_f(&y.e[j % kN], fmaf(u, a.x, -(v * a.y)));
                    store_f(&y.e[j % kN + 1], fmaf(v, a.x, u * a.y));
                }
            } else {
                float2 a[kN];
                const float2* from = cs + (p.interleaved ? c0 >> 1 : c0);
#pragma unroll
                for (int j = 0; j < kN; ++j) a[j] = from[j];
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const float u = load_f(&x0[n].e[j]), v = load_f(&x1[n].e[j]);
                    store_f(&x0[n].e[j], fmaf(u, a[j].x, -(v * a[j].y)));
                    store_f(&x1[n].e[j], fmaf(v, a[j].x, u * a[j].y));
                }
            }
        }
        if (job != 2 && out.p != nullptr) {
            T* y = static_cast<T*>(out.p) + x.b * out.b + x.t * out.l + head[n] * out.h;
            *reinterpret_cast<Raw*>(y + c0) = x0[n].raw;
            if (two) *reinterpret_cast<Raw*>(y + c1) = x1[n].raw;
        }
        if (pages != nullptr && x.slot >= 0) {
            T* z = pages + x.slot + head[n] * p.cache.head_stride;
            *reinterpret_cast<Raw*>(z + c0) = x0[n].raw;
            if (two) *reinterpret_cast<Raw*>(z + c1) = x1[n].raw;
        }
    }
}

// Whether every chunk of n elements is aligned and, unless they go through shared memory, every pair of chunks turns together.
template <typename T>
bool chunks_fit(const RotaryParams& p, int n, bool staged = false) {
    const size_t bytes = n * sizeof(T);
    auto tensor = [&](const Strided& x) {
        return x.p == nullptr || (reinterpret_cast<uintptr_t>(x.p) % bytes == 0 && x.b % n == 0 && x.l % n == 0 && x.h % n == 0);
    };
    return p.d % n == 0 && (staged || p.interleaved || (p.rot % n == 0 && p.rot / 2 % n == 0)) && tensor(p.q) && tensor(p.q_out) &&
           tensor(p.k) && tensor(p.k_out) && tensor(p.v) &&
           (p.cache.k == nullptr ||
            (reinterpret_cast<uintptr_t>(p.cache.k) % bytes == 0 && reinterpret_cast<uintptr_t>(p.cache.v) % bytes == 0 &&
             p.cache.page_stride % n == 0 && p.cache.slot_stride % n == 0 && p.cache.head_stride % n == 0));
}

template <typename T, int kN, bool kStaged = false>
cudaError_t launch_n(const RotaryParams& p, cudaStream_t s) {
    constexpr int kPair = 2 * kN;
    RowPlan plan;
    // interleaved pairs of several elements lie inside a chunk: the border may fall inside an item there, and all items
    // are of the kind that turns
    const bool inside = p.interleaved && kN > 1;
    plan.turn = inside ? (p.d + kPair - 1) / kPair : (p.rot + kPair - 1) / kPair;
    plan.items = plan.turn + (inside ? 0 : (p.d - p.rot + kPair - 1) / kPair);
    if (kStaged) {
        plan.half = fast_div(static_cast<uint32_t>(p.rot / 2));
        plan.turn = (p.rot + kN - 1) / kN;
        plan.items = p.d / kN;
    }
    plan.rows = kThreads / plan.items;
    plan.total = static_cast<int64_t>(p.B) * p.T;
    const int nq = p.q.p != nullptr ? p.h : 0, nk = p.k.p != nullptr ? p.h_kv : 0;
    plan.q = fast_div(static_cast<uint32_t>(std::max(nq, 1)));
    plan.k = fast_div(static_cast<uint32_t>(std::max(nk, 1)));
    // the tokens of a CTA's rows (of the fewest heads) have their cos and sin in 32 KB
    const int fewest = nk > 0 && (nq == 0 || nk < nq) ? nk : nq;
    const size_t token_bytes = sizeof(TokenInfo) + sizeof(float2) * (p.rot / 2);
    const int64_t most = std::max<int64_t>(1, static_cast<int64_t>((32 << 10) / token_bytes) - 1) * fewest;
    const int64_t all_rows = plan.total * (nq + (p.v.p != nullptr ? 2 : 1) * nk);
    // kRows rows a thread where that leaves two CTAs on each of 152 SMs (equal waves of smaller CTAs were no faster)
    const int64_t spread = (all_rows + 303) / 304;
    plan.per_cta = static_cast<int>(std::max<int64_t>(1, std::min({static_cast<int64_t>(kRows) * plan.rows, most, spread})));
    plan.tokens = (plan.per_cta + fewest - 1) / fewest + 1;
    auto ctas = [&](int n) { return static_cast<int>((plan.total * n + plan.per_cta - 1) / plan.per_cta); };
    plan.ctas_q = ctas(nq);
    plan.ctas_k = ctas(nk);
    const int64_t grid = static_cast<int64_t>(plan.ctas_q) + plan.ctas_k + (p.v.p != nullptr ? ctas(nk) : 0);
    // tokens' part: at most 32 KB; the rows: kRows * kThreads chunks of 16 bytes at most
    plan.stage_at = static_cast<int>((plan.tokens * token_bytes + 15) / 16 * 16);
    const size_t smem = plan.stage_at + (kStaged ? kRows * plan.rows * p.d * sizeof(T) : 0);
    return launch_pdl(rotary_kernel<T, kN, kStaged>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, s, p, plan);
}

template <typename T>
cudaError_t launch_t(RotaryParams p, cudaStream_t s) {
    p.by_t = fast_div(static_cast<uint32_t>(p.T));
    constexpr int kWide = 16 / sizeof(T);
    if (chunks_fit<T>(p, kWide)) return launch_n<T, kWide>(p, s);
    if constexpr (kWide == 8)
        if (chunks_fit<T>(p, 4)) return launch_n<T, 4>(p, s);
    if (!p.interleaved && p.rot > 0 && chunks_fit<T>(p, kWide, true)) return launch_n<T, kWide, true>(p, s);
    if (chunks_fit<T>(p, 2)) return launch_n<T, 2>(p, s);
    return launch_n<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace mha
