// paged_line.cuh -- the way of attention of one new token a sequence through a paged cache: which keys a CTA takes, their
// loads, and the join of the parts. What a warp does with a step of keys is the policy W of its kernel (paged_attn.cu: bf16
// and fp32 caches; coded_attn.cuh: caches in 8 bits).
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
#pragma once

#include <algorithm>

#include <math_constants.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx_serve.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kSlotsPerSm = 192;        // slots of the workspace for a CTA an SM
constexpr int kMaxRows = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;           // log2 units the maximum may grow before o and l are rescaled

// One step of a warp: kKeys keys, their kBytes bytes of keys and as many of values, elements of kElem bytes. kScales: the
// scales of kScales neighbouring key heads besides, [keys / values][head][key % 8][key / 8]. Up to 32 keys: lane i looks up key i.
// A CTA has kWarps warps, each with kStages steps in shared memory; kPerSm of them run on an SM.
// A unit's end costs as much as kTail blocks.
template <int kRow_, int kElem_, int kKeys_, int kStages_, int kScales_, int kWarps_, int kTail_, int kPerSm_, int kWhole_>
struct StepOf {
    static constexpr int kElem = kElem_, kKeys = kKeys_, kStages = kStages_, kScales = kScales_, kWarps = kWarps_, kTail = kTail_, kWhole = kWhole_, kPerSm = kPerSm_, kSlots = kPerSm * kSlotsPerSm;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRow = kRow_;                      // bytes of a key
    static constexpr int kBytes = kKeys * kRow;
    static constexpr int kChunks = kRow / 16;
    static constexpr int kStage = 2 * kBytes + 2 * 4 * kKeys * kScales;
    static_assert(kKeys <= 32 && kChunks <= 32 && kBytes % 512 == 0, "a step of a warp");
};

struct JoinDesc {
    int c0, c1;         // CTAs whose pieces make up the unit; c1 < c0: nothing to join
    int b, unit;
    int first_slot;     // slot of c0's piece (every later CTA's is 0)
};

// One piece in the workspace: m[16], l[16], o[16][kD]
template <int kD>
__host__ __device__ constexpr int slot_floats() { return 2 * kMaxRows + kMaxRows * kD; }

inline size_t line_workspace(int d, int per_sm) {
    const size_t slots = static_cast<size_t>(per_sm) * kSlotsPerSm;
    const size_t slot = (2 * kMaxRows + kMaxRows * static_cast<size_t>(d)) * sizeof(float);
    return (slots * 2 * slot + slots * sizeof(JoinDesc) + 255) / 256 * 256;
}

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

// ------------------------------------------------------------ the line of blocks
struct Cursor {
    int b, unit;        // unit of the sequence: key head * head tiles + head tile
    int blk, nblk;
    int n;              // the sequence's length
};

template <int kTail>
struct Lens {
    const int32_t* kv_lens;
    int64_t room;
    int block;          // keys of a block
    __device__ __forceinline__ int len(int b) const {
        const int n = max(kv_lens[b], 0);
        return static_cast<int>(min(static_cast<int64_t>(n), room));
    }
    __device__ __forceinline__ int blocks(int n) const { return n / block + (n % block != 0); }
    // of the line: a unit's blocks, and kTail for its end
    __device__ __forceinline__ int places(int n) const { return kTail == 0 ? blocks(n) : n > 0 ? blocks(n) + kTail : 0; }
};

struct Found {
    long long before;    // blocks before sequence b
    int b;
};

template <int kWarps>
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
__global__ void __launch_bounds__(W::Step::kThreads, W::Step::kPerSm) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    using T = typename W::T;
    using S = typename W::Step;
    constexpr int kKeys = S::kKeys;
    constexpr int kSlot = slot_floats<kD>(), kStages = S::kStages, kWarps = S::kWarps, kThreads = S::kThreads, kTail = S::kTail;
    constexpr bool kSided = S::kScales > 0;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared<kWarps> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = p.h / p.h_kv;
    const int head_tiles = (group + W::kRows - 1) / W::kRows;
    // kSided: the line is that of every p.side-th unit, p.side CTAs to a piece
    const int sides = kSided ? static_cast<int>(p.side.d) : 1;
    const int units = kSided ? p.side.div(p.h_kv * head_tiles) : p.h_kv * head_tiles;
    const int c = kSided ? p.side.div(blockIdx.x) : blockIdx.x, my_side = kSided ? static_cast<int>(blockIdx.x) - c * sides : 0;
    // positions stay below 2^31 with a block to spare
    const int64_t room = min(static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d, static_cast<int64_t>(0x7ffff000));
    const Lens<kTail> lens{p.kv_lens, room, kKeys * kWarps};
    JoinDesc* join = reinterpret_cast<JoinDesc*>(p.partial + static_cast<int64_t>(S::kSlots) * 2 * kSlot);
    pdl_trigger();
    pdl_wait();

    Cursor at;               // the block that is computed
    long long t0, t1;        // the CTA's places of the line
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
        // ---- total number of places, and the sequences that have none. Up to 32 sequences are summed by every warp for
        // itself, without a barrier before the first loads.
        const bool few = p.B <= 32;
        long long total = 0, inc = 0, v = 0;     // few: places (of one unit) up to and of sequence `lane`
        if (few) {
            if (lane < p.B) {
                v = lens.places(lens.len(lane));
                if (p.kv_lens[lane] > room) atomicCAS(p.status, 0, 0x501);
            }
            inc = warp_scan64(v, lane);
            total = __shfl_sync(0xffffffffu, inc, 31);
        } else {
            for (int b = threadIdx.x; b < p.B; b += kThreads) {
                if (p.kv_lens[b] > room) atomicCAS(p.status, 0, 0x501);
                v += lens.places(lens.len(b));
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
        const int ctas = static_cast<int>(min(static_cast<long long>(kSided ? p.side.div(gridDim.x) : gridDim.x), total));
        if (c >= ctas) {
            if (threadIdx.x == 0 && !p.whole) join[blockIdx.x] = JoinDesc{0, -1, 0, 0, 0};
            return;
        }
        // CTA c takes places [c total / ctas, (c + 1) total / ctas); place t belongs to the last CTA that starts at or before it
        const bool small = total < (1ll << 32) / S::kSlots;       // S::kSlots * total fits 32 bits: divisions a quarter as long
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
            long long acc = 0;   // places (of one unit) before sequence b0
            for (int b0 = 0; b0 < p.B; b0 += kThreads) {
                const int b = b0 + threadIdx.x;
                v = b < p.B ? lens.places(lens.len(b)) : 0;
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
            const int each = x.nblk + kTail;
            x.unit = small ? static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(each)) : static_cast<int>(rem / each);
            x.blk = static_cast<int>(rem - static_cast<long long>(x.unit) * each);
            return x;
        };
        at = cursor_at(t0, found[0]);
        if (p.whole) {
            // units are not split: a CTA takes those that start in its piece of the line
            if (t1 < total) {
                const Cursor e = cursor_at(t1, found[1]);
                if (e.blk > 0) t1 += e.nblk + kTail - e.blk;
            }
        } else if (threadIdx.x == 0) {
            JoinDesc d{0, -1, 0, 0, 0};
            const long long u0 = t0 - at.blk;       // the unit's first place
            if (at.blk > 0 && (kTail == 0 || at.blk < at.nblk) && owner(u0) == c - 1) {  // the first of the CTAs that continue it describes the join
                d.c0 = c - 1;
                d.c1 = owner(u0 + at.nblk - 1);
                d.b = at.b;
                d.unit = at.unit * sides + my_side;
                d.first_slot = start_of(c - 1) + kTail >= u0 ? 0 : 1;       // in the end of the unit before: nothing of that
            }
            join[blockIdx.x] = d;
        }
    }
    auto advance = [&](Cursor& x, long long& t) {
        ++t;
        if (++x.blk < x.nblk) return;
        t += kTail;
        x.blk = 0;
        if (++x.unit < units) return;
        x.unit = 0;
        do {
            if (++x.b >= p.B) { x.b = p.B; return; }   // past the last block: never followed
            x.n = lens.len(x.b);
            x.nblk = lens.blocks(x.n);
        } while (x.n == 0);
    };

    if ((kTail > 0 && at.blk >= at.nblk) || (p.whole && at.blk > 0)) {      // never where a CTA has a unit of its own
        t0 += at.nblk - 1 - at.blk;
        at.blk = at.nblk - 1;
        advance(at, t0);
    }

    // ---- loads: lane i looks up the page of key i of the step one step ahead of its loads
    Cursor ahead = at;
    long long t_ahead = t0;
    int page = -1, slot = 0, kvh = 0;
    bool inside = false;
    const uint32_t stage0 = smem_u32(smem) + warp * (kStages * S::kStage);
    // the lane's chunk of a row; of two key heads each has half of the row, and p.cache.head_stride is that of a pair
    constexpr int kOfHead = S::kChunks / (S::kScales == 2 ? 2 : 1);
    const char* k_lane = static_cast<const char*>(p.cache.k) + lane % kOfHead * 16 +
                         (lane % S::kChunks / kOfHead) * (p.cache.head_stride / 2) * S::kElem;
    const long long v_minus_k = static_cast<const char*>(p.cache.v) - static_cast<const char*>(p.cache.k);
    auto look_up = [&](bool first = false) {
        inside = false;
        if (t_ahead < t1) {
            const int key = (ahead.blk * kWarps + warp) * kKeys + lane;
            kvh = (ahead.unit * sides + my_side) / head_tiles;
            if (lane < kKeys && key < ahead.n) {
                const int i = p.cache.page.div(key);
                slot = key - i * static_cast<int>(p.cache.page.d);
                page = first && p.direct ? early : p.cache.table[ahead.b * p.cache.table_stride + i];
                inside = true;
            }
            advance(ahead, t_ahead);
        } else if (kTail == 0) {
            ++t_ahead;           // without tails it stays a step count ahead of the block that is computed, and needs no registers of its own
        }
    };
    auto issue = [&](int stage) -> uint32_t {
        const bool ok = inside && page >= 0 && page < p.cache.n_pages;
        if (inside && !ok) atomicCAS(p.status, 0, 0x501);
        const long long off = ok ? (page * p.cache.page_stride + slot * p.cache.slot_stride + kvh * p.cache.head_stride) *
                                       S::kElem : 0;
        const uint32_t live = __ballot_sync(0xffffffffu, ok);
        if (live != 0) {
            constexpr int kRowsPer = 32 / S::kChunks > 0 ? 32 / S::kChunks : 1;   // rows an instruction of the warp covers
            const int row0 = lane / S::kChunks, col = lane % S::kChunks;
            const uint32_t k = stage0 + stage * S::kStage + row0 * S::kRow;
#pragma unroll
            for (int i = 0; i < S::kBytes / 512; ++i) {
                const int row = i * kRowsPer + row0;
                const char* src = k_lane + __shfl_sync(0xffffffffu, off, row);
                const bool on = (live >> row) & 1u;
                const uint32_t dst = k + i * (kRowsPer * S::kRow) + ((col ^ W::swizzle(row)) << 4);
                cp_async16(dst, src, on);
                cp_async16(dst + S::kBytes, src + v_minus_k, on);
            }
            if constexpr (S::kScales > 0) {     // of the lane's key
                static_assert(S::kKeys == 32, "a key a lane");
                const int64_t at = ok ? static_cast<int64_t>(page) * p.page_scales + (p.scale_block.div(slot) * p.h_kv + kvh) * S::kScales : 0;
                const uint32_t to = stage0 + stage * S::kStage + 2 * S::kBytes + 16 * (lane & 7) + 4 * (lane >> 3);
#pragma unroll
                for (int i = 0; i < S::kScales; ++i) {
                    cp_async4(to + 128 * i, p.k_scales + at + i, ok);
                    cp_async4(to + 128 * (S::kScales + i), p.v_scales + at + i, ok);
                }
            }
        }
        cp_commit();
        return live;
    };
    W w;
    bool fresh = true, first_piece = true;
    int piece_blk = at.blk, stage = 0, rows = 0, head0 = 0;
    float* buf = reinterpret_cast<float*>(smem + kWarps * kStages * S::kStage);   // kBufs x [rows][kD], then the query rows (fp32)
    uint32_t live[kStages];
    look_up(true);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        live[s] = issue(s);
        look_up();
    }

    const ScoreForm form{p.cap > 0.0f ? p.scale / p.cap : p.scale * kLog2e, p.cap * kLog2e, p.cap > 0.0f};
    for (long long t = t0; t < t1;) {
        if (fresh) {
            const int unit = at.unit * sides + my_side, kh = unit / head_tiles, ht = unit - kh * head_tiles;
            rows = min(group - ht * W::kRows, W::kRows);
            head0 = kh * group + ht * W::kRows;
            w.start(p, buf + W::kBufs * W::kRows * kD, at.b, head0, rows, lane);
            piece_blk = at.blk;
            fresh = false;
        }
        cp_wait<kStages - 2>();
        __syncwarp();
        const int next = stage + kStages - 1 >= kStages ? stage - 1 : stage + kStages - 1;
        live[kStages - 1] = issue(next);
        look_up();
        if (live[0] != 0) {
            const uint32_t k = stage0 + stage * S::kStage;
            w.step(k, k + S::kBytes, (at.blk * kWarps + warp) * kKeys, live[0], at.n, form, rows, lane);
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s + 1 < kStages; ++s) live[s] = live[s + 1];
        stage = stage + 1 == kStages ? 0 : stage + 1;

        const bool unit_done = at.blk + 1 == at.nblk;
        if (unit_done || t + 1 == t1) {
            // ---- join the warps: the last kBufs put their scaled sums in buffers, the others add theirs, all sum the buffers
            w.put_stats(sh.m[warp], sh.l[warp], lane);
            __syncthreads();
            if (lane < W::kRows) {
                float M = -CUDART_INF_F;
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sh.m[i][lane]);
                const float mw = sh.m[warp][lane];
                sh.f[warp][lane] = mw == -CUDART_INF_F ? 0.0f : ex2_approx(mw - M);
            }
            __syncwarp();
            static_assert((W::kBufs & (W::kBufs - 1)) == 0, "a mask");
            float* own = buf + (warp & (W::kBufs - 1)) * (W::kRows * kD);
#pragma unroll
            for (int r = kWarps / W::kBufs - 1; r >= 0; --r) {
                if ((r == 0 || warp >= r * W::kBufs) && (r + 1 == kWarps / W::kBufs || warp < (r + 1) * W::kBufs)) w.put(own, sh.f[warp], r != kWarps / W::kBufs - 1, rows, lane);
                __syncthreads();
            }
            const bool whole = unit_done && piece_blk == 0;
            float* slot_m = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (first_piece ? 0 : 1)) * kSlot;
            for (int i = threadIdx.x; i < rows * kD; i += kThreads) {
                const int row = i / kD;
                float a = 0.0f;
#pragma unroll
                for (int s = 0; s < W::kBufs; ++s) a += buf[s * (W::kRows * kD) + i];
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
        advance(at, t);
    }
    cp_wait<0>();
}

// Joins the pieces of a unit that several CTAs share: block (c, row). Thread i weighs piece i (there are
// at most kSlots), then groups of kD / 4 threads sum every kGroups-th piece, 16 bytes a thread.
__host__ __device__ constexpr int join_threads(int slots) { return slots <= 256 ? 256 : 512; }
constexpr int kEarly = 8;        // loads of a thread that do not wait for the weights (one of 131071: 31.8 -> 30.5 us, of 16000: 12.9 -> 12.1)
template <typename T, int kD, int kSlots, bool kSided>
__global__ void __launch_bounds__(join_threads(kSlots)) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int rows_tile) {
    constexpr int kSlot = slot_floats<kD>();
    constexpr int kCols = kD / 4;
    constexpr int kJoinThreads = join_threads(kSlots), kGroups = kJoinThreads / kCols;
    static_assert(kSlots <= kJoinThreads, "one thread a piece");
    __shared__ float sh_f[kJoinThreads], sh_x[2][kJoinThreads / 32];
    __shared__ float4 sh_o[kGroups][kCols];
    pdl_trigger();
    pdl_wait();
    const JoinDesc d = reinterpret_cast<const JoinDesc*>(p.partial + static_cast<int64_t>(kSlots) * 2 * kSlot)[blockIdx.x];
    if (d.c1 < d.c0) return;
    const int group = p.h / p.h_kv;
    const int head_tiles = (group + rows_tile - 1) / rows_tile;
    const int kh = d.unit / head_tiles, ht = d.unit - kh * head_tiles;
    const int row = blockIdx.y;
    if (row >= min(group - ht * rows_tile, rows_tile)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pieces = d.c1 - d.c0 + 1;
    const int sides = kSided ? static_cast<int>(p.side.d) : 1, step = 2 * sides;
    const int my_side = kSided ? static_cast<int>(blockIdx.x) - p.side.div(blockIdx.x) * sides : 0;
    // piece i at i step kSlot, piece 0 at first_slot
    const float* slots = p.partial + (static_cast<int64_t>(d.c0) * sides + my_side) * 2 * kSlot;
    const float* mine = slots + (tid == 0 ? d.first_slot : step * tid) * kSlot;
    const int g = tid / kCols, x = tid % kCols;
    auto at = [&](int i) {
        return reinterpret_cast<const float4*>(slots + (i == 0 ? d.first_slot : step * i) * kSlot + 2 * kMaxRows + row * kD)[x];
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
    constexpr int kWarps = W::Step::kWarps, kThreads = W::Step::kThreads;
    constexpr int kSmem = kWarps * W::Step::kStages * W::Step::kStage + (W::kBufs * W::kRows * kD + W::kQFloats) * static_cast<int>(sizeof(float));
    static_assert((kSmem + sizeof(Shared<kWarps>) + 1024) * W::Step::kPerSm <= 233472, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<W, kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    int sms = 0;
    if (e == cudaSuccess) e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(sms, kSlotsPerSm) * W::Step::kPerSm;
    // Sequences of kWhole blocks at most are not worth the second kernel: a CTA takes longer over a unit by less
    // than the join costs (64 x 300, 32 / 8 heads of 128: 31 against 34 us; one of 500, 16 / 4 heads of 64: 10.8
    // against 13.0 us with the launches). The lengths are on the device, so the host goes by what the table has room for:
    // the same sequences behind a wider table take the two launches.
    constexpr int kBlock = W::Step::kKeys * kWarps;
    p.whole = static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d <= W::Step::kWhole * kBlock;
    const int64_t units = static_cast<int64_t>(p.B) * p.h_kv * ((p.h / p.h_kv + W::kRows - 1) / W::kRows);
    p.direct = p.whole && units <= (W::kSplits ? ctas : 0x7fffffff);        // the hardware hands out more than fit (200 x 20: 15.8 -> 13.0 us)
    // Neighbouring key heads lie side by side in a slot: CTAs that take their units in step read whole rows of memory between them
    // (24 sequences of 15000, 8 heads of 128, e4m3: 136 -> 120 us). As many as divide the units of a sequence, up to eight; not where units are short.
    int side = 1;
    if (W::Step::kScales > 0 && !p.whole)
        for (int i = 2; i <= 8; ++i)
            if (units / p.B % i == 0) side = i;
    p.side = fast_div(static_cast<uint32_t>(side));
    if (p.whole) {
        return launch_pdl(paged_attn_kernel<W, kD>, dim3(static_cast<unsigned>(p.direct ? units : std::min<int64_t>(units, ctas))), dim3(kThreads),
                          kSmem, s, p);
    }
    if constexpr (W::kSplits) {
        const int grid = ctas / side * side;
        if ((e = launch_pdl(paged_attn_kernel<W, kD>, dim3(grid), dim3(kThreads), kSmem, s, p)) != cudaSuccess) return e;
        const int rows = std::min(p.h / p.h_kv, W::kRows);
        return launch_pdl(paged_join_kernel<typename W::T, kD, W::Step::kSlots, (W::Step::kScales > 0)>, dim3(grid, rows), dim3(join_threads(W::Step::kSlots)), 0, s, p, static_cast<int>(W::kRows));
    } else {
        return cudaErrorInvalidConfiguration;       // its launcher has none that are not whole
    }
}
}  // namespace
}  // namespace mha
