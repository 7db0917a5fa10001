// coded_append.cuh -- rotary positions of new queries and keys, and the append of keys and values to a paged cache in 8 bits.
//
// A block of `block` tokens of one key head has a scale 2^e, the smallest power of two with max |x| <= top 2^e (top: 448 in
// e4m3, 127 in int8), and codes round(x / 2^e), x the turned key in fp32 (rounded once, not to the input's type before). Powers of
// two cost int8 half a bit on average and e4m3 nothing, and let a block grow: new tokens may raise the scale of a block
// that is in part filled, whose codes are then rounded again, which in e4m3 is exact but for subnormals. The maximum
// carries a NaN, so that or an infinity in a block makes its scale NaN.
//
// HBM-bound: q and k read and written, v read, codes written: 24.5 KB a token at 32 + 8 heads of 128 in bf16. Measured, 4 x 8192 of those,
// blocks of 64: half of each head turned 137-141 us (805 MB, 5.7-5.9 TB/s, 0.86 of measured copy bandwidth), nothing turned 125, all 160, halves
// of odd length (126) 270; 16 + 16 heads of 64 98 us; blocks of 16 136, of 8 132, of 4 143, of 256 192 (rows read twice, and cos and
// sin of 256 tokens leave one CTA an SM). int8 the same (131 us for 131, calls captured). fp32, 43 KB a token: 219 us, 1.41 GB, 6.4 TB/s in both codes. One token 4.5 us,
// 61 sequences of one token 4.5 us, 7 x 333 in fp32 5.8 us.
//
// A CTA takes a tile of neighbouring blocks of one sequence and a part of the heads. It computes the tile's cos and sin into shared
// memory, then its teams of warps take (block, key head) tasks of keys and of values: a row of d_k elements is
// kLanes lanes with two chunks of 16 bytes each, the two that turn together; kKeep passes of rows stay in shared memory between the
// maximum and the codes (longer blocks are read again, from L2). Then all warps turn the tile's rows of queries.
#pragma once

#include <algorithm>

#include <cuda_fp8.h>

#include "elem.cuh"
#include "launch.h"
#include "mha_internal.h"
#include "ptx_serve.cuh"
#include "serve.h"
#include "turn.cuh"

namespace mha {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;               // tokens of a tile, unless a block is longer
constexpr int kLongest = 256;           // tokens of a block: what cos and sin of a tile have room for
constexpr float kLeast = 0x1p-120f;     // least scale

struct TilePlan {
    int tiles;          // of a sequence
    int blocks;         // of a tile
    int tokens;         // of a tile, at most
    int parts;          // of the heads: as many CTAs a tile
    int kv_heads;       // of a part; the last may have fewer, or none
    FastDiv q_heads;    // of a part, equal for all
    FastDiv half;       // pairs that turn
    int team;           // warps of a task
    int room;           // floats a token of cos (and of sin): half, rounded up so that the rows behind them are aligned to 16 bytes
};

// Where a block lies: elements from the pages' start to its first slot, or -1; its place among the scales, without the head.
struct BlockInfo {
    int64_t slot, scale;
};

__device__ __forceinline__ uint32_t code4(bool int8, float a, float b, float c, float d) {
    if (int8) {
        uint32_t hi, r;
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(hi) : "r"(__float2int_rn(d)), "r"(__float2int_rn(c)));
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(__float2int_rn(b)), "r"(__float2int_rn(a)), "r"(hi));
        return r;
    } else {
        return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) |
               static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
    }
}
__device__ __forceinline__ float value_of(bool int8, uint32_t byte) {
    if (int8) return static_cast<float>(static_cast<int8_t>(byte));
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// The least power of two s with x <= top s, for the bits of x >= 0; NaN for those of no finite number.
__device__ __forceinline__ float scale_for(bool int8, uint32_t bits) {
    const uint32_t top = int8 ? 0x7e0000u : 0x600000u;           // the fraction of 127 = 1.984375 * 2^6, of 448 = 1.75 * 2^8
    const uint32_t power = int8 ? 6u : 8u;
    if (bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    const uint32_t e = (bits + (0x7fffffu - top)) >> 23;         // carries where the fraction is above the top's
    return e <= power + 7u ? kLeast : fmaxf(__uint_as_float((e - power) << 23), kLeast);
}

// Values over their block's scale: a product where that is a power of two (always, for scales that this kernel made).
template <int kN>
__device__ __forceinline__ void divide(float (&x)[kN], float (&y)[kN], float scale, float inv, bool power) {
    if (power) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            x[e] *= inv;
            y[e] *= inv;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            x[e] = __fdiv_rn(x[e], scale);
            y[e] = __fdiv_rn(y[e], scale);
        }
    }
}
// max(|a|, |b|, |c|), NaN where one is
__device__ __forceinline__ float most3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two chunks of a row: elements c0 .. c0 + kN - 1 and c1 .. c1 + kN - 1.
template <typename T>
struct Pair {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    uint4 a, b;
    __device__ __forceinline__ void load_shared(uint32_t at, bool on) {
        a = b = make_uint4(0, 0, 0, 0);
        if (!on) return;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w) : "r"(at));
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "r"(at + 512));
    }
    __device__ __forceinline__ void values(float (&x)[kN], float (&y)[kN]) const {
        const T* pa = reinterpret_cast<const T*>(&a);
        const T* pb = reinterpret_cast<const T*>(&b);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            x[i] = load_f(pa + i);
            y[i] = load_f(pb + i);
        }
    }
};
template <typename T>
__device__ __forceinline__ void store_chunk(T* p, const float* x) {
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    else
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// How pairs lie in a row: nothing turns; neighbours; halves whose elements meet in a lane's two chunks; halves that do not, which
// go through shared memory.
enum Turn { kNone, kNeighbours, kHalves, kStaged };

// kKeep passes of rows in a step, 32 bytes a lane each; kPerSm CTAs an SM
template <typename T, int kD, int kTurn, int kKeep, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) coded_append_kernel(const __grid_constant__ CodedAppendParams p, const __grid_constant__ TilePlan plan) {
    constexpr int kN = Pair<T>::kN;
    constexpr int kLanes = kD / (2 * kN);          // of a row
    constexpr int kRows = 32 / kLanes;             // of a warp at a time
    constexpr int kStep = kKeep * 1024;            // bytes
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ BlockInfo info[kTile];
    __shared__ uint32_t peak[2][kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x / plan.tiles, tile = blockIdx.x - b * plan.tiles, part = blockIdx.y;
    const int block = static_cast<int>(p.block.d), half = p.rot / 2;
    const bool int8 = p.int8 != 0;
    const int n = p.new_lens != nullptr ? min(max(p.new_lens[b], 0), p.T) : p.T;
    const long long start = p.start[b];
    // blocks of positions; those in front of position 0 exist in number only
    const long long blk0 = (start >= 0 ? p.block.div(static_cast<int>(start)) : -((block - 1 - start) / block)) + static_cast<long long>(tile) * plan.blocks;
    const int t0 = static_cast<int>(max(blk0 * block - start, 0ll));
    const int t1 = static_cast<int>(min((blk0 + plan.blocks) * block - start, static_cast<long long>(n)));
    if (t0 >= t1) return;
    const int tokens = t1 - t0;

    // ---- the lane's chunks of a row
    const int lr = lane / kLanes, li = lane - lr * kLanes;
    // neighbouring lanes' first chunks are neighbours, and so are their second ones: whole sectors an access
    int c0 = li * kN, c1 = c0 + kD / 2;
    if (kTurn == kHalves) {
        const int turning = half / kN;
        c0 = li < turning ? li * kN : p.rot + (li - turning) * kN;
        c1 = c0 + (li < turning ? half : (kD - p.rot) / 2);
    }

    // ---- A task is a block, a key head, and its keys or its values; a step of it is kKeep passes of rows. Behind those come steps of rows of
    // queries. Steps come into shared memory by asynchronous copies, the next one's while one is worked on; a lane reads what it
    // has copied.
    const int h0 = part * plan.kv_heads, kv_heads = max(min(plan.kv_heads, p.h_kv - h0), 0);
    const int q_heads = static_cast<int>(plan.q_heads.d), q0 = part * q_heads;
    const int tasks = plan.blocks * kv_heads * 2, teams = kWarps / plan.team;
    const int team = warp / plan.team, member = warp - team * plan.team;
    const int q_rows = q0 < p.h ? tokens * q_heads : 0;
    enum { kKeys, kValues, kQueries };
    struct Step {
        int kind, task;             // kQueries: task is the first row, of all rows of queries
        int step, rounds;           // every round for the maximum, then, from the last one back, for the codes
        int block, head, from, to;  // of the tile; the block's new tokens
        __device__ __forceinline__ int round() const { return step < rounds ? step : 2 * rounds - 2 - step; }
    };
    auto settle = [&](Step& x) {       // the first step of x.task, or of the next that has tokens
        for (; x.task < tasks; x.task += teams) {
            x.kind = x.task & 1;
            const int n = x.task >> 1;
            x.block = plan.blocks == 1 ? 0 : n / kv_heads;
            x.head = h0 + n - x.block * kv_heads;
            const long long first = (blk0 + x.block) * block;
            x.from = static_cast<int>(max(first - start, static_cast<long long>(t0)));
            x.to = static_cast<int>(min(first + block - start, static_cast<long long>(t1)));
            if (x.from >= x.to) continue;
            x.step = 0;
            x.rounds = 1;
            for (int rows = plan.team * kRows * kKeep; x.from + x.rounds * rows < x.to;) ++x.rounds;
            return;
        }
        x.kind = kQueries;
        x.task = warp * kRows * kKeep;
    };
    auto advance = [&](Step& x) {
        if (x.kind == kQueries) {
            x.task += kWarps * kRows * kKeep;
        } else if (++x.step == 2 * x.rounds - 1) {
            x.task += teams;
            settle(x);
        }
    };
    auto pending = [&](const Step& x) { return x.kind != kQueries || x.task < q_rows; };
    // a lane's token in pass i of a step of keys or values, at or behind x.to where there is none
    const int apart = plan.team * kRows;
    auto token_of = [&](const Step& x, int i) {
        return x.from + (x.round() * kKeep * plan.team + member) * kRows + lr + i * apart;
    };
    const uint32_t mine = smem_u32(smem) + warp * (2 * kStep) + lane * 16;
    auto fetch = [&](const Step& x, int buffer) {
        const uint32_t to = mine + buffer * kStep;
        if (x.kind != kQueries) {
            const Strided& in = x.kind == kValues ? p.v : p.k;
            const T* rows = static_cast<const T*>(in.p) + b * in.b + x.head * in.h;
            const T* first = rows + token_of(x, 0) * in.l;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int t = token_of(x, i);
                if (t >= x.to) continue;
                const T* row = first + i * (apart * in.l);
                cp_async16(to + i * 1024, row + c0, true);
                cp_async16(to + i * 1024 + 512, row + c1, true);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int r = x.task + i * kRows + lr;
                if (r >= q_rows) break;
                const int t = plan.q_heads.div(r);
                const T* row = static_cast<const T*>(p.q.p) + b * p.q.b + (t0 + t) * p.q.l + (q0 + r - t * q_heads) * p.q.h;
                cp_async16(to + i * 1024, row + c0, true);
                cp_async16(to + i * 1024 + 512, row + c1, true);
            }
        }
        cp_commit();
    };
    Step now{};
    now.task = team;
    settle(now);
    fetch(now, 0);

    // ---- cos and sin of the tile, [tokens][half] each; where the blocks lie
    float* cosines = reinterpret_cast<float*>(smem + kWarps * 2 * kStep);
    float* sines = cosines + plan.tokens * plan.room;
    if (kTurn != kNone) {
        for (int i = tid; i < tokens * half; i += kThreads) {
            const int t = i / half, e = i - t * half;
            const float2 cs = turn_of(static_cast<int>(start + t0 + t), p.inv_freq[e]);
            cosines[i] = cs.x * p.scale;
            sines[i] = cs.y * p.scale;
        }
    }
    for (int i = tid; i < plan.blocks; i += kThreads) {
        const long long first = (blk0 + i) * block;        // position
        BlockInfo x{-1, -1};
        const long long last = min(first + block, start + t1) - 1;
        if (last >= max(first, start + t0)) {
            int page = -1, pg = 0;
            // a block lies in one page, so one look-up does for all its positions
            if (first >= 0 && last <= 0x7fffffffll) {
                pg = p.cache.page.div(static_cast<int>(first));
                if (pg < p.cache.max_pages) page = p.cache.table[b * p.cache.table_stride + pg];
            }
            if (page >= 0 && page < p.cache.n_pages) {
                const int slot = static_cast<int>(first) - pg * static_cast<int>(p.cache.page.d);
                x.slot = page * p.cache.page_stride + slot * p.cache.slot_stride;
                x.scale = page * p.page_scales + static_cast<int64_t>(p.block.div(slot)) * p.h_kv;
            } else {
                atomicCAS(p.status, 0, MHA_PAGED_BAD_PAGE);     // its tokens are not appended
            }
        }
        info[i] = x;
    }

    float* stage = sines + plan.tokens * plan.room + warp * (kRows * kD);       // kStaged: a pass of rows
    __syncthreads();

    auto turn = [&](float (&x)[kN], float (&y)[kN], int t, bool on) {
        if (kTurn == kNone) return;
        const float* cs = cosines + t * half;
        const float* sn = sines + t * half;
        if (kTurn == kStaged) {
            // the pass's rows in shared memory, a pair a lane at a time; a short block leaves passes empty (6 x 468 in blocks of 8: 24.0 -> 22.9 us)
            if (__ballot_sync(0xffffffffu, on) == 0) return;
            float* row = stage + lr * kD;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                *reinterpret_cast<float4*>(row + c0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                *reinterpret_cast<float4*>(row + c1 + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
            __syncwarp();
            for (int i0 = 0; i0 < kRows * half; i0 += 32) {
                const int i = min(i0 + lane, kRows * half - 1), n = plan.half.div(i), e = i - n * half;
                const int of = __shfl_sync(0xffffffffu, t, n * kLanes);
                if (i0 + lane >= kRows * half) continue;
                float* pair = stage + n * kD + e;
                const float c = cosines[of * half + e], s = sines[of * half + e], u = pair[0], v = pair[half];
                pair[0] = fmaf(u, c, -(v * s));
                pair[half] = fmaf(v, c, u * s);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                const float4 a = *reinterpret_cast<const float4*>(row + c0 + i), b = *reinterpret_cast<const float4*>(row + c1 + i);
                x[i] = a.x; x[i + 1] = a.y; x[i + 2] = a.z; x[i + 3] = a.w;
                y[i] = b.x; y[i + 1] = b.y; y[i + 2] = b.z; y[i + 3] = b.w;
            }
        } else if (kTurn == kNeighbours) {
            if (!on) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float (&z)[kN] = h == 0 ? x : y;
                const int at = h == 0 ? c0 : c1;
#pragma unroll
                for (int i = 0; i < kN; i += 2) {
                    if (at + i >= p.rot) break;          // what does not turn stays, beside an infinity too
                    const float c = cs[(at + i) / 2], s = sn[(at + i) / 2], u = z[i], v = z[i + 1];
                    z[i] = fmaf(u, c, -(v * s));
                    z[i + 1] = fmaf(v, c, u * s);
                }
            }
        } else {
            if (!on || c0 >= half) return;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const float c = cs[c0 + i], s = sn[c0 + i], u0 = x[i];
                x[i] = fmaf(u0, c, -(y[i] * s));
                y[i] = fmaf(y[i], c, u0 * s);
            }
        }
    };

    int flip = 0, buffer = 0;
    float top = 0.0f, scale = 1.0f;
    // A block's scale, from the largest of its new values: written, and the codes in front of them rounded again where it grows.
    auto settle_scale = [&](const Step& x, uint32_t most) {
        if (plan.team > 1) {
            if (lane == 0) peak[flip][warp] = most;
            named_bar_sync(1 + team, 32 * plan.team);
            for (int i = 0; i < plan.team; ++i) most = max(most, peak[flip][team * plan.team + i]);
            flip ^= 1;                             // the other half is free: its readers have passed this barrier
        }
        float s = scale_for(int8, most);
        const BlockInfo where = info[x.block];
        const bool kept = where.slot >= 0;
        float* scale_at = (x.kind == kValues ? p.v_scales : p.k_scales) + (kept ? where.scale + x.head : 0);
        // slots of the block that hold earlier tokens: only of the tile's first
        const int filled = static_cast<int>(start + x.from - (blk0 + x.block) * block);
        if (kept && filled > 0) {
            const float old = *scale_at;
            if (!(old <= s)) s = isnan(s) ? s : old;     // the larger; NaN stays
            else if (old < s) {
                const float ratio = old / s;
                uint8_t* codes = static_cast<uint8_t*>(x.kind == kValues ? p.cache.v : p.cache.k) + where.slot + x.head * p.cache.head_stride;
                for (int i = member * kRows + lr; i < filled; i += apart) {
                    uint8_t* row = codes + i * p.cache.slot_stride;
#pragma unroll 1
                    for (int e = 0; e < 2 * kN; e += 4) {
                        uint32_t* w = reinterpret_cast<uint32_t*>(row + (e < kN ? c0 + e : c1 + e - kN));
                        const uint32_t c = *w;
                        *w = code4(int8, value_of(int8, c & 0xffu) * ratio, value_of(int8, (c >> 8) & 0xffu) * ratio,
                                   value_of(int8, (c >> 16) & 0xffu) * ratio, value_of(int8, c >> 24) * ratio);
                    }
                }
            }
        }
        // every warp of the team has read the old scale before one writes the new
        if (plan.team > 1 && filled > 0) named_bar_sync(1 + team, 32 * plan.team);
        else __syncwarp();
        if (kept && member == 0 && lane == 0) *scale_at = s;
        return s;
    };

    while (pending(now)) {
        Step next = now;
        advance(next);
        fetch(next, buffer ^ 1);
        cp_wait<1>();
        const uint32_t at = mine + buffer * kStep;
        if (now.kind == kQueries) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int r = now.task + i * kRows + lr;
                const bool on = r < q_rows;
                if (kTurn != kStaged && !on) break;
                const int t = plan.q_heads.div(on ? r : 0);
                Pair<T> raw;
                raw.load_shared(at + i * 1024, on);
                float x[kN], y[kN];
                raw.values(x, y);
                turn(x, y, t, on);
                if (!on) continue;
                T* row = static_cast<T*>(p.q_out.p) + b * p.q_out.b + (t0 + t) * p.q_out.l + (q0 + r - t * q_heads) * p.q_out.h;
                store_chunk(row + c0, x);
                store_chunk(row + c1, y);
            }
        } else {
            float x[kKeep][kN], y[kKeep][kN];
            float most[kKeep];
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int t = token_of(now, i);
                const bool on = t < now.to;
                Pair<T> raw;
                raw.load_shared(at + i * 1024, on);
                raw.values(x[i], y[i]);
                if (now.kind == kKeys) turn(x[i], y[i], min(t, now.to - 1) - t0, on);
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < kN; ++e) m = most3(m, x[i][e], y[i][e]);
                most[i] = m;
            }
            if (now.step == 0) top = 0.0f;
            if (now.step < now.rounds) {
#pragma unroll
                for (int i = 0; i < kKeep; ++i) top = most3(top, most[i], 0.0f);
            }
            if (now.step == now.rounds - 1) scale = settle_scale(now, __reduce_max_sync(0xffffffffu, __float_as_uint(top)));      // NaN is above all
            if (now.step >= now.rounds - 1) {
                const int t_first = token_of(now, 0);
                if (now.kind == kKeys && p.k_out.p != nullptr) {
                    T* rows = static_cast<T*>(p.k_out.p) + b * p.k_out.b + now.head * p.k_out.h;
                    T* first = rows + t_first * p.k_out.l;
#pragma unroll
                    for (int i = 0; i < kKeep; ++i) {
                        const int t = token_of(now, i);
                        if (t >= now.to) continue;
                        T* row = first + i * (apart * p.k_out.l);
                        store_chunk(row + c0, x[i]);
                        store_chunk(row + c1, y[i]);
                    }
                }
                const BlockInfo where = info[now.block];
                if (where.slot < 0) now.to = 0;          // nothing is stored
                uint8_t* const pages = static_cast<uint8_t*>(now.kind == kValues ? p.cache.v : p.cache.k) + now.head * p.cache.head_stride;
                uint8_t* const first = pages + where.slot + static_cast<int>(start + t_first - (blk0 + now.block) * block) * p.cache.slot_stride;
                const float inv = 1.0f / scale;
                const bool power = (__float_as_uint(scale) & 0x7fffffu) == 0;
#pragma unroll
                for (int i = 0; i < kKeep; ++i) {
                    const int t = token_of(now, i);
                    if (t >= now.to) continue;
                    uint8_t* row = first + i * (apart * p.cache.slot_stride);
                    divide(x[i], y[i], scale, inv, power);
                    uint32_t u[kN / 4], v[kN / 4];
#pragma unroll
                    for (int e = 0; e < kN / 4; ++e) {
                        u[e] = code4(int8, x[i][4 * e], x[i][4 * e + 1], x[i][4 * e + 2], x[i][4 * e + 3]);
                        v[e] = code4(int8, y[i][4 * e], y[i][4 * e + 1], y[i][4 * e + 2], y[i][4 * e + 3]);
                    }
                    if constexpr (kN == 8) {
                        *reinterpret_cast<uint2*>(row + c0) = make_uint2(u[0], u[1]);
                        *reinterpret_cast<uint2*>(row + c1) = make_uint2(v[0], v[1]);
                    } else {
                        *reinterpret_cast<uint32_t*>(row + c0) = u[0];
                        *reinterpret_cast<uint32_t*>(row + c1) = v[0];
                    }
                }
            }
        }
        now = next;
        buffer ^= 1;
    }
    cp_wait<0>();
}

// Of steps, cos and sin of `tokens` tokens with room for `room` floats each, and a pass of rows that turn in shared memory: up to 208 KB (256 tokens,
// halves of 57 to 63 pairs).
template <typename T, int kD, int kKeep>
constexpr size_t shared_bytes(int turn, int tokens, int room) {
    constexpr int kRows = 64 * Pair<T>::kN / kD;
    return kWarps * 2 * kKeep * 1024 + static_cast<size_t>(tokens) * room * 2 * sizeof(float) + (turn == kStaged ? kWarps * kRows * kD * sizeof(float) : 0);
}

template <typename T, int kD, int kKeep, int kPerSm>
cudaError_t launch_n(const CodedAppendParams& p, TilePlan plan, int sms, cudaStream_t s) {
    constexpr int kN = Pair<T>::kN, kRows = 64 * kN / kD;
    const int block = static_cast<int>(p.block.d), half = p.rot / 2;
    plan.team = 1;
    while (plan.team < kWarps && std::min(block, p.T) > plan.team * kRows * kKeep) plan.team *= 2;
    // Parts of the heads: where tiles are fewer than one wave, to fill that, and no further for a few tokens a sequence
    // (61 x 1, 32 / 8 heads of 128: 4.4 us, twice as many CTAs 8.7); where they are more, to three waves, whose ends even out (4 x 8192 ragged, 516
    // tiles: two parts 105 us, one 113). Short blocks are many tasks a CTA: two waves (9 x 397 in blocks of 4, 16 heads of 64: 57 -> 30 us).
    const int64_t wave = static_cast<int64_t>(kPerSm) * sms;
    const int64_t alone = static_cast<int64_t>(p.B) * plan.tiles;
    const int64_t wanted = alone >= wave ? (3 * wave + alone - 1) / alone
                           : p.T < kTile ? wave / alone
                                         : ((block <= kRows ? 2 : 1) * wave + alone - 1) / alone;
    const int heads = std::max(p.h_kv, p.h), parts = static_cast<int>(std::min<int64_t>(wanted, heads));
    auto each = [&](int h, int n) { return (h + n - 1) / n; };
    plan.kv_heads = each(p.h_kv, std::min(parts, p.h_kv));
    // equal numbers of query heads: the next divisor of theirs, unless that is far
    int q_parts = std::min(parts, std::max(p.h, 1));
    while (p.h % q_parts != 0 && q_parts < 4 * parts) ++q_parts;
    while (p.h % q_parts != 0) --q_parts;
    plan.q_heads = fast_div(static_cast<uint32_t>(std::max(p.h / q_parts, 1)));
    plan.parts = std::max(each(p.h_kv, plan.kv_heads), p.h > 0 ? q_parts : 1);
    plan.room = (half + kN - 1) / kN * kN;
    plan.half = fast_div(static_cast<uint32_t>(std::max(half, 1)));
    const int turn = half == 0 ? kNone : p.interleaved != 0 ? kNeighbours : half % kN == 0 ? kHalves : kStaged;
    const auto kernel = turn == kNone         ? coded_append_kernel<T, kD, kNone, kKeep, kPerSm>
                        : turn == kNeighbours ? coded_append_kernel<T, kD, kNeighbours, kKeep, kPerSm>
                        : turn == kHalves     ? coded_append_kernel<T, kD, kHalves, kKeep, kPerSm>
                                              : coded_append_kernel<T, kD, kStaged, kKeep, kPerSm>;
    // The limit is the kernel's in the whole process, and another thread's call may come between this and the launch: it is the most that
    // any call of this kernel needs, never what this one does.
    constexpr int kTokens = kKeep == 4 ? kLongest : kTile;
    static_assert(shared_bytes<T, kD, kKeep>(kStaged, kLongest, kD / 2) + 1024 <= 227 * 1024, "shared memory budget");
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(shared_bytes<T, kD, kKeep>(turn, kTokens, turn == kNone ? 0 : kD / 2)));
    if (e != cudaSuccess) return e;
    const size_t smem = shared_bytes<T, kD, kKeep>(turn, plan.tokens, plan.room);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * plan.tiles), plan.parts), dim3(kThreads), smem, s, p, plan);
}

// A step has the passes that a block fills, up to four: fewer take less issue and fewer registers, so more CTAs run on an SM (4 x 8000 in blocks of 4,
// 32 / 8 heads of 128: one pass 139 us, four 180; of 8: two 129, four 142; of 16: 140 and 133; 16 heads of 64, of 4: 154 and 251; of 8: 92 and 143). The last CTA an SM
// costs spills, which many tiles pay back and few do not (one pass, 4 / 3 an SM: the first 139 / 148, 3 x 700 8.5 / 7.0, 200 x 1 6.7 / 5.1; two, 3 / 2: blocks of 8 129 / 141,
// 6 x 468, 16 / 8 heads 11.5 / 9.9).
template <typename T, int kD>
cudaError_t launch_d(const CodedAppendParams& p, cudaStream_t s) {
    constexpr int kRows = 64 * Pair<T>::kN / kD;
    const int block = static_cast<int>(p.block.d), rows = std::min(block, p.T);
    TilePlan plan{};
    // tiles of about kTile tokens, so that cos and sin serve many heads and a CTA has rows for all its warps; of one block where
    // that is longer
    plan.blocks = std::max(1, std::min(kTile, p.T) / block);
    plan.tokens = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(plan.blocks) * block, p.T));
    const int64_t most = (static_cast<int64_t>(p.T) + block - 2) / block + 1;         // blocks that T tokens touch
    plan.tiles = static_cast<int>((most + plan.blocks - 1) / plan.blocks);
    int sms = 0;
    if (const cudaError_t e = sm_count(&sms); e != cudaSuccess) return e;
    const bool many = static_cast<int64_t>(p.B) * plan.tiles >= sms && p.T >= kTile;
    if (rows <= kRows) return many ? launch_n<T, kD, 1, 4>(p, plan, sms, s) : launch_n<T, kD, 1, 3>(p, plan, sms, s);
    if (rows <= 2 * kRows) return many ? launch_n<T, kD, 2, 3>(p, plan, sms, s) : launch_n<T, kD, 2, 2>(p, plan, sms, s);
    return launch_n<T, kD, 4, 2>(p, plan, sms, s);
}

template <typename T>
cudaError_t launch_t(const CodedAppendParams& p, cudaStream_t s) {
    return p.d == 64 ? launch_d<T, 64>(p, s) : launch_d<T, 128>(p, s);
}

}  // namespace
}  // namespace mha
