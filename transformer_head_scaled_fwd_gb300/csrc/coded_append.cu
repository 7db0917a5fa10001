// coded_append.cu -- rotary positions of new queries and keys, and the append of keys and values to a paged cache in 8 bits.
//
// A block of `block` tokens of one key head has a scale 2^e, the smallest power of two with max |x| <= top 2^e (top: 448 in
// e4m3, 127 in int8), and codes round(x / 2^e), x the turned key in fp32 (rounded once, not to the input's type before). Powers of
// two cost int8 half a bit on average and e4m3 nothing, and let a block grow: new tokens may raise the scale of a block
// that is in part filled, whose codes are then rounded again, which in e4m3 is exact but for subnormals. The maximum
// carries a NaN, so that or an infinity in a block makes its scale NaN.
//
// HBM-bound: q and k read and written, v read, codes written: 24.5 KB a token at 32 + 8 heads of 128 in bf16.
//
// A CTA takes a tile of neighbouring blocks of one sequence and a part of the heads. It computes the tile's cos and sin into shared
// memory, then its teams of warps take (block, key head) tasks of keys and of values: a row of d_k elements is
// kLanes lanes with two chunks of 16 bytes each, the two that turn together; kKeep passes of rows stay in shared memory between the
// maximum and the codes (longer blocks are read again, from L2). Then all warps turn the tile's rows of queries.
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
constexpr float kLeast = 0x1p-120f;     // least scale

struct TilePlan {
    int tiles;          // of a sequence
    int blocks;         // of a tile
    int parts;          // of the heads
    int team;           // warps of a task
    int stride;         // floats of a token's row of cos (and of sin)
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
    __device__ __forceinline__ void load(const T* row, int c0, int c1) {
        a = *reinterpret_cast<const uint4*>(row + c0);
        b = *reinterpret_cast<const uint4*>(row + c1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load_shared(uint32_t at) {
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

template <typename T, int kD, int kTurn>
__global__ void __launch_bounds__(kThreads, 3) coded_append_kernel(const __grid_constant__ CodedAppendParams p, const __grid_constant__ TilePlan plan) {
    constexpr int kN = Pair<T>::kN;
    constexpr int kLanes = kD / (2 * kN);          // of a row
    constexpr int kRows = 32 / kLanes;             // of a warp at a time
    constexpr int kKeep = 4;                       // passes in a step, 32 bytes a lane each
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
    int c0 = li * 2 * kN, c1 = c0 + kN;
    if (kTurn == kHalves) {
        const int turning = half / kN;
        c0 = li < turning ? li * kN : p.rot + (li - turning) * 2 * kN;
        c1 = li < turning ? c0 + half : c0 + kN;
    }

    // ---- keys and values: a task is a block, a key head, and one of the two; a step of it is kKeep passes of rows. Steps come into shared
    // memory by asynchronous copies, the next one's while one is worked on; a lane reads what it has copied.
    const int h0 = static_cast<int>(static_cast<int64_t>(part) * p.h_kv / plan.parts);
    const int heads = static_cast<int>(static_cast<int64_t>(part + 1) * p.h_kv / plan.parts) - h0;
    const int tasks = plan.blocks * heads * 2, teams = kWarps / plan.team;
    const int team = warp / plan.team, member = warp - team * plan.team;
    struct Step {
        int task, step, rounds;     // every round for the maximum, then, from the last one back, for the codes
        int block, head, from, to;  // of the tile; the block's new tokens
        bool values;
        __device__ __forceinline__ int round() const { return step < rounds ? step : 2 * rounds - 2 - step; }
    };
    auto settle = [&](Step& x) {       // the first step of x.task, or of the next that has tokens
        for (; x.task < tasks; x.task += teams) {
            x.values = x.task & 1;
            x.block = (x.task >> 1) / heads;
            x.head = h0 + (x.task >> 1) - x.block * heads;
            const long long first = (blk0 + x.block) * block;
            x.from = static_cast<int>(max(first - start, static_cast<long long>(t0)));
            x.to = static_cast<int>(min(first + block - start, static_cast<long long>(t1)));
            x.step = 0;
            const int passes = (x.to - x.from + plan.team * kRows - 1) / (plan.team * kRows);
            x.rounds = (passes + kKeep - 1) / kKeep;
            if (x.from < x.to) return;
        }
    };
    auto advance = [&](Step& x) {
        if (++x.step < 2 * x.rounds - 1) return;
        x.task += teams;
        settle(x);
    };
    auto row_of = [&](const Step& x, int i) { return x.from + ((x.round() * kKeep + i) * plan.team + member) * kRows + lr; };
    const uint32_t mine = smem_u32(smem) + warp * (2 * kStep) + lane * 16;
    auto fetch = [&](const Step& x, int buffer) {
        if (x.task < tasks) {
            const Strided& in = x.values ? p.v : p.k;
            const T* src = static_cast<const T*>(in.p) + b * in.b + x.head * in.h;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int t = row_of(x, i);
                if (t >= x.to) continue;
                const T* row = src + t * in.l;
                cp_async16(mine + buffer * kStep + i * 1024, row + c0, true);
                cp_async16(mine + buffer * kStep + i * 1024 + 512, row + c1, true);
            }
        }
        cp_commit();
    };
    Step now{};
    now.task = team;
    settle(now);
    fetch(now, 0);

    // ---- cos and sin of the tile, [tokens][stride] each; where the blocks lie
    float* cosines = reinterpret_cast<float*>(smem + kWarps * 2 * kStep);
    float* sines = cosines + plan.blocks * block * plan.stride;
    const int span = plan.stride;
    if (kTurn != kNone) {
        for (int i = tid; i < tokens * span; i += kThreads) {
            const int t = i / span, e = i - t * span;
            float2 cs = make_float2(1.0f, 0.0f);       // behind the pairs that turn
            if (e < half) {
                cs = turn_of(static_cast<int>(start + t0 + t), p.inv_freq[e]);
                cs.x *= p.scale;
                cs.y *= p.scale;
            }
            cosines[i] = cs.x;
            sines[i] = cs.y;
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

    float* stage = sines + plan.blocks * block * plan.stride + warp * (kRows * kD);       // kStaged: a pass of rows
    __syncthreads();

    auto turn = [&](float (&x)[kN], float (&y)[kN], int t, bool on) {
        if (kTurn == kNone) return;
        const float* cs = cosines + t * span;
        const float* sn = sines + t * span;
        if (kTurn == kStaged) {
            float* row = stage + lr * kD;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                row[c0 + i] = x[i];
                row[c1 + i] = y[i];
            }
            __syncwarp();
            if (!on) return;
#pragma unroll
            for (int i = 0; i < 2 * kN; ++i) {
                const int e = c0 + i;          // c1 = c0 + kN here
                if (e >= p.rot) break;
                float& v = i < kN ? x[i % kN] : y[i % kN];
                const int pr = e < half ? e : e - half;
                const float other = row[e < half ? e + half : pr];
                v = e < half ? fmaf(v, cs[pr], -(other * sn[pr])) : fmaf(v, cs[pr], other * sn[pr]);
            }
        } else if (kTurn == kNeighbours) {
            if (!on || c0 >= p.rot) return;
#pragma unroll
            for (int i = 0; i < 2 * kN; i += 2) {
                float& u = i < kN ? x[i % kN] : y[i % kN];
                float& v = i < kN ? x[i % kN + 1] : y[i % kN + 1];
                const float c = cs[c0 / 2 + i / 2], s = sn[c0 / 2 + i / 2], u0 = u;
                u = fmaf(u0, c, -(v * s));
                v = fmaf(v, c, u0 * s);
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
    while (now.task < tasks) {
        Step next = now;
        advance(next);
        fetch(next, buffer ^ 1);
        cp_wait<1>();
        const long long first = (blk0 + now.block) * block;
        const uint32_t at = mine + buffer * kStep;
        if (now.step == 0) top = 0.0f;
        if (now.step < now.rounds) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int t = row_of(now, i);
                if (kTurn != kStaged && t >= now.to) continue;
                Pair<T> raw;
                if (t < now.to) raw.load_shared(at + i * 1024);
                else raw.zero();
                float x[kN], y[kN];
                raw.values(x, y);
                if (!now.values) turn(x, y, min(t, now.to - 1) - t0, t < now.to);
#pragma unroll
                for (int e = 0; e < kN; ++e) top = most3(top, x[e], y[e]);
            }
        }
        if (now.step >= now.rounds - 1) {
            const BlockInfo where = info[now.block];
            const bool kept = where.slot >= 0;
            uint8_t* codes = static_cast<uint8_t*>(now.values ? p.cache.v : p.cache.k) + (kept ? where.slot + now.head * p.cache.head_stride : 0);
            if (now.step == now.rounds - 1) {
                uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));      // NaN is above all
                if (plan.team > 1) {
                    if (lane == 0) peak[flip][warp] = most;
                    named_bar_sync(1 + team, 32 * plan.team);
                    for (int i = 0; i < plan.team; ++i) most = max(most, peak[flip][team * plan.team + i]);
                    flip ^= 1;                             // the other half is free: its readers have passed this barrier
                }
                scale = scale_for(int8, most);
                float* scale_at = (now.values ? p.v_scales : p.k_scales) + (kept ? where.scale + now.head : 0);
                const int filled = static_cast<int>(start + now.from - first);       // slots of the block that hold earlier tokens
                if (kept && filled > 0) {
                    const float old = *scale_at;
                    if (!(old <= scale)) scale = isnan(scale) ? scale : old;     // the larger; NaN stays
                    else if (old < scale) {
                        const float ratio = old / scale;
                        for (int i = member * kRows + lr; i < filled; i += plan.team * kRows) {
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
                if (kept && member == 0 && lane == 0) *scale_at = scale;
            }
            T* const turned = now.values ? nullptr : static_cast<T*>(p.k_out.p);
            const float inv = 1.0f / scale;
            const bool power = (__float_as_uint(scale) & 0x7fffffu) == 0;
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int t = row_of(now, i);
                if (kTurn != kStaged && t >= now.to) continue;
                Pair<T> raw;
                if (t < now.to) raw.load_shared(at + i * 1024);
                else raw.zero();
                float x[kN], y[kN];
                raw.values(x, y);
                if (!now.values) turn(x, y, min(t, now.to - 1) - t0, t < now.to);
                if (t >= now.to) continue;
                if (turned != nullptr) {
                    T* row = turned + b * p.k_out.b + t * p.k_out.l + now.head * p.k_out.h;
                    store_chunk(row + c0, x);
                    store_chunk(row + c1, y);
                }
                if (!kept) continue;
                divide(x, y, scale, inv, power);
                uint8_t* row = codes + static_cast<int>(start + t - first) * p.cache.slot_stride;
                uint32_t u[kN / 4], v[kN / 4];
#pragma unroll
                for (int e = 0; e < kN / 4; ++e) {
                    u[e] = code4(int8, x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    v[e] = code4(int8, y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
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
        now = next;
        buffer ^= 1;
    }
    cp_wait<0>();

    // ---- queries
    if (p.q.p == nullptr) return;
    const int q0 = static_cast<int>(static_cast<int64_t>(part) * p.h / plan.parts);
    const int qh = static_cast<int>(static_cast<int64_t>(part + 1) * p.h / plan.parts) - q0;
    constexpr int kAtOnce = 2;
    const int all = tokens * qh;
    for (int r0 = warp * kRows * kAtOnce; r0 < all; r0 += kWarps * kRows * kAtOnce) {
        Pair<T> raw[kAtOnce];
        int t[kAtOnce], hd[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int row = r0 + i * kRows + lr;
            t[i] = row < all ? row / qh : -1;
            hd[i] = q0 + row - t[i] * qh;
            if (t[i] >= 0) raw[i].load(static_cast<const T*>(p.q.p) + b * p.q.b + (t0 + t[i]) * p.q.l + hd[i] * p.q.h, c0, c1);
            else raw[i].zero();
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            float x[kN], y[kN];
            raw[i].values(x, y);
            turn(x, y, max(t[i], 0), t[i] >= 0);
            if (t[i] < 0) continue;
            T* row = static_cast<T*>(p.q_out.p) + b * p.q_out.b + (t0 + t[i]) * p.q_out.l + hd[i] * p.q_out.h;
            store_chunk(row + c0, x);
            store_chunk(row + c1, y);
        }
    }
}

template <typename T, int kD>
cudaError_t launch_n(const CodedAppendParams& p, cudaStream_t s) {
    constexpr int kN = Pair<T>::kN, kRows = 64 * kN / kD, kKeep = 4;
    const int block = static_cast<int>(p.block.d), half = p.rot / 2;
    TilePlan plan{};
    // tiles of about kTile tokens, so that cos and sin serve many heads and a CTA has rows for all its warps; of one block where
    // that is longer
    plan.blocks = std::max(1, std::min(kTile, p.T) / block);
    const int64_t most = (static_cast<int64_t>(p.T) + block - 2) / block + 1;         // blocks that T tokens touch
    plan.tiles = static_cast<int>((most + plan.blocks - 1) / plan.blocks);
    plan.team = 1;
    while (plan.team < kWarps && std::min(block, p.T) > plan.team * kRows * kKeep) plan.team *= 2;
    // parts of the heads, while the CTAs are fewer than eight an SM
    plan.parts = 1;
    while (plan.parts * 2 <= p.h_kv && static_cast<int64_t>(p.B) * plan.tiles * plan.parts < 152 * 8) plan.parts *= 2;
    plan.stride = (half + kN - 1) / kN * kN;
    const Turn turn = half == 0 ? kNone : p.interleaved != 0 ? kNeighbours : half % kN == 0 ? kHalves : kStaged;
    const size_t smem = kWarps * 2 * kKeep * 1024 + static_cast<size_t>(plan.blocks) * block * plan.stride * 2 * sizeof(float) + (turn == kStaged ? kWarps * kRows * kD * sizeof(float) : 0);
    const auto kernel = turn == kNone ? coded_append_kernel<T, kD, kNone> : turn == kNeighbours ? coded_append_kernel<T, kD, kNeighbours>
                        : turn == kHalves ? coded_append_kernel<T, kD, kHalves> : coded_append_kernel<T, kD, kStaged>;
    {        // up to 211 KB: 256 tokens, 64 pairs
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * plan.tiles), plan.parts), dim3(kThreads), smem, s, p, plan);
}

template <typename T>
cudaError_t launch_t(const CodedAppendParams& p, cudaStream_t s) {
    return p.d == 64 ? launch_n<T, 64>(p, s) : launch_n<T, 128>(p, s);
}

}  // namespace

cudaError_t launch_coded_append(const CodedAppendParams& p, bool bf16, cudaStream_t s) {
    CodedAppendParams q = p;
    if (p.q.p != nullptr && static_cast<int64_t>(p.B) * p.T * p.h * p.d >= (1 << 20)) {
        // many queries: by the kernel that turns without a cache
        RotaryParams r{};
        r.q = p.q; r.q_out = p.q_out;
        r.start = p.start; r.new_lens = p.new_lens;
        r.inv_freq = p.inv_freq; r.rot = p.rot; r.interleaved = p.interleaved; r.scale = p.scale;
        r.B = p.B; r.T = p.T; r.h = p.h; r.d = p.d; r.status = p.status;
        const cudaError_t e = launch_rotary(r, bf16, s);
        if (e != cudaSuccess) return e;
        q.q.p = q.q_out.p = nullptr;
        q.h = 0;
    }
    return bf16 ? launch_t<__nv_bfloat16>(q, s) : launch_t<float>(q, s);
}

}  // namespace mha
