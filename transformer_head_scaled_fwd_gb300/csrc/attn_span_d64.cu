// attn_span_d64.cu -- attention under span masks for heads of 64 over long key ranges (attn_span.cu has the masks, the
// formulas, and the kernel for everything else).
//
// At d_k = 64 the two products of a tile take half as long as at 128, the softmax as long as ever. The warps of one
// scheduler then stand in the same phase of the same tile: all in their exponentials (512 cycles of the special
// function unit a tile), then none. So a unit of work is two query tiles of 128 rows of one head, two threads a row,
// and the two tiles' warps are independent but for the loads: warpgroup pair t has the rows of tile t, its scores S_t,
// weights P_t and output O_t in tensor memory, and one tile's exponentials pass while the other waits for its scores
// or stores its weights. Each key and value tile is loaded once for both, and computed only for the query tiles whose
// rows can see it.
//
// Measured, 4 x 8192 causal, 16 heads: 541 us, 1017 TFLOP/s (0.53 of measured bf16 peak; all keys 1072); the kernel of
// one query tile 660 us; two query tiles with one thread a row (eight softmax warps) 581 us, all keys 987 against 1026
// us. With a distance bias 814 us (in the other layout 896). Capped scores
// without a bias stay with the other kernel (documents of 1024 190 us there, 207 us with an instance here; 4 x 8192 causal 916
// and 870 us).
//
// Tensor memory (512 columns): S_0 S_1 (fp32, 128 each), P_0 P_1 (bf16, 64 each), O_0 O_1 (fp32, 64 each).
// Shared memory: two Q buffers of two tiles, K and V rings of four tiles, the two output tiles on their way out. Warps:
// 0-7 / 8-15 softmax of tile 0 / 1, then scheduler and Q, K loads; score MMAs; P.V MMAs; V loads. Registers: 96 a
// thread at launch; the last warpgroup drops to 56, the others rise to 104 (128 * 56 + 512 * 104 = 60416 <= 640 * 96).
#include <algorithm>

#include "attn_span.cuh"
#include "launch.h"

namespace mha {
namespace {

constexpr int BM = 128;                      // rows of a query tile
constexpr int kRowsUnit = 2 * BM;
constexpr int kParts = 2;                    // softmax threads a row: each takes 64 keys of a tile
constexpr int kKeys = BN / kParts;
constexpr int kGroup = 128 * kParts;         // softmax threads of a query tile
constexpr int kSoftWarps = 2 * kGroup / 32;
constexpr int kThreads = 2 * kGroup + 128;
constexpr int kD = 64;
constexpr uint32_t kTile = kHalf;            // 128 x 64 bf16
constexpr int kStages = 4;                   // of K and of V
constexpr uint32_t kColP = 256;              // + 64 t
constexpr uint32_t kColO = 384;              // + 64 t
constexpr uint32_t kOffK = 4 * kTile;        // two Q buffers of two tiles first
constexpr uint32_t kOffV = kOffK + kStages * kTile;
constexpr uint32_t kOffO = kOffV + kStages * kTile;   // the output tiles on their way out
constexpr uint32_t kOffBar = kOffO + 2 * kTile;

// One unit as the scheduler publishes it; b < 0 means no more work.
struct UnitInfo {
    int b, head, q0;
    int j0, n;                   // key tiles j0 .. j0 + n - 1 (n = 0: no row has a key)
    int from[2], to[2];          // of those, the ones that query tile t needs: from <= j < to, counted from j0
    int lo_max[2], hi_min[2];    // keys [lo_max, hi_min) are allowed to every row of query tile t
    int valid, seen;             // valid length; prefix that all rows see
};

struct Smem64 {
    uint64_t q_full[2];                      // Q buffer loaded
    uint64_t q_empty[2];                     // its unit's score MMAs done (commit), and the other four roles have read
                                             // the unit's slot (a unit without keys gives them nothing else to do)
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t v_full[kStages], v_empty[kStages];
    uint64_t v_edge;                         // the tile that holds the valid length has arrived
    uint64_t s_full[2], s_free[2];           // S_t computed (commit) / loaded (one arrival a warp)
    uint64_t p_full[2], p_free[2];           // P_t written (one arrival a warp) / P.V done (commit)
    uint64_t unit_full[2];                   // unit slot published by the scheduler
    uint64_t steal_full[2];                  // answer to a request for another unit
    alignas(16) uint32_t steal[2][4];
    UnitInfo unit[2];
    uint32_t tmem_base;
    int abort_flag;
    float mx[2][kParts][BM];                 // the parts' tile maxima, exchanged when a row's maximum grows
};
constexpr size_t kSmemBytes = kOffBar + sizeof(Smem64);

// Unit u of the schedule (a whole warp): groups of kHeadGroup (batch, head) pairs, whose keys and values
// stay in L2, inside a group the query tiles from the last (longest under a causal mask) to the first.
__device__ __forceinline__ UnitInfo unit_of(const SpanAttnParams& p, int u, int lane) {
    const int planes = p.B * p.h;
    const int tiles = (p.Lq + kRowsUnit - 1) / kRowsUnit;
    const int grp = u / (kHeadGroup * tiles);
    const int g_heads = min(kHeadGroup, planes - grp * kHeadGroup);
    const int r = u - grp * kHeadGroup * tiles;
    const int qt = tiles - 1 - r / g_heads;
    const int plane = grp * kHeadGroup + r % g_heads;
    UnitInfo x;
    x.b = plane / p.h;
    x.head = plane - x.b * p.h;
    x.q0 = qt * kRowsUnit;
    x.valid = p.valid_lens != nullptr ? min(max(p.valid_lens[x.b], 0), p.Lk) : p.Lk;
    x.seen = p.prefix_lens != nullptr ? p.prefix_lens[x.b] : 0;
    int lo[2], hi[2];        // keys that some row of tile t may see
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = x.q0 + t * BM, last = min(first + BM, p.Lq) - 1;
        int lo_min = p.Lk, lo_max = 0, hi_min = p.Lk, hi_max = 0;
        if (p.spans == nullptr) {   // hi grows with i
            if (first <= last) {
                lo_min = 0;
                hi_min = interval_of(p, x.valid, x.seen, make_int2(0, p.Lk), first).y;
                hi_max = interval_of(p, x.valid, x.seen, make_int2(0, p.Lk), last).y;
            }
        } else {
            for (int i = first + lane; i <= last; i += 32) {
                const int2 iv = interval_of(p, x.valid, x.seen, span_of(p, x.b, i), i);
                lo_max = max(lo_max, iv.x);
                hi_min = min(hi_min, iv.y);
                if (iv.y > iv.x) {
                    lo_min = min(lo_min, iv.x);
                    hi_max = max(hi_max, iv.y);
                }
            }
            lo_max = __reduce_max_sync(0xffffffffu, lo_max);
            hi_min = __reduce_min_sync(0xffffffffu, hi_min);
            lo_min = __reduce_min_sync(0xffffffffu, lo_min);
            hi_max = __reduce_max_sync(0xffffffffu, hi_max);
        }
        lo[t] = lo_min;
        hi[t] = hi_max;
        x.lo_max[t] = lo_max;
        x.hi_min[t] = hi_min;
    }
    x.j0 = min(hi[0] > lo[0] ? lo[0] / BN : 0x7fffffff, hi[1] > lo[1] ? lo[1] / BN : 0x7fffffff);
    int end = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const bool any = hi[t] > lo[t];
        x.from[t] = any ? lo[t] / BN - x.j0 : 0;
        x.to[t] = any ? (hi[t] + BN - 1) / BN - x.j0 : 0;
        end = max(end, x.to[t]);
    }
    x.n = end;
    return x;
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1) span_attn_d64_kernel(const __grid_constant__ SpanAttnParams p,
                                                                    const __grid_constant__ SpanMaps maps) {
    constexpr int kOut = kD / kParts;            // output features of a softmax thread
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw;
    Smem64* sm = reinterpret_cast<Smem64*>(base + kOffBar);
    pdl_trigger();
    if ((smem_u32(base) & 1023u) != 0) {
        // the 128-byte-swizzled tiles need 1024-byte alignment: refuse rather than compute garbage
        pdl_wait();
        if (threadIdx.x == 0) atomicCAS(p.status, 0, 0x803);
        return;
    }
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->q_full[i], 1);
            mbar_init(&sm->q_empty[i], 5);
            mbar_init(&sm->unit_full[i], 1);
            mbar_init(&sm->steal_full[i], 1);
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->s_free[i], 4 * kParts);
            mbar_init(&sm->p_full[i], 4 * kParts);
            mbar_init(&sm->p_free[i], 1);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm->k_full[s], 1);
            mbar_init(&sm->k_empty[s], 1);
            mbar_init(&sm->v_full[s], 1);
            mbar_init(&sm->v_empty[s], 1);
        }
        mbar_init(&sm->v_edge, 1);
        sm->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.out);
    }
    if (warp == kSoftWarps + 1) {
        tmem_alloc(&sm->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem_base;
    volatile int* abort_flag = &sm->abort_flag;
    pdl_wait();   // the tensors and the mask parts come from earlier kernels

    if (warp >= kSoftWarps) {
        regs_dec<56>();
        if (warp == kSoftWarps) {
            // ------------------------------------------------ scheduler, Q and K loads
            int u = blockIdx.x;
            uint32_t gk = 0;       // K tiles issued so far
            int loaded = 0;        // units whose Q was
            for (int k = 0;; ++k, ++loaded) {
                const int qb = k & 1;
                // the score MMAs of unit k - 2 have read this Q buffer, and every role its slot
                if (k >= 2) mbar_wait(&sm->q_empty[qb], ((k >> 1) - 1) & 1, abort_flag, p.status, 0x830);
                if (k >= 1) {
                    const int a = (k - 1) & 1;
                    const bool ok = mbar_wait(&sm->steal_full[a], ((k - 1) >> 1) & 1, abort_flag, p.status, 0x831);
                    u = ok ? steal_answer(&sm->steal[a][0]) : -1;
                    fence_proxy_async_smem();   // the slot may take the answer after next
                }
                u = __shfl_sync(0xffffffffu, u, 0);
                if (__any_sync(0xffffffffu, u < 0 || *abort_flag != 0)) {
                    if (lane == 0) {
                        sm->unit[qb].b = -1;
                        mbar_arrive(&sm->unit_full[qb]);
                    }
                    break;
                }
                if (lane == 0) steal_request(&sm->steal[qb][0], &sm->steal_full[qb]);
                const UnitInfo x = unit_of(p, u, lane);
                if (lane == 0) {
                    sm->unit[qb] = x;
                    mbar_arrive(&sm->unit_full[qb]);
                    const int kvh = x.head / (p.h / p.h_kv);
                    mbar_arrive_expect_tx(&sm->q_full[qb], 2 * kTile);
                    for (int t = 0; t < 2; ++t)
                        tma_load_5d(&maps.q, &sm->q_full[qb], base + (2 * qb + t) * kTile, x.q0 + t * BM, at_h(p.q, x.head),
                                    at_b(p.q, x.b));
                    for (int j = 0; j < x.n; ++j, ++gk) {
                        const int s = gk % kStages;
                        mbar_wait(&sm->k_empty[s], ((gk / kStages) & 1) ^ 1, abort_flag, p.status, 0x832);
                        mbar_arrive_expect_tx(&sm->k_full[s], kTile);
                        tma_load_5d(&maps.k, &sm->k_full[s], base + kOffK + s * kTile, (x.j0 + j) * BN, at_h(p.k, kvh),
                                    at_b(p.k, x.b));
                    }
                }
                __syncwarp();
            }
            if (lane == 0 && *abort_flag) {
                drain_ring<kStages>(sm->k_full, gk);
                drain_ring<2>(sm->q_full, loaded);
                drain_ring<2>(sm->steal_full, loaded);
            }
        } else if (warp == kSoftWarps + 3) {
            // ------------------------------------------------ V loads
            uint32_t gv = 0, edges = 0;
            for (int k = 0;; ++k) {
                const int qb = k & 1;
                const bool ok = mbar_wait(&sm->unit_full[qb], (k >> 1) & 1, abort_flag, p.status, 0x833);
                const UnitInfo x = sm->unit[qb];
                if (!__all_sync(0xffffffffu, ok && x.b >= 0)) break;
                if (lane == 0) mbar_arrive(&sm->q_empty[qb]);
                const int kvh = x.head / (p.h / p.h_kv);
                for (int j = 0; j < x.n; ++j, ++gv) {
                    const int s = gv % kStages;
                    const int r0 = x.valid - (x.j0 + j) * BN;   // rows of the tile before the valid length
                    uint8_t* dst = base + kOffV + s * kTile;
                    mbar_wait(&sm->v_empty[s], ((gv / kStages) & 1) ^ 1, abort_flag, p.status, 0x834);
                    __syncwarp();
                    if (r0 >= BN || x.valid >= p.Lk) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sm->v_full[s], kTile);
                            tma_load_5d(&maps.v, &sm->v_full[s], dst, (x.j0 + j) * BN, at_h(p.v, kvh), at_b(p.v, x.b));
                        }
                    } else {
                        // values behind the valid length may be anything, and 0 * NaN is NaN: zeros in their place
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sm->v_edge, kTile);
                            tma_load_5d(&maps.v, &sm->v_edge, dst, (x.j0 + j) * BN, at_h(p.v, kvh), at_b(p.v, x.b));
                        }
                        mbar_wait(&sm->v_edge, edges++ & 1, abort_flag, p.status, 0x835);
                        __syncwarp();
                        for (uint32_t o = max(r0, 0) * 128 + lane * 16; o < kTile; o += 512)
                            st_shared_v4(smem_u32(dst) + o, 0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm->v_full[s]);
                    }
                }
            }
            if (lane == 0 && *abort_flag) {
                drain_ring<kStages>(sm->v_full, gv);
                if (edges > 0) drain(&sm->v_edge, (edges - 1) & 1);
            }
        } else if (warp == kSoftWarps + 1 && lane == 0) {
            // ------------------------------------------------ score MMAs: S_t(j) = Q_t K_j^T
            constexpr uint32_t idesc_s = idesc_bf16(BM, BN, false, false);
            const uint32_t k_addr = smem_u32(base + kOffK);
            uint32_t gk = 0, c[2] = {0, 0};   // K tiles used, score tiles issued for each query tile
            for (int k = 0;; ++k) {
                const int qb = k & 1;
                if (!mbar_wait(&sm->unit_full[qb], (k >> 1) & 1, abort_flag, p.status, 0x836)) break;
                const UnitInfo x = sm->unit[qb];
                if (x.b < 0) break;
                mbar_wait(&sm->q_full[qb], (k >> 1) & 1, abort_flag, p.status, 0x837);
                for (int j = 0; j < x.n; ++j, ++gk) {
                    const int s = gk % kStages;
                    mbar_wait(&sm->k_full[s], (gk / kStages) & 1, abort_flag, p.status, 0x838);
                    const uint32_t ka = k_addr + s * kTile;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j < x.from[t] || j >= x.to[t]) continue;
                        if (c[t] >= 1) mbar_wait(&sm->s_free[t], (c[t] - 1) & 1, abort_flag, p.status, 0x839);
                        tc_fence_after();
                        const uint32_t qa = smem_u32(base + (2 * qb + t) * kTile);
#pragma unroll
                        for (int kk = 0; kk < kD / 16; ++kk)
                            mma_ss(tmem + t * 128, sdesc_sw128(qa + kk * 32, 16, 1024), sdesc_sw128(ka + kk * 32, 16, 1024),
                                   idesc_s, kk > 0);
                        tc_commit(&sm->s_full[t]);
                        ++c[t];
                    }
                    tc_commit(&sm->k_empty[s]);
                }
                tc_commit(&sm->q_empty[qb]);
            }
        } else if (warp == kSoftWarps + 2 && lane == 0) {
            // ------------------------------------------------ P.V MMAs: O_t += P_t(j) V_j
            constexpr uint32_t idesc_o = idesc_bf16(BM, kD, false, true);
            const uint32_t v_addr = smem_u32(base + kOffV);
            uint32_t gv = 0, c[2] = {0, 0};
            for (int k = 0;; ++k) {
                const int qb = k & 1;
                if (!mbar_wait(&sm->unit_full[qb], (k >> 1) & 1, abort_flag, p.status, 0x83a)) break;
                const UnitInfo x = sm->unit[qb];
                if (x.b < 0) break;
                mbar_arrive(&sm->q_empty[qb]);
                for (int j = 0; j < x.n; ++j, ++gv) {
                    const int s = gv % kStages;
                    mbar_wait(&sm->v_full[s], (gv / kStages) & 1, abort_flag, p.status, 0x83b);
                    const uint32_t va = v_addr + s * kTile;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (j < x.from[t] || j >= x.to[t]) continue;
                        // P_t(j) written; for the first tile also: the previous unit's output has been read out of O_t
                        mbar_wait(&sm->p_full[t], c[t] & 1, abort_flag, p.status, 0x83c);
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)   // keys 16 kk .. 16 kk + 15: columns 8 kk ..
                            mma_ts(tmem + kColO + t * 64, tmem + kColP + t * 64 + kk * 8, sdesc_sw128(va + kk * 2048, kHalf, 1024),
                                   idesc_o, (j > x.from[t] || kk > 0) ? 1u : 0u);
                        tc_commit(&sm->p_free[t]);
                        ++c[t];
                    }
                    tc_commit(&sm->v_empty[s]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        named_bar_sync(3, kThreads);
        if (warp == kSoftWarps + 1) {
            __syncwarp();
            tc_fence_after();
            tmem_dealloc(tmem, kTmemCols);
        }
    } else {
        regs_inc<104>();
        // ------------------------------------------------ softmax: thread (t, h, row), keys 64 h .. 64 h + 63 of a tile
        const int t = warp / (kSoftWarps / 2), h = (warp >> 2) % kParts, q = warp & 3;
        const int row = q * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t s_tmem = tmem + lane_off + t * 128 + h * kKeys;
        const uint32_t p_tmem = tmem + lane_off + kColP + t * 64 + h * (kKeys / 2);
        const uint32_t o_tmem = tmem + lane_off + kColO + t * 64 + h * kOut;     // this part's output features
        const int pair = 4 + t * 4 + q;                                          // barrier of the warps that share rows
        const bool first = warp % (kSoftWarps / 2) == 0 && lane == 0;            // one thread of the group
        const float scale_log2 = p.scale * kLog2e;
        const TanhForm<false> capped(p.cap > 0.0f ? p.scale / p.cap : 1.0f, p.cap * kLog2e);
        uint32_t g = 0;   // score tiles of this query tile consumed so far
        bool ok = mbar_wait(&sm->unit_full[0], 0, abort_flag, p.status, 0x83d);
        UnitInfo x = sm->unit[0];
        int2 span = ok && x.b >= 0 ? span_of(p, x.b, x.q0 + t * BM + row) : make_int2(0, 0);
        for (int k = 0;; ++k) {
            const int qb = k & 1;
            __syncwarp();
            // every thread of the group takes the same decision (a give-up in one thread stops all)
            if (!named_bar_and(1 + t, kGroup, ok && x.b >= 0)) break;
            if (first) mbar_arrive(&sm->q_empty[qb]);      // all of the group have read the slot
            const int b = x.b, head = x.head, q0 = x.q0 + t * BM, j0 = x.j0;
            const int from = t ? x.from[1] : x.from[0], to = t ? x.to[1] : x.to[0];
            const int lo_max = t ? x.lo_max[1] : x.lo_max[0], hi_min = t ? x.hi_min[1] : x.hi_min[0];
            const int2 iv = interval_of(p, x.valid, x.seen, span, q0 + row);
            const float slope = kMode == kGeneral && p.slopes != nullptr ? p.slopes[head] * kLog2e : 0.0f;
            float m = -CUDART_INF_F;   // the row's reference max (log2 units), common to its parts
            float l = 0.0f;            // this part's share of the row sum
            for (int j = from; j < to; ++j, ++g) {
                mbar_wait(&sm->s_full[t], g & 1, abort_flag, p.status, 0x83e);
                __syncwarp();
                tc_fence_after();
                uint32_t u[kKeys];
                tmem_ld_x64(s_tmem, u);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->s_free[t]);
                const int k0 = (j0 + j) * BN + h * kKeys;   // first key of this part
                const bool edge = k0 < lo_max || k0 + kKeys > hi_min;
                float sc = 1.0f;
                if constexpr (kMode == kPlain) {
                    if (edge) {
                        scale_scores(u, scale_log2);
                    } else {
                        sc = scale_log2;
                    }
                } else {
                    if (p.cap > 0.0f) cap_scores(u, capped, 0.0f);
                    const float by = p.cap > 0.0f ? 1.0f : scale_log2;
                    if (slope != 0.0f) bias_scores(u, by, static_cast<float>(q0 + row + p.q_offset - k0), slope);
                    else if (by != 1.0f) scale_scores(u, by);
                }
                if (edge) {
                    const uint32_t first = iv.x - k0, many = max(iv.y - iv.x, 0);   // keys first .. first + many - 1 of u
#pragma unroll
                    for (int c = 0; c < kKeys; ++c)
                        if (static_cast<uint32_t>(c) - first >= many) u[c] = __float_as_uint(-CUDART_INF_F);
                }
                float alpha = 1.0f;
                bool grow = false;
                float a4[4];
#pragma unroll
                for (int c2 = 0; c2 < 4; ++c2) {
                    float a = fmax3(__uint_as_float(u[16 * c2]), __uint_as_float(u[16 * c2 + 1]),
                                    __uint_as_float(u[16 * c2 + 2]));
#pragma unroll
                    for (int e = 3; e < 15; e += 2)
                        a = fmax3(a, __uint_as_float(u[16 * c2 + e]), __uint_as_float(u[16 * c2 + e + 1]));
                    a4[c2] = fmaxf(a, __uint_as_float(u[16 * c2 + 15]));
                }
                // The reference moves only when the tile passes it by 2^8 (or holds the row's first keys); whether any
                // row of these 32 does is agreed by a barrier of the two warps, and only then are the parts'
                // maxima exchanged.
                const float mth = fmaxf(fmax3(a4[0], a4[1], a4[2]), a4[3]) * sc;   // this part's tile max (log2 units)
                if (named_bar_or(pair, 32 * kParts, mth > m + kRescaleThreshold)) {
                    sm->mx[t][h][row] = mth;
                    named_bar_sync(pair, 32 * kParts);
                    const float top = fmaxf(mth, sm->mx[t][h ^ 1][row]);
                    if (top > m + kRescaleThreshold) {
                        grow = m != -CUDART_INF_F;
                        alpha = ex2_approx(m - top);   // 0 for the first keys
                        l *= alpha;
                        m = top;
                    }
                }
                // with no key of the row yet (m = -inf) every weight is exp2(-inf) = 0
                const float mref = (m == -CUDART_INF_F) ? 0.0f : m;
                const float2 sc2 = make_float2(sc, sc);
                const float2 nm2 = make_float2(-mref, -mref);
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[kKeys / 2];
#pragma unroll
                for (int c = 0; c < kKeys / 2; ++c) {
                    float2 e2 = make_float2(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1]));
                    if constexpr (kMode == kPlain) e2 = ffma2(e2, sc2, nm2);
                    if constexpr (kMode == kGeneral) e2 = fadd2(e2, nm2);
                    e2.x = ex2_approx(e2.x);
                    e2.y = ex2_approx(e2.y);
                    acc[c & 1] = fadd2(acc[c & 1], e2);
                    // the weights are rounded to bf16 for the product; the sum takes them unrounded
                    pk[c] = pack_bf16x2(e2.x, e2.y);
                }
                const float2 s2 = fadd2(acc[0], acc[1]);
                l += s2.x + s2.y;
                // P_t and O_t are free once P.V(g - 1) has completed
                if (g >= 1) {
                    mbar_wait(&sm->p_free[t], (g - 1) & 1, abort_flag, p.status, 0x83f);
                    __syncwarp();
                    tc_fence_after();
                }
                if (j > from && __any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int q4 = 0; q4 < kOut / 16; ++q4) {
                        uint32_t o[16];
                        tmem_ld_x16(o_tmem + q4 * 16, o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tmem_st_x16(o_tmem + q4 * 16, o);
                    }
                }
#pragma unroll
                for (int q4 = 0; q4 < kKeys / 32; ++q4)
                    tmem_st_x16_nowait(p_tmem + q4 * 16, *reinterpret_cast<const uint32_t(*)[16]>(&pk[16 * q4]));
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->p_full[t]);
            }
            // The next unit's slot and spans are read now: their latency passes behind the output.
            const int nb = (k + 1) & 1;
            ok = mbar_wait(&sm->unit_full[nb], ((k + 1) >> 1) & 1, abort_flag, p.status, 0x840);
            x = sm->unit[nb];
            if (ok && x.b >= 0) span = span_of(p, x.b, x.q0 + t * BM + row);
            // ---------------- output: thread (h, row) writes its features of O / (l_0 + l_1). The output tile's buffer first
            // carries l_h of both parts and every row; the previous unit's store has read it.
            uint8_t* obuf = base + kOffO + t * kTile;
            if (first) tma_store_wait_read();
            named_bar_sync(1 + t, kGroup);
            float* lsum = reinterpret_cast<float*>(obuf);
            lsum[h * BM + row] = l;
            named_bar_sync(pair, 32 * kParts);
            const float L = lsum[row] + lsum[BM + row];
            const bool none = L == 0.0f;              // no key: a row of zeros, O may hold 0 * NaN from the tile's other rows' keys
            const float inv = L > 0.0f ? 1.0f / L : L;   // NaN stays
            uint32_t o[kOut];
            if (to > from) {
                mbar_wait(&sm->p_free[t], (g - 1) & 1, abort_flag, p.status, 0x842);   // the last P.V completes O
                __syncwarp();
                tc_fence_after();
                tmem_ld_x32(o_tmem, o);
            } else {
#pragma unroll
                for (int c = 0; c < kOut; ++c) o[c] = 0u;
            }
            named_bar_sync(1 + t, kGroup);   // every thread has read the sums the staging overwrites
#pragma unroll
            for (int ch = 0; ch < kOut / 8; ++ch) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = none ? 0u : pack_bf16x2(__uint_as_float(o[ch * 8 + 2 * e]) * inv, __uint_as_float(o[ch * 8 + 2 * e + 1]) * inv);
                st_shared_v4(smem_u32(obuf) + row * 128 + (((h * (kOut / 8) + ch) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();   // O has been read: the next unit's first P.V may overwrite it
            named_bar_sync(1 + t, kGroup);
            if (first && !*abort_flag && q0 < p.Lq) {
                asm volatile(
                    "cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %2, %4, %5}], [%1];" ::"l"(
                        reinterpret_cast<uint64_t>(&maps.out)),
                    "r"(smem_u32(obuf)), "r"(0), "r"(q0), "r"(head), "r"(b)
                    : "memory");
                tma_store_commit();
            }
        }
        if (first) tma_store_wait_all();
        tc_fence_before();
        named_bar_sync(3, kThreads);
    }
}

template <int kMode>
cudaError_t launch_mode(const SpanAttnParams& p, const SpanMaps& maps, cudaStream_t s) {
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(span_attn_d64_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.h * ((p.Lq + kRowsUnit - 1) / kRowsUnit));
    return launch_pdl(span_attn_d64_kernel<kMode>, dim3(grid), dim3(kThreads), kSmemBytes, s, p, maps);
}

}  // namespace

cudaError_t launch_span_attn_d64(const SpanAttnParams& p, const SpanMaps& maps, int mode, cudaStream_t s) {
    return mode == kPlain ? launch_mode<kPlain>(p, maps, s) : launch_mode<kGeneral>(p, maps, s);
}

}  // namespace mha
