// attn_span.cu -- attention under span masks; document spans.
//
// Grouped heads over strided tensors, capped and biased scores, and masks that leave each query one
// interval of keys (document spans, prefix, causal, valid length: their intersection is an interval
// [lo, hi)), so a tile is either inside every row's interval, and not masked at all, or needs two comparisons a
// score. An empty interval gives a row of zeros.
//
//   m, l, O: running maximum (log2 units), sum and output of a row over the key tiles seen so far; a tile's weights
//   are exp2(s - m), O and l are rescaled when m grows by more than 8 (exact: the final O / l uses the same m).
//
// Tensor- and issue-bound: 4 d_k flop a (query, key) pair on tcgen05, one exponential and about seven instructions a
// score on the softmax warps. Unit of work: 128 query rows of one head. Warps: 16 softmax warps, four threads a row
// (with two, 4 x 8192 causal took 389 us instead of 361 us: eight warps do not cover their own latencies), and four
// that schedule and load Q and K, issue score MMAs, issue P.V MMAs, and load V. Scores and weights are double-buffered
// in tensor memory, so the score MMAs of tile j + 1 run during the softmax of tile j, and the next unit's loads and
// first scores run during this unit's last tiles and output. Registers: 96 a thread at launch; the last warpgroup drops to 56 and the
// softmax warps rise to 104 (128 * 56 + 512 * 104 = 60416 <= 640 * 96).
// Few units (few queries over long keys): the CTAs of a cluster share one, see pieces_of.
// Measured, 4 x 8192 causal, 8 heads: 361 us, 1522 TFLOP/s (0.79 of measured bf16 peak; all keys 0.84), capped 476 us, with a
// distance bias 471 us.
#include <algorithm>
#include <cfloat>

#include "attn_span.cuh"

namespace mha {
namespace {

constexpr int BM = 128;          // queries of a unit
constexpr int kParts = 4;        // softmax threads a query row: each takes 32 keys of a tile
constexpr int kKeys = BN / kParts;
constexpr int kSoftWarps = 4 * kParts;
constexpr int kSoft = 32 * kSoftWarps;
constexpr int kThreads = kSoft + 128;
// Unit slots. Unit k + kSlots is published after the score MMAs of unit k + kSlots - 2, for which the softmax has begun
// unit k + kSlots - 4 and so ended unit k + kSlots - 5, whose P.V are done: from five slots on, every role has read
// unit k's by then.
constexpr int kSlots = 8;
// d_k = 64: from here on the kernel of two query tiles a unit (4 x L causal, 16 heads: L = 1024 31.2 against 28.7 us,
// 1536 44.0 against 45.1 us, 4096 169 against 190 us), where there are more units of one tile than SMs (1024 queries over
// 4096 keys: 24 heads 42.5 against 48.4 us, 19 heads, all of whose units run at once, 41.6 against 27.7 us).
constexpr int kLongKeys = 1536;
constexpr uint32_t kColS = 0;                // + 128 b: score buffers S_0, S_1
constexpr uint32_t kColP = 256;              // + 64 b + 16 h: weight buffers P_0, P_1
constexpr uint32_t kColO = 384;              // output accumulator, d_k features

// One unit as the scheduler publishes it; n == 0 means no more work.
struct UnitInfo {
    int b, head, q0;
    int j0, n;             // key tiles j0 .. j0 + n - 1
    int lo_max, hi_min;    // keys [lo_max, hi_min) are allowed to every row of the unit
    int valid, seen;       // valid length; prefix that all rows see
};

// Key tile of step j of n. Under a causal mask a distance bias raises the scores towards the query: from the last tile to
// the first the maximum stands after the first steps, from the first to the last it grows with most tiles and O is
// rescaled as often (4 x 8192, 8 heads of 128: 471 against 592 us, capped too 594 against 716 us). With two query tiles a
// unit the order changes nothing (819 against 814 us), and the other modes keep the plain count, which costs less.
template <int kMode>
__device__ __forceinline__ int tile_of(const SpanAttnParams& p, int j, int n) {
    if constexpr (kMode == kPlain || kMode == kCapped) return j;
    return p.slopes != nullptr && p.causal ? n - 1 - j : j;
}

template <int kD>
struct Tiles {
    static constexpr int kSlabs = kD / 64;
    static constexpr uint32_t kTile = kSlabs * kHalf;       // 128 x d_k bf16
    static constexpr int kStagesK = kD == 128 ? 2 : 4;
    static constexpr int kStagesV = kD == 128 ? 2 : 4;
    static constexpr uint32_t kOffK = 2 * kTile;            // two Q buffers first
    static constexpr uint32_t kOffV = kOffK + kStagesK * kTile;
    static constexpr uint32_t kOffO = kOffV + kStagesV * kTile;   // the output tile on its way out
    static constexpr uint32_t kOffBar = kOffO + kTile;
};

struct SmemSpan {
    uint64_t q_full[2], q_empty[2];          // Q buffer loaded / read by the unit's last score MMA (commit)
    uint64_t k_full[4], k_empty[4];
    uint64_t v_full[4], v_empty[4];
    uint64_t v_edge;                         // the tile that holds the valid length has arrived
    uint64_t s_full[2];                      // score buffer b holds S(j) (commit)
    uint64_t s_free[2];                      // S(j) of buffer b loaded (one arrival a softmax warp)
    uint64_t p_full[2];                      // P(j) of weight buffer b written (one arrival a softmax warp)
    uint64_t p_free[2];                      // P.V(j) of weight buffer b done (commit)
    uint64_t unit_full[kSlots];              // unit slot published by the scheduler
    uint64_t steal_full[2];                  // answer to a request for another unit
    alignas(16) uint32_t steal[2][4];
    UnitInfo unit[kSlots];
    uint32_t tmem_base;
    int abort_flag;
    float mx[kParts][BM];                    // the parts' tile maxima, exchanged when a row's maximum grows; kSplit, at the end:
                                             // maximum [0] and sum [1] of this CTA's part
};
template <int kD>
constexpr size_t smem_bytes() { return Tiles<kD>::kOffBar + sizeof(SmemSpan); }

// Place of unit u of the schedule: groups of kHeadGroup (batch, head) pairs, whose keys and values
// stay in L2, inside a group the query tiles from the last (longest under a causal mask) to the first.
__device__ __forceinline__ UnitInfo place_of(const SpanAttnParams& p, int u) {
    const int planes = p.B * p.h;
    const int tiles = (p.Lq + BM - 1) / BM;
    const int grp = u / (kHeadGroup * tiles);
    const int g_heads = min(kHeadGroup, planes - grp * kHeadGroup);
    const int r = u - grp * kHeadGroup * tiles;
    const int qt = tiles - 1 - r / g_heads;
    const int plane = grp * kHeadGroup + r % g_heads;
    UnitInfo x;
    x.b = plane / p.h;
    x.head = plane - x.b * p.h;
    x.q0 = qt * BM;
    return x;
}

// Unit u (a whole warp).
__device__ __forceinline__ UnitInfo unit_of(const SpanAttnParams& p, int u, int lane) {
    UnitInfo x = place_of(p, u);
    x.valid = p.valid_lens != nullptr ? min(max(p.valid_lens[x.b], 0), p.Lk) : p.Lk;
    x.seen = p.prefix_lens != nullptr ? p.prefix_lens[x.b] : 0;
    int lo_min = p.Lk, lo_max = 0, hi_min = p.Lk, hi_max = 0;
    const int last = min(x.q0 + BM, p.Lq) - 1;
    if (p.spans == nullptr) {   // hi grows with i
        const int2 first = interval_of(p, x.valid, x.seen, make_int2(0, p.Lk), x.q0);
        lo_min = 0;
        hi_min = first.y;
        hi_max = interval_of(p, x.valid, x.seen, make_int2(0, p.Lk), last).y;
    } else {
        for (int i = x.q0 + lane; i <= last; i += 32) {
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
    // no row has a key: one tile all the same, which the masks leave without weight
    const bool any = hi_max > lo_min;
    x.j0 = any ? lo_min / BN : 0;
    x.n = any ? (hi_max + BN - 1) / BN - x.j0 : 1;
    x.lo_max = lo_max;
    x.hi_min = hi_min;
    return x;
}

// kSplit: the CTAs of a cluster share a unit, each with its piece of the key tiles; they join their parts through one
// another's shared memory.
template <int kD, int kMode, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) span_attn_kernel(const __grid_constant__ SpanAttnParams p,
                                                                const __grid_constant__ SpanMaps maps) {
    using G = Tiles<kD>;
    constexpr uint32_t kTile = G::kTile;
    constexpr int kOut = kD / kParts;      // output features of a softmax thread
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw;
    SmemSpan* sm = reinterpret_cast<SmemSpan*>(base + G::kOffBar);
    const int pieces = kSplit ? p.pieces : 1, piece = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
    pdl_trigger();
    if ((smem_u32(base) & 1023u) != 0) {
        // the 128-byte-swizzled tiles need 1024-byte alignment: refuse rather than compute garbage (all CTAs of a
        // cluster alike)
        pdl_wait();
        if (threadIdx.x == 0) atomicCAS(p.status, 0, 0x802);
        return;
    }
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->q_full[i], 1);
            mbar_init(&sm->q_empty[i], 1);
            mbar_init(&sm->steal_full[i], 1);
            mbar_init(&sm->s_full[i], 1);
            mbar_init(&sm->s_free[i], kSoftWarps);
            mbar_init(&sm->p_full[i], kSoftWarps);
            mbar_init(&sm->p_free[i], 1);
        }
        for (int s = 0; s < G::kStagesK; ++s) {
            mbar_init(&sm->k_full[s], 1);
            mbar_init(&sm->k_empty[s], 1);
        }
        for (int s = 0; s < G::kStagesV; ++s) {
            mbar_init(&sm->v_full[s], 1);
            mbar_init(&sm->v_empty[s], 1);
        }
        for (int s = 0; s < kSlots; ++s) mbar_init(&sm->unit_full[s], 1);
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
            int u = blockIdx.x / pieces;
            uint32_t gk = 0;       // K tiles issued so far
            int loaded = 0;        // units whose Q was
            for (int k = 0;; ++k, ++loaded) {
                const int qb = k & 1;
                // the score MMAs of unit k - 2 have read this Q buffer
                if (k >= 2) mbar_wait(&sm->q_empty[qb], ((k >> 1) - 1) & 1, abort_flag, p.status, 0x810);
                if (kSplit && k >= 1) {
                    u = -1;
                } else if (k >= 1) {
                    const int a = (k - 1) & 1;
                    const bool ok = mbar_wait(&sm->steal_full[a], ((k - 1) >> 1) & 1, abort_flag, p.status, 0x811);
                    u = ok ? steal_answer(&sm->steal[a][0]) : -1;
                    fence_proxy_async_smem();   // the slot may take the answer after next
                }
                u = __shfl_sync(0xffffffffu, u, 0);
                if (__any_sync(0xffffffffu, u < 0 || *abort_flag != 0)) {
                    if (lane == 0) {
                        sm->unit[k % kSlots].n = 0;
                        mbar_arrive(&sm->unit_full[k % kSlots]);
                    }
                    break;
                }
                if (!kSplit && lane == 0) steal_request(&sm->steal[qb][0], &sm->steal_full[qb]);
                UnitInfo x = unit_of(p, u, lane);
                if constexpr (kSplit) {
                    const int first = static_cast<int>(static_cast<int64_t>(x.n) * piece / pieces);
                    x.n = static_cast<int>(static_cast<int64_t>(x.n) * (piece + 1) / pieces) - first;
                    x.j0 += first;
                    if (x.n == 0) {   // fewer tiles than pieces
                        if (lane == 0) {
                            sm->unit[0].n = 0;
                            mbar_arrive(&sm->unit_full[0]);
                        }
                        break;
                    }
                }
                if (lane == 0) {
                    sm->unit[k % kSlots] = x;
                    mbar_arrive(&sm->unit_full[k % kSlots]);
                    const int kvh = x.head / (p.h / p.h_kv);
                    mbar_arrive_expect_tx(&sm->q_full[qb], kTile);
                    tma_load_5d(&maps.q, &sm->q_full[qb], base + qb * kTile, x.q0, at_h(p.q, x.head),
                                at_b(p.q, x.b));
                    for (int j = 0; j < x.n; ++j, ++gk) {
                        const int s = gk % G::kStagesK;
                        mbar_wait(&sm->k_empty[s], ((gk / G::kStagesK) & 1) ^ 1, abort_flag, p.status, 0x812);
                        mbar_arrive_expect_tx(&sm->k_full[s], kTile);
                        tma_load_5d(&maps.k, &sm->k_full[s], base + G::kOffK + s * kTile,
                                    (x.j0 + tile_of<kMode>(p, j, x.n)) * BN,
                                    at_h(p.k, kvh), at_b(p.k, x.b));
                    }
                }
                __syncwarp();
            }
            if (lane == 0 && *abort_flag) {
                drain_ring<G::kStagesK>(sm->k_full, gk);
                drain_ring<2>(sm->q_full, loaded);
                if (!kSplit) drain_ring<2>(sm->steal_full, loaded);
            }
        } else if (warp == kSoftWarps + 3) {
            // ------------------------------------------------ V loads
            uint32_t gv = 0, edges = 0;
            for (int k = 0;; ++k) {
                const bool ok = mbar_wait(&sm->unit_full[k % kSlots], (k / kSlots) & 1, abort_flag, p.status, 0x813);
                const UnitInfo x = sm->unit[k % kSlots];
                if (!__all_sync(0xffffffffu, ok && x.n > 0)) break;
                const int kvh = x.head / (p.h / p.h_kv);
                for (int j = 0; j < x.n; ++j, ++gv) {
                    const int s = gv % G::kStagesV;
                    const int key0 = (x.j0 + tile_of<kMode>(p, j, x.n)) * BN;
                    const int r0 = x.valid - key0;   // rows of the tile before the valid length
                    uint8_t* dst = base + G::kOffV + s * kTile;
                    mbar_wait(&sm->v_empty[s], ((gv / G::kStagesV) & 1) ^ 1, abort_flag, p.status, 0x814);
                    __syncwarp();
                    if (r0 >= BN || x.valid >= p.Lk) {
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sm->v_full[s], kTile);
                            tma_load_5d(&maps.v, &sm->v_full[s], dst, key0, at_h(p.v, kvh), at_b(p.v, x.b));
                        }
                    } else {
                        // values behind the valid length may be anything, and 0 * NaN is NaN: zeros in their place
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&sm->v_edge, kTile);
                            tma_load_5d(&maps.v, &sm->v_edge, dst, key0, at_h(p.v, kvh), at_b(p.v, x.b));
                        }
                        mbar_wait(&sm->v_edge, edges++ & 1, abort_flag, p.status, 0x815);
                        __syncwarp();
                        for (int sl = 0; sl < G::kSlabs; ++sl)
                            for (uint32_t o = max(r0, 0) * 128 + lane * 16; o < kHalf; o += 512)
                                st_shared_v4(smem_u32(dst + sl * kHalf) + o, 0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm->v_full[s]);
                    }
                }
            }
            if (lane == 0 && *abort_flag) {
                drain_ring<G::kStagesV>(sm->v_full, gv);
                if (edges > 0) drain(&sm->v_edge, (edges - 1) & 1);
            }
        } else if (warp == kSoftWarps + 1 && lane == 0) {
            // ------------------------------------------------ score MMAs: S(j) = Q K_j^T
            constexpr uint32_t idesc_s = idesc_bf16(BM, BN, false, false);
            const uint32_t k_addr = smem_u32(base + G::kOffK);
            uint32_t gk = 0;   // score tiles issued so far
            for (int k = 0;; ++k) {
                const int qb = k & 1;
                if (!mbar_wait(&sm->unit_full[k % kSlots], (k / kSlots) & 1, abort_flag, p.status, 0x816)) break;
                const int n = sm->unit[k % kSlots].n;
                if (n == 0) break;
                const uint32_t qa = smem_u32(base + qb * kTile);
                mbar_wait(&sm->q_full[qb], (k >> 1) & 1, abort_flag, p.status, 0x817);
                for (int j = 0; j < n; ++j, ++gk) {
                    const int s = gk % G::kStagesK;
                    mbar_wait(&sm->k_full[s], (gk / G::kStagesK) & 1, abort_flag, p.status, 0x818);
                    // buffer gk mod 2 is free once all softmax warps have loaded score tile gk - 2
                    const int sb = gk & 1;
                    if (gk >= 2) mbar_wait(&sm->s_free[sb], ((gk >> 1) - 1) & 1, abort_flag, p.status, 0x819);
                    tc_fence_after();
                    const uint32_t ka = k_addr + s * kTile;
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                        mma_ss(tmem + kColS + sb * 128, sdesc_sw128(qa + off, 16, 1024), sdesc_sw128(ka + off, 16, 1024),
                               idesc_s, kk > 0);
                    }
                    tc_commit(&sm->s_full[sb]);
                    tc_commit(&sm->k_empty[s]);
                }
                tc_commit(&sm->q_empty[qb]);
            }
        } else if (warp == kSoftWarps + 2 && lane == 0) {
            // ------------------------------------------------ P.V MMAs: O += P(j) V_j
            constexpr uint32_t idesc_o = idesc_bf16(BM, kD, false, true);
            const uint32_t v_addr = smem_u32(base + G::kOffV);
            uint32_t gv = 0;   // P.V steps issued so far
            for (int k = 0;; ++k) {
                if (!mbar_wait(&sm->unit_full[k % kSlots], (k / kSlots) & 1, abort_flag, p.status, 0x81a)) break;
                const int n = sm->unit[k % kSlots].n;
                if (n == 0) break;
                for (int j = 0; j < n; ++j, ++gv) {
                    const int s = gv % G::kStagesV;
                    mbar_wait(&sm->v_full[s], (gv / G::kStagesV) & 1, abort_flag, p.status, 0x81b);
                    // P(j) written; for j = 0 also: the previous unit's output has been read out of O
                    mbar_wait(&sm->p_full[gv & 1], (gv >> 1) & 1, abort_flag, p.status, 0x81c);
                    tc_fence_after();
                    const uint32_t va = v_addr + s * kTile;
                    const uint32_t pa = tmem + kColP + (gv & 1) * 64;   // keys 16 kk .. 16 kk + 15: columns 8 kk ..
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + kColO, pa + kk * 8, sdesc_sw128(va + kk * 2048, kHalf, 1024), idesc_o,
                               (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(&sm->p_free[gv & 1]);
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
        if constexpr (kSplit) {   // the softmax warps' two
            __syncwarp();
            cluster_sync_all();
            cluster_sync_all();
        }
    } else {
        regs_inc<104>();
        // ------------------------------------------------ softmax: thread (h, row), keys 32 h .. 32 h + 31 of a tile
        const int h = warp >> 2;
        const int q = warp & 3;   // lane quarter; warps q, q + 4, ... hold the parts of the same rows
        const int row = q * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t s_tmem = tmem + lane_off + kColS + h * kKeys;          // + 128 b
        const uint32_t p_tmem = tmem + lane_off + kColP + h * (kKeys / 2);    // + 64 b
        const uint32_t o_tmem = tmem + lane_off + kColO + h * kOut;           // this part's output features
        const float scale_log2 = p.scale * kLog2e;
        const float inv_scale = 1.0f / fabsf(scale_log2);
        const TanhForm<kMode == kSingle> capped(p.cap > 0.0f ? p.scale / p.cap : 1.0f, p.cap * kLog2e);
        uint32_t g = 0;   // score tiles consumed so far
        bool ok = mbar_wait(&sm->unit_full[0], 0, abort_flag, p.status, 0x81d);
        UnitInfo x = sm->unit[0];
        int2 span = ok && x.n > 0 ? span_of(p, x.b, x.q0 + row) : make_int2(0, 0);
        // kSplit: this CTA's part, [row][kPitch], in place of the key and value tiles
        constexpr int kPitch = part_pitch(kD);
        float* const part = reinterpret_cast<float*>(base + G::kOffK);
        static_assert(BM * kPitch * 4 <= static_cast<int>(G::kOffO - G::kOffK), "a part fits the tiles");
        if (kSplit && h == 0) {
            sm->mx[0][row] = -CUDART_INF_F;
            sm->mx[1][row] = 0.0f;
        }
        for (int k = 0;; ++k) {
            __syncwarp();
            // every softmax thread takes the same decision (a give-up in one thread stops all)
            if (!named_bar_and(1, kSoft, ok && x.n > 0)) break;
            const int n = x.n, q0 = x.q0, b = x.b, head = x.head;
            const int2 iv = interval_of(p, x.valid, x.seen, span, q0 + row);
            const float slope = kMode >= kGeneral && p.slopes != nullptr ? p.slopes[head] * kLog2e : 0.0f;
            float m = -CUDART_INF_F;   // the row's reference max (log2 units), common to its parts
            float mref = 0.0f;         // m, or 0 while it is -inf
            float far = -1.0f;         // kCapped: (u before the cap)^2 up to which no score passes the reference by 2^8
            float l = 0.0f;            // this part's share of the row sum
            for (int j = 0; j < n; ++j, ++g) {
                const uint32_t sb = g & 1;
                mbar_wait(&sm->s_full[sb], (g >> 1) & 1, abort_flag, p.status, 0x81e);
                __syncwarp();
                tc_fence_after();
                uint32_t u[kKeys];
                tmem_ld_x32(s_tmem + sb * 128, u);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->s_free[sb]);
                const int k0 = (x.j0 + tile_of<kMode>(p, j, n)) * BN + h * kKeys;   // first key of this part
                const bool edge = k0 < x.lo_max || k0 + kKeys > x.hi_min;
                float sc = 1.0f;
                float farthest = 0.0f;
                if constexpr (kMode == kPlain) {
                    if (edge) {
                        scale_scores(u, scale_log2);
                    } else {
                        sc = scale_log2;
                    }
                } else if constexpr (kMode == kCapped) {
                    farthest = cap_scores(u, capped, mref);
                } else {
                    if (kMode == kSingle || p.cap > 0.0f) cap_scores(u, capped, 0.0f);
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
                auto tile_max = [&] {
                    float a2[2];
#pragma unroll
                    for (int c2 = 0; c2 < 2; ++c2) {
                        float a = fmax3(__uint_as_float(u[16 * c2]), __uint_as_float(u[16 * c2 + 1]),
                                        __uint_as_float(u[16 * c2 + 2]));
#pragma unroll
                        for (int e = 3; e < 15; e += 2)
                            a = fmax3(a, __uint_as_float(u[16 * c2 + e]), __uint_as_float(u[16 * c2 + e + 1]));
                        a2[c2] = fmaxf(a, __uint_as_float(u[16 * c2 + 15]));
                    }
                    return fmaxf(a2[0], a2[1]) * sc;   // log2 units
                };
                // The largest of the parts' values
                auto exchange = [&](float mine) {
                    sm->mx[h][row] = mine;
                    named_bar_sync(4 + q, 32 * kParts);
#pragma unroll
                    for (int o = 1; o < kParts; ++o) mine = fmaxf(mine, sm->mx[(h + o) % kParts][row]);
                    return mine;
                };
                // The reference moves only when the tile passes it by 2^8 (or holds the row's first keys); whether any
                // row of these 32 does is agreed by a barrier of the four warps, and only then are the parts'
                // maxima exchanged.
                if constexpr (kMode == kCapped) {
                    // u is relative to the reference. No score passes it by 2^8 where all |u| before the cap are below
                    // `far`, so only otherwise is the maximum itself formed.
                    if (named_bar_or(4 + q, 32 * kParts, farthest > far)) {
                        const float top = exchange(tile_max());
                        if (top > (m == -CUDART_INF_F ? -CUDART_INF_F : kRescaleThreshold)) {
                            grow = m != -CUDART_INF_F;
                            alpha = grow ? ex2_approx(-top) : 0.0f;
                            l *= alpha;
                            mref += top;
                            m = mref;
                            const float reach = fmaxf(m + kRescaleThreshold, 0.0f) * inv_scale;
                            far = m + kRescaleThreshold < 0.0f ? -1.0f : m + kRescaleThreshold > capped.top ? CUDART_INF_F : fminf(reach * reach, FLT_MAX);
#pragma unroll
                            for (int c = 0; c < kKeys; ++c) u[c] = __float_as_uint(__uint_as_float(u[c]) - top);
                        }
                    }
                } else {
                    const float mth = tile_max();   // of this part
                    if (named_bar_or(4 + q, 32 * kParts, mth > m + kRescaleThreshold)) {
                        const float top = exchange(mth);
                        if (top > m + kRescaleThreshold) {
                            grow = m != -CUDART_INF_F;
                            alpha = ex2_approx(m - top);   // 0 for the first keys
                            l *= alpha;
                            m = top;
                        }
                    }
                    // with no key of the row yet (m = -inf) every weight is exp2(-inf) = 0
                    mref = (m == -CUDART_INF_F) ? 0.0f : m;
                }
                const float2 sc2 = make_float2(sc, sc);
                const float2 nm2 = make_float2(-mref, -mref);
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pk[kKeys / 2];
#pragma unroll
                for (int c = 0; c < kKeys / 2; ++c) {
                    float2 e2 = make_float2(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1]));
                    if constexpr (kMode == kPlain) e2 = ffma2(e2, sc2, nm2);
                    if constexpr (kMode >= kGeneral) e2 = fadd2(e2, nm2);
                    e2.x = ex2_approx(e2.x);
                    e2.y = ex2_approx(e2.y);
                    acc[c & 1] = fadd2(acc[c & 1], e2);
                    // the weights are rounded to bf16 for the product; the sum takes them unrounded
                    pk[c] = pack_bf16x2(e2.x, e2.y);
                }
                const float2 s2 = fadd2(acc[0], acc[1]);
                l += s2.x + s2.y;
                // weight buffer sb is free once P.V(g - 2) has read it
                if (g >= 2) {
                    mbar_wait(&sm->p_free[sb], ((g >> 1) - 1) & 1, abort_flag, p.status, 0x81f);
                    __syncwarp();
                    tc_fence_after();
                }
                if (j > 0 && __any_sync(0xffffffffu, grow)) {
                    // O is rescaled (this part's features) once P.V(g - 1) has completed; at j = 0 the first
                    // P.V overwrites O, after the previous unit's output has been read
                    mbar_wait(&sm->p_free[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, p.status, 0x820);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll
                    for (int q4 = 0; q4 < kOut / 16; ++q4) {
                        uint32_t o[16];
                        tmem_ld_x16(o_tmem + q4 * 16, o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                        tmem_st_x16(o_tmem + q4 * 16, o);
                    }
                }
                tmem_st_x16_nowait(p_tmem + sb * 64, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm->p_full[sb]);
            }
            // The next unit's slot and spans are read now: their latency passes behind the output.
            const int next = k + 1;
            ok = mbar_wait(&sm->unit_full[next % kSlots], (next / kSlots) & 1, abort_flag, p.status, 0x821);
            x = sm->unit[next % kSlots];
            if (ok && x.n > 0) span = span_of(p, x.b, x.q0 + row);
            // ---------------- output: thread (h, row) writes its features of O / (l_0 + ... + l_3). The output tile's
            // buffer first carries l_h of every part and row; the previous unit's store has read it.
            uint8_t* obuf = base + G::kOffO;
            if (warp == 0 && lane == 0) tma_store_wait_read();
            named_bar_sync(1, kSoft);
            float* lsum = reinterpret_cast<float*>(obuf);
            lsum[h * BM + row] = l;
            named_bar_sync(4 + q, 32 * kParts);   // the four warps of these rows
            const float L = (lsum[row] + lsum[BM + row]) + (lsum[2 * BM + row] + lsum[3 * BM + row]);
            const bool none = L == 0.0f;              // no key: a row of zeros, O may hold 0 * NaN from the tile's other rows' keys
            const float inv = L > 0.0f ? 1.0f / L : L;   // NaN stays
            const uint32_t gl = g - 1;   // the unit's last tile: its P.V completes O
            mbar_wait(&sm->p_free[gl & 1], (gl >> 1) & 1, abort_flag, p.status, 0x822);
            __syncwarp();
            tc_fence_after();
            uint32_t o[kOut];
            if constexpr (kOut == 32) tmem_ld_x32(o_tmem, o);
            else tmem_ld_x16(o_tmem, o);
            if constexpr (kSplit) {
                // the only unit of this CTA: every copy and product that used the tiles has completed
#pragma unroll
                for (int c = 0; c < kOut; c += 4)
                    *reinterpret_cast<uint4*>(part + row * kPitch + h * kOut + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                if (h == 0) {
                    sm->mx[0][row] = m;
                    sm->mx[1][row] = L;
                }
                continue;
            }
            named_bar_sync(1, kSoft);   // every thread has read the sums the staging overwrites
#pragma unroll
            for (int ch = 0; ch < kOut / 8; ++ch) {
                const int col = h * kOut + 8 * ch;   // feature: slab col / 64, 16-byte chunk (col % 64) / 8
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = none ? 0u : pack_bf16x2(__uint_as_float(o[ch * 8 + 2 * e]) * inv, __uint_as_float(o[ch * 8 + 2 * e + 1]) * inv);
                st_shared_v4(smem_u32(obuf + (col / 64) * kHalf) + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4), w[0],
                             w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();   // O has been read: the next unit's first P.V may overwrite it
            named_bar_sync(1, kSoft);
            if (warp == 0 && lane == 0) {
                if (!*abort_flag) {
                    asm volatile(
                        "cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %2, %4, %5}], [%1];" ::"l"(
                            reinterpret_cast<uint64_t>(&maps.out)),
                        "r"(smem_u32(obuf)), "r"(0), "r"(q0), "r"(head), "r"(b)
                        : "memory");
                    tma_store_commit();
                }
            }
        }
        if (warp == 0 && lane == 0) tma_store_wait_all();
        tc_fence_before();
        named_bar_sync(3, kThreads);
        if constexpr (kSplit) {
            // ------------------------------------------------ join: a CTA takes BM / pieces rows of all parts
            __syncwarp();
            cluster_sync_all();
            const UnitInfo at = place_of(p, blockIdx.x / pieces);
            const uint32_t m_at = smem_u32(&sm->mx[0][0]), o_at = smem_u32(part);
            join_parts<__nv_bfloat16, kD, BM, kSoft>(p, at.b, at.head, at.q0, pieces, piece, m_at, o_at);
            __syncwarp();
            cluster_sync_all();   // the others have read this CTA's part
        }
    }
}

// spans[b, i]: the run of equal ids around i. A thread per position, a CTA per 1024 of them: the nearest change
// before and after a position comes from its warp's ballots, then from one value a warp; where the CTA holds none, it
// looks through its neighbours' positions, 1024 at a time, until it meets one. (A CTA a sequence, with a scan over
// strided positions, took 18.7 us at 4 x 8192.)
constexpr int kSpanThreads = 1024;
__global__ void __launch_bounds__(kSpanThreads) document_spans_kernel(const int32_t* ids, int L, int32_t* spans) {
    __shared__ int last_of[32], first_of[32];
    pdl_trigger();
    pdl_wait();
    const int32_t* x = ids + static_cast<int64_t>(blockIdx.y) * L;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int at = blockIdx.x * kSpanThreads;
    const int i = at + threadIdx.x;
    auto starts = [&](int n) { return n < L && (n == 0 || x[n] != x[n - 1]); };
    auto ends = [&](int n) { return n < L && (n + 1 == L || x[n] != x[n + 1]); };
    const unsigned s = __ballot_sync(0xffffffffu, starts(i)), e = __ballot_sync(0xffffffffu, ends(i));
    if (lane == 0) {
        last_of[warp] = s ? at + warp * 32 + 31 - __clz(s) : -1;
        first_of[warp] = e ? at + warp * 32 + __ffs(e) : 0x7fffffff;     // one past the end
    }
    __syncthreads();
    int before = __reduce_max_sync(0xffffffffu, lane < warp ? last_of[lane] : -1);
    int after = __reduce_min_sync(0xffffffffu, lane > warp ? first_of[lane] : 0x7fffffff);
    // what lies outside the CTA, for the positions before its first start and behind its last end
    int outside_before = -1, outside_after = 0x7fffffff;
    for (int c = at - kSpanThreads; c >= 0 && outside_before < 0 && !starts(at); c -= kSpanThreads) {
        const unsigned m = __ballot_sync(0xffffffffu, starts(c + threadIdx.x));
        __syncthreads();
        if (lane == 0) last_of[warp] = m ? c + warp * 32 + 31 - __clz(m) : -1;
        __syncthreads();
        outside_before = __reduce_max_sync(0xffffffffu, last_of[lane]);
    }
    const int end_of = min(at + kSpanThreads, L);
    for (int c = end_of; c < L && outside_after == 0x7fffffff && !ends(end_of - 1); c += kSpanThreads) {
        const unsigned m = __ballot_sync(0xffffffffu, ends(c + threadIdx.x));
        __syncthreads();
        if (lane == 0) first_of[warp] = m ? c + warp * 32 + __ffs(m) : 0x7fffffff;
        __syncthreads();
        outside_after = __reduce_min_sync(0xffffffffu, first_of[lane]);
    }
    if (i >= L) return;
    const unsigned s_here = s & (0xffffffffu >> (31 - lane)), e_here = e & (0xffffffffu << lane);
    const int start = s_here ? at + warp * 32 + 31 - __clz(s_here) : before >= 0 ? before : outside_before;
    const int end = e_here ? at + warp * 32 + __ffs(e_here) : after != 0x7fffffff ? after : outside_after;
    reinterpret_cast<int2*>(spans)[static_cast<int64_t>(blockIdx.y) * L + i] = x[i] < 0 ? make_int2(0, 0) : make_int2(start, end);
}

}  // namespace

cudaError_t launch_document_spans(const int32_t* ids, int B, int L, int32_t* spans, cudaStream_t s) {
    return launch_pdl(document_spans_kernel, dim3((L + kSpanThreads - 1) / kSpanThreads, B), dim3(kSpanThreads), 0, s, ids, L, spans);
}

static int64_t units_of(const SpanAttnParams& p) { return static_cast<int64_t>(p.B) * p.h * ((p.Lq + BM - 1) / BM); }

template <int kD, int kMode, bool kSplit>
static cudaError_t launch_as(const SpanAttnParams& p, const SpanMaps& maps, cudaStream_t s) {
    static_assert(smem_bytes<kD>() <= 232448, "shared memory budget");
    auto kernel = span_attn_kernel<kD, kMode, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_bytes<kD>()));
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(units_of(p) * p.pieces));
    return kSplit ? launch_pdl_cluster(kernel, grid, dim3(kThreads), p.pieces, smem_bytes<kD>(), s, p, maps)
                  : launch_pdl(kernel, grid, dim3(kThreads), smem_bytes<kD>(), s, p, maps);
}
template <int kD, int kMode>
static cudaError_t launch_mode(const SpanAttnParams& p, const SpanMaps& maps, cudaStream_t s) {
    return p.pieces > 1 ? launch_as<kD, kMode, true>(p, maps, s) : launch_as<kD, kMode, false>(p, maps, s);
}
static int clusters_at_once(int size) {
    static ClusterRoom room;      // an SM holds one CTA of any instance
    auto kernel = span_attn_kernel<128, kGeneral, true>;
    constexpr size_t kBytes = smem_bytes<128>();
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kBytes)) != cudaSuccess) return 0;
    return room.at_once(kernel, kThreads, kBytes, size);
}

// CTAs that share a unit: with few units (few queries over long keys) most SMs would stand idle and a unit would go
// through its keys alone. As many as let all units run at once, from a number of keys on that pays for the two cluster
// barriers and the join (2 to 3 us). 128 queries, 8 heads of 64 (128), us alone and shared: 2048 keys 17.2 (16.3), by two 12.7
// (14.2), four 10.5 (12.3), eight 9.9 (11.5); one query, 4096 keys, by eight 28.9 -> 9.4 (26.7 -> 10.3). Where the clusters do
// not run at once they cost twice that: 16 units by eight 17.8 (20.9).
static int pieces_of(const SpanAttnParams& p) {
    const int64_t reach = p.causal && p.prefix_lens == nullptr ? std::min<int64_t>(p.Lk, static_cast<int64_t>(p.q_offset) + p.Lq) : p.Lk;
    const int64_t units = units_of(p);
    if (reach < 768 || units > 256) return 1;
    if (units <= clusters_at_once(8)) return 8;                       // one query, 768 keys: 7.3 against 8.1 us
    if (reach >= 1024 && units <= clusters_at_once(4)) return 4;      // 30 units, 1024 keys: 9.7 against 10.2 (d_k = 128: 11.4, 11.0)
    if (reach >= 1536 && units <= clusters_at_once(2)) return 2;      // 60 units, 1536 keys: 12.3 against 14.8 (14.3, 14.4)
    return 1;
}

template <int kD>
static cudaError_t launch_d(const SpanAttnParams& p, const SpanMaps& maps, int mode, cudaStream_t s) {
    return mode == kPlain    ? launch_mode<kD, kPlain>(p, maps, s)
           : mode == kCapped ? launch_mode<kD, kCapped>(p, maps, s)
           : mode == kSingle ? launch_mode<kD, kSingle>(p, maps, s)
                             : launch_mode<kD, kGeneral>(p, maps, s);
}

// [B, L, H, d] as {64, L, d / 64, H, B}: a 64-column slab of 128 rows is one swizzled half tile
static bool map_strided(CUtensorMap* m, const Strided& t, int B, int L, int H, int d) {
    const uint64_t dims[5] = {64, (uint64_t)L, (uint64_t)d / 64, t.h != 0 ? (uint64_t)H : 1, t.b != 0 ? (uint64_t)B : 1};
    const uint64_t str[4] = {(uint64_t)t.l * 2, 128, t.h != 0 ? (uint64_t)t.h * 2 : 128, t.b != 0 ? (uint64_t)t.b * 2 : 128};
    const uint32_t box[5] = {64, 128, (uint32_t)d / 64, 1, 1};
    return encode_bf16_tiled(m, t.p, 5, dims, str, box, true);
}

cudaError_t launch_span_attn(const SpanAttnParams& given, cudaStream_t s) {
    SpanAttnParams p = given;
    p.pieces = pieces_of(p);
    SpanMaps maps;
    if (!map_strided(&maps.q, p.q, p.B, p.Lq, p.h, p.d) || !map_strided(&maps.k, p.k, p.B, p.Lk, p.h_kv, p.d) ||
        !map_strided(&maps.v, p.v, p.B, p.Lk, p.h_kv, p.d) || !map_strided(&maps.out, p.out, p.B, p.Lq, p.h, p.d))
        return cudaErrorInvalidValue;
    const int mode = p.cap > 0.0f && !tanh_folds(p.scale / p.cap) ? kSingle
                     : p.slopes == nullptr && p.cap > 0.0f ? kCapped
                     : p.slopes == nullptr && p.cap == 0.0f && p.scale > 0.0f ? kPlain
                                                                             : kGeneral;
    if (p.d == 128) return launch_d<128>(p, maps, mode, s);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (mode != kCapped && mode != kSingle && p.Lk >= kLongKeys && p.Lq > BM && units_of(p) > sms) return launch_span_attn_d64(p, maps, mode, s);
    return launch_d<64>(p, maps, mode, s);
}

}  // namespace mha
