// resize.cu -- the block table of a paged cache as sequences grow, shrink and end: pages come from and go back to a stack of
// free ones, and every new token gets its slot.
//
// Sequence b goes from held to want positions, from have to then pages, n pages being ceil(positions / page). With
// down = max(have - then, 0), up = max(then - have, 0) and their exclusive sums D, U over the sequences: page `then + i` of a
// sequence that shrinks goes to stack position count + sum(down) - 1 - (D + i), and page `have + i` of one that grows is
// the one at F - 1 - (U + i) of the F that are then free, so a step back returns the same stack. Served are those whose U + up is
// at most F; needs are positive, so they are the first ones.
//
// A latency, not a bandwidth: a step of one token moves a few hundred bytes. One launch (a second for the slots of very many tokens): the CTAs of a cluster each
// sum the lengths of all sequences for themselves (two loads and two scans a kThreads sequences), divide the pages and slots among them,
// and meet at one cluster barrier: after the pages that went back are on the stack, if any did, else before the new
// count is written. Pages are found from the flat number of a grant by bisection in the sums, so a sequence of 10^5 positions
// is as well divided as 10^5 of one.
#include <algorithm>

#include "launch.h"
#include "mha_internal.h"
#include "ptx_pair.cuh"
#include "ptx_serve.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kSlots = 8, kPages = 4;       // of a thread at a time: their loads are in flight together

struct Span {
    int held, want, have, then;     // pages that the table holds; after the step
};

__device__ __forceinline__ int pages_of(const ResizeParams& p, int n) {
    const int q = p.page.div(n);
    return q + (static_cast<int64_t>(q) * p.page.d < n ? 1 : 0);
}

// A sequence that wants more than its row of the table holds stays as it is; one that holds more than that has the row's pages.
__device__ __forceinline__ Span span_of(const ResizeParams& p, int b) {
    Span s{0, 0, 0, 0};
    if (b >= p.B) return s;
    s.held = max(p.held[b], 0);
    s.want = max(p.want[b], 0);
    s.have = min(pages_of(p, s.held), p.max_pages);
    s.then = pages_of(p, s.want);
    if (s.then > p.max_pages) {
        if (s.want > s.held) s.want = s.held;
        s.then = min(pages_of(p, s.want), p.max_pages);
    }
    return s;
}

// Pages that sequences get and give back, in sums
struct Moves {
    long long up, down;
};

template <int kThreads>
struct Shared {
    Moves warps[kThreads / 32];
    int off[kThreads];              // exclusive sums of the pages that move, of the chunk's sequences
    int first[kThreads];            // the first page that moves
    int held[kThreads], add[kThreads];
    int granted;
};

__device__ __forceinline__ Moves warp_sums(Moves v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, v.up, o), down = __shfl_up_sync(0xffffffffu, v.down, o);
        if (lane >= o) {
            v.up += up;
            v.down += down;
        }
    }
    return v;
}

// Inclusive sums over the block's sequences, and all of them. The block has met since the last call's sums were read.
template <int kThreads>
__device__ __forceinline__ Moves block_sums(Shared<kThreads>& sh, const Span& s, Moves* all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Moves inc = warp_sums(Moves{max(s.then - s.have, 0), max(s.have - s.then, 0)}, lane);
    if (lane == 31) sh.warps[warp] = inc;
    __syncthreads();
    static_assert(kThreads <= 1024, "a warp's sum a lane");
    const Moves w = warp_sums(lane < kThreads / 32 ? sh.warps[lane] : Moves{0, 0}, lane);
    if (warp > 0) {
        inc.up += __shfl_sync(0xffffffffu, w.up, warp - 1);
        inc.down += __shfl_sync(0xffffffffu, w.down, warp - 1);
    }
    all->up = __shfl_sync(0xffffffffu, w.up, 31);
    all->down = __shfl_sync(0xffffffffu, w.down, 31);
    return inc;
}

// The last i of off[0 .. n) with off[i] <= x, off[0] = 0; sequences that move nothing share their successor's sum.
__device__ __forceinline__ int owner_of(const int* off, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Slots of `most` new tokens, those of sequence i and token t by where(i, t, position): the address of its page's number, or
// nullptr where there is none.
template <typename Where>
__device__ __forceinline__ void slots_of(const ResizeParams& p, long long most, int me, int all, int64_t first, bool& bad, Where&& where) {
    for (long long x0 = me; x0 < most; x0 += static_cast<long long>(kSlots) * all) {
        int page[kSlots], at[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const long long x = x0 + static_cast<long long>(k) * all;
            at[k] = -1;
            if (x >= most) continue;
            const int i = p.by_t.div(static_cast<int>(x)), t = static_cast<int>(x) - i * p.T;
            const int32_t* from = where(i, t, at[k]);
            if (from != nullptr) page[k] = *from;
        }
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const long long x = x0 + static_cast<long long>(k) * all;
            if (x >= most) continue;
            int64_t slot = -1;
            if (at[k] >= 0) {
                if (page[k] >= 0 && page[k] < p.n_pages)
                    slot = static_cast<int64_t>(page[k]) * p.page.d + (at[k] - p.page.div(at[k]) * static_cast<int>(p.page.d));
                else
                    bad = true;
            }
            p.slots[first + x] = slot;
        }
    }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) resize_kernel(const __grid_constant__ ResizeParams p) {
    __shared__ Shared<kThreads> sh;
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_ctarank()), ctas = gridDim.x;
    const int me = rank * kThreads + tid, all = ctas * kThreads;
    pdl_trigger();
    pdl_wait();
    // the first kThreads sequences are summed once, the others again where they are needed
    const Span mine = span_of(p, tid);
    if (tid == 0) sh.granted = 0;
    const int count = min(max(*p.free_count, 0), p.n_pages);
    Moves my_all;
    const Moves my_inc = block_sums(sh, mine, &my_all);
    long long back = my_all.down;
    for (int b0 = kThreads; b0 < p.B; b0 += kThreads) {
        Moves total;
        __syncthreads();
        block_sums(sh, span_of(p, b0 + tid), &total);
        back += total.down;
    }

    // ---- pages that go back
    bool bad = false;
    if (back > 0) {
        long long before = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int n = min(p.B - b0, kThreads);
            Span s = mine;
            Moves inc = my_inc, total = my_all;
            if (b0 > 0) {
                __syncthreads();                   // the sums and the last chunk's arrays have been read
                s = span_of(p, b0 + tid);
                inc = block_sums(sh, s, &total);
            }
            // a chunk's pages are fewer than 2^31 unless pages are returned twice: those beyond are not looked at
            const int most = static_cast<int>(min(total.down, 0x7fffffffll));
            sh.off[tid] = static_cast<int>(min(inc.down - max(s.have - s.then, 0), 0x7fffffffll));
            sh.first[tid] = s.then;
            __syncthreads();
            for (long long x0 = me; x0 < most; x0 += static_cast<long long>(kPages) * all) {
                int32_t* entry[kPages];
                int page[kPages];
#pragma unroll
                for (int k = 0; k < kPages; ++k) {
                    const long long x = x0 + static_cast<long long>(k) * all;
                    entry[k] = nullptr;
                    if (x >= most) continue;
                    const int i = owner_of(sh.off, n, static_cast<int>(x));
                    entry[k] = p.table + (b0 + i) * p.table_stride + sh.first[i] + (static_cast<int>(x) - sh.off[i]);
                    page[k] = *entry[k];
                }
#pragma unroll
                for (int k = 0; k < kPages; ++k) {
                    if (entry[k] == nullptr) continue;
                    const long long at = count + back - 1 - (before + x0 + static_cast<long long>(k) * all);
                    if (at < p.n_pages) p.free_pages[at] = page[k];
                    bad |= at >= p.n_pages || page[k] < 0 || page[k] >= p.n_pages;
                    *entry[k] = -1;
                }
            }
            before += total.down;
        }
        cluster_sync_all();
    }

    // ---- pages granted, and slots
    const int pool = static_cast<int>(min(count + back, static_cast<long long>(p.n_pages)));
    long long before = 0;
    int used = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid, n = min(p.B - b0, kThreads);
        Span s = mine;
        Moves inc = my_inc, total = my_all;
        if (b0 > 0 || back > 0) __syncthreads();
        if (b0 > 0) {
            if (tid == 0) sh.granted = used;
            s = span_of(p, b);
            inc = block_sums(sh, s, &total);
        }
        const int up = max(s.then - s.have, 0);
        inc.up += before;
        const bool served = up == 0 || inc.up <= pool;
        const int lens = served ? s.want : s.held, add = max(lens - s.held, 0);
        if (inc.up <= pool && up > 0) atomicMax(&sh.granted, static_cast<int>(inc.up));
        // sums beyond the pool belong to sequences that get nothing
        sh.off[tid] = static_cast<int>(min(inc.up - up, static_cast<long long>(pool))) - used;
        sh.first[tid] = s.have;
        sh.held[tid] = s.held;
        sh.add[tid] = add;
        if (rank == 0 && b < p.B) {
            p.lens[b] = lens;
            if (p.new_lens != nullptr) p.new_lens[b] = add;
        }
        __syncthreads();
        const int now = sh.granted;
        const int32_t* top = p.free_pages + (pool - 1 - used);     // of the chunk's first grant
        for (long long x0 = me; x0 < now - used; x0 += static_cast<long long>(kPages) * all) {
            int32_t* entry[kPages];
            int page[kPages];
#pragma unroll
            for (int k = 0; k < kPages; ++k) {
                const long long x = x0 + static_cast<long long>(k) * all;
                entry[k] = nullptr;
                if (x >= now - used) continue;
                page[k] = *(top - x);
                const int i = owner_of(sh.off, n, static_cast<int>(x));
                entry[k] = p.table + (b0 + i) * p.table_stride + sh.first[i] + (static_cast<int>(x) - sh.off[i]);
            }
#pragma unroll
            for (int k = 0; k < kPages; ++k) {
                if (entry[k] == nullptr) continue;
                bad |= page[k] < 0 || page[k] >= p.n_pages;
                *entry[k] = page[k];
            }
        }
        if (p.slots != nullptr && !p.slots_after) {
            slots_of(p, static_cast<long long>(n) * p.T, me, all, static_cast<int64_t>(b0) * p.T, bad, [&](int i, int t, int& at) {
                if (t >= sh.add[i]) return static_cast<const int32_t*>(nullptr);
                at = sh.held[i] + t;
                const int pg = p.page.div(at);
                // a page granted now is read where it was on the stack: another CTA may be writing it into the table
                return pg >= sh.first[i] ? top - (sh.off[i] + pg - sh.first[i]) : p.table + (b0 + i) * p.table_stride + pg;
            });
        }
        before += total.up;
        used = now;
    }
    if (bad) atomicCAS(p.status, 0, MHA_PAGED_BAD_PAGE);
    if (back == 0) cluster_sync_all();        // every CTA has read the count
    if (rank == 0 && tid == 0) *p.free_count = pool - used;
}

// The slots of many new tokens, from the table and the lengths as they are after the step.
constexpr int kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const __grid_constant__ ResizeParams p) {
    pdl_trigger();
    pdl_wait();
    bool bad = false;
    slots_of(p, static_cast<long long>(p.B) * p.T, blockIdx.x * kSlotThreads + threadIdx.x, gridDim.x * kSlotThreads, 0, bad, [&](int b, int t, int& at) {
        const int held = max(p.held[b], 0);
        if (t >= p.lens[b] - held) return static_cast<const int32_t*>(nullptr);
        at = held + t;
        return static_cast<const int32_t*>(p.table + b * p.table_stride + p.page.div(at));
    });
    if (bad) atomicCAS(p.status, 0, MHA_PAGED_BAD_PAGE);
}

}  // namespace

cudaError_t launch_resize(const ResizeParams& p, cudaStream_t s) {
    // A cluster's CTAs cost nothing where there is nothing for them (16 sequences, a token each, there and back: 8.7 us with one
    // as with eight), and 16 of them pay from a few thousand pages or slots on (64 prompts of up to 8192: 37 us with eight, 24 with 16). The
    // slots of many more tokens are left to a kernel of their own, on the whole GPU (the same: 13 us; 16 prompts, 131072 slots: 10.6 against
    // 11.2 us; 8: 10.1 against 9.0). More sequences than threads are taken in turns, so there are 1024 from 513 sequences on (1024 sequences,
    // a token each: 10.9 us, with 512 threads 15.2; 256 sequences: 9.6 us with 1024 threads, 7.5 with 512).
    constexpr int kCtas = 16;
    constexpr int64_t kFewSlots = 1 << 17;
    ResizeParams q = p;
    const int64_t slots = p.slots != nullptr ? static_cast<int64_t>(p.B) * p.T : 0;
    q.slots_after = slots >= kFewSlots;
    const bool few = p.B <= 512;
    const int threads = few ? 512 : 1024;
    const auto kernel = few ? resize_kernel<512> : resize_kernel<1024>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    // a part of a device, or a smaller one, may have no room for 16 side by side; the kernel takes any number
    static ClusterRoom rooms[2];
    int ctas = kCtas;
    while (ctas > 1 && rooms[few].at_once(kernel, threads, 0, ctas) < 1) ctas /= 2;
    e = launch_pdl_cluster(kernel, dim3(ctas), dim3(threads), ctas, 0, s, q);
    if (e != cudaSuccess || !q.slots_after) return e;
    int sms = 0;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    const int64_t wide = std::min<int64_t>(8 * sms, (slots + kSlots * kSlotThreads - 1) / (kSlots * kSlotThreads));
    return launch_pdl(slots_kernel, dim3(static_cast<unsigned>(wide)), dim3(kSlotThreads), 0, s, q);
}

}  // namespace mha
