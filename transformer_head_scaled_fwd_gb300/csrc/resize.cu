// resize.cu -- the block table of a paged cache as sequences grow, shrink and end: pages come from and go back to a stack of
// free ones, and every new token gets its slot.
//
// Sequence b goes from held to want positions, from have to then pages, n pages being ceil(positions / page). With
// down = max(have - then, 0), up = max(then - have, 0) and their exclusive sums D, U over the sequences: page `then + i` of a
// sequence that shrinks goes to stack position count + sum(down) - 1 - (D + i), and page `have + i` of one that grows is
// the one at F - 1 - (U + i) of the F that are then free, so a step back returns the same stack. Served are those whose U + up is
// at most F; needs are positive, so they are the first ones.
//
// A latency, not a bandwidth: a step of one token moves a few hundred bytes. One launch: the CTAs of a cluster each
// sum the lengths of all sequences for themselves (two loads and two scans a kThreads sequences), divide the pages and slots among them,
// and meet at one cluster barrier: after the pages that went back are on the stack, if any did, else before the new
// count is written. Pages are found from the flat number of a grant by bisection in the sums, so a sequence of 10^5 positions
// is as well divided as 10^5 of one.
#include "launch.h"
#include "mha_internal.h"
#include "ptx_pair.cuh"
#include "ptx_serve.cuh"
#include "serve.h"

namespace mha {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Span {
    int held, want, have, then;     // pages that the table holds; after the step
};

__device__ __forceinline__ int pages_of(const ResizeParams& p, int n) {
    const int q = p.page.div(n);
    return q + (static_cast<int64_t>(q) * p.page.d < n ? 1 : 0);
}

// A sequence that wants more than its row of the table holds stays as it is; one that holds more than that has the row's pages.
__device__ __forceinline__ Span span_of(const ResizeParams& p, int b) {
    Span s;
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

__device__ __forceinline__ long long warp_inclusive(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long other = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += other;
    }
    return v;
}

struct Shared {
    long long scan[kWarps];
    int off[kThreads];              // exclusive sums of the pages that move, of the chunk's sequences
    int first[kThreads];            // the first page that moves
    int held[kThreads], add[kThreads];
    int granted;
};

// Inclusive sums over the block, and the block's total.
__device__ __forceinline__ long long block_inclusive(Shared& sh, long long v, long long* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long inc = warp_inclusive(v, lane);
    __syncthreads();
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const long long x = sh.scan[w];
        if (w < warp) inc += x;
        all += x;
    }
    *total = all;
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

__global__ void __launch_bounds__(kThreads) resize_kernel(const __grid_constant__ ResizeParams p) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, rank = static_cast<int>(cluster_ctarank()), ctas = gridDim.x;
    const int me = rank * kThreads + tid, all = ctas * kThreads;
    pdl_trigger();
    pdl_wait();
    const int count = min(max(*p.free_count, 0), p.n_pages);
    Span mine{0, 0, 0, 0};
    if (tid < p.B) mine = span_of(p, tid);

    // ---- pages that go back
    long long back = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        const Span s = b0 == 0 ? mine : b < p.B ? span_of(p, b) : Span{0, 0, 0, 0};
        back += max(s.have - s.then, 0);
    }
    block_inclusive(sh, back, &back);
    if (back > 0) {
        long long before = 0;
        for (int b0 = 0; b0 < p.B; b0 += kThreads) {
            const int b = b0 + tid, n = min(p.B - b0, kThreads);
            const Span s = b0 == 0 ? mine : b < p.B ? span_of(p, b) : Span{0, 0, 0, 0};
            const int down = max(s.have - s.then, 0);
            long long total;
            const long long inc = block_inclusive(sh, down, &total);
            // a chunk's pages are fewer than 2^31 unless pages are returned twice: those beyond are not looked at
            const int most = static_cast<int>(min(total, 0x7fffffffll));
            sh.off[tid] = static_cast<int>(min(inc - down, 0x7fffffffll));
            sh.first[tid] = s.then;
            __syncthreads();
            for (long long x = me; x < most; x += all) {
                const int i = owner_of(sh.off, n, static_cast<int>(x));
                int32_t* entry = p.table + (b0 + i) * p.table_stride + sh.first[i] + (static_cast<int>(x) - sh.off[i]);
                const long long at = count + back - 1 - (before + x);
                const int page = *entry;
                if (at < p.n_pages) p.free_pages[at] = page;
                if (at >= p.n_pages || page < 0 || page >= p.n_pages) atomicCAS(p.status, 0, MHA_PAGED_BAD_PAGE);
                *entry = -1;
            }
            before += total;
            __syncthreads();
        }
        cluster_sync_all();
    }

    // ---- pages granted, and slots
    const int pool = static_cast<int>(min(count + back, static_cast<long long>(p.n_pages)));
    long long before = 0;
    int used = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid, n = min(p.B - b0, kThreads);
        const Span s = b0 == 0 ? mine : b < p.B ? span_of(p, b) : Span{0, 0, 0, 0};
        const int up = max(s.then - s.have, 0);
        if (tid == 0) sh.granted = used;
        long long total;
        const long long inc = before + block_inclusive(sh, up, &total);
        const bool served = up == 0 || inc <= pool;
        if (inc <= pool) atomicMax(&sh.granted, static_cast<int>(inc));
        const int lens = served ? s.want : s.held, add = max(lens - s.held, 0);
        // sums beyond the pool belong to sequences that get nothing
        sh.off[tid] = static_cast<int>(min(inc - up, static_cast<long long>(pool))) - used;
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
        for (int x = me; x < now - used; x += all) {
            const int i = owner_of(sh.off, n, x);
            const int page = __ldcg(top - x);
            if (page < 0 || page >= p.n_pages) atomicCAS(p.status, 0, MHA_PAGED_BAD_PAGE);
            p.table[(b0 + i) * p.table_stride + sh.first[i] + (x - sh.off[i])] = page;
        }
        if (p.slots != nullptr) {
            for (long long x = me; x < static_cast<long long>(n) * p.T; x += all) {
                const int i = p.by_t.div(static_cast<int>(x)), t = static_cast<int>(x) - i * p.T;
                int64_t slot = -1;
                if (t < sh.add[i]) {
                    const int at = sh.held[i] + t, pg = p.page.div(at);
                    const int page = pg >= sh.first[i] ? __ldcg(top - (sh.off[i] + pg - sh.first[i]))
                                                       : p.table[(b0 + i) * p.table_stride + pg];
                    if (page >= 0 && page < p.n_pages)
                        slot = static_cast<int64_t>(page) * p.page.d + (at - pg * static_cast<int>(p.page.d));
                    else
                        atomicCAS(p.status, 0, MHA_PAGED_BAD_PAGE);
                }
                p.slots[static_cast<int64_t>(b0) * p.T + x] = slot;
            }
        }
        before += total;
        used = now;
        __syncthreads();
    }
    if (back == 0) cluster_sync_all();        // every CTA has read the count
    if (rank == 0 && tid == 0) *p.free_count = pool - used;
}

}  // namespace

cudaError_t launch_resize(const ResizeParams& p, cudaStream_t s) {
    // A CTA where the work is a few accesses a thread, else the eight of a portable cluster.
    const int64_t work = static_cast<int64_t>(p.B) * (p.slots != nullptr ? p.T : 1);
    const int ctas = work <= 4 * kThreads ? 1 : 8;
    return launch_pdl_cluster(resize_kernel, dim3(ctas), dim3(kThreads), ctas, 0, s, p);
}

}  // namespace mha
