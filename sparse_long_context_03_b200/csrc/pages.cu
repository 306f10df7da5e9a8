// pages.cu -- the pages of a paged cache: granting them to sequences, forking
// sequences, freeing them, copying pages and compacting the pool.
//
// The pool's only state is a count per page (0: free), a block table row and
// a length per sequence slot.  A grant takes the lowest free page ids, in the
// order of the call's entries, so every result is a function of that state
// and no list of free pages has to be kept right.  Counts change by integer
// atomics, whose order does not show.
//
// Granting is one cluster of up to 8 CTAs: every warp counts the free pages
// of its own stretch of the counts, the CTAs exchange their totals through
// distributed shared memory, and the warps whose first free page is wanted go
// over their stretch once more and write the ids.  The entries (at most 1024,
// one per thread) are worked out by every CTA for itself.  Bound by latency:
// loads, a barrier across the cluster, loads again.  Freeing 32 sequences and
// granting their room anew from 13K pages takes 8.7 us; with one CTA and a
// load per round of 32 ids it took 20.7.
//
// Copying moves pages in pieces of 1024 units, four 16-byte loads in flight to
// a thread.  2048 pages of 69 KB: 49.4 us, 5.7 TB/s read and written, 88 % of a
// plain copy's 6.55.  Compacting 720 of 1800 pages: 24.7 us, of which the moved
// bytes' copy would take 15.
#include <cooperative_groups.h>

#include "kernels.h"
#include "kv8.cuh"

namespace cg = cooperative_groups;

namespace dsa {

namespace {

constexpr int kPageTokens = 64;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;

// Pools whose counts one CTA reads alone: one batch of loads, and no exchange.
constexpr int kOneCtaPages = 4096;
constexpr int kHash = 2 * kPagesMaxEntries;
static_assert(kPagesMaxEntries <= kThreads, "one entry per thread");

// Sums of wanted pages stop here, above every pool's size: 1024 entries may
// together want more than 31 bits hold.
constexpr int kMostWanted = 1 << 25;

enum : int32_t { kOk = 0, kNoSpace = 1, kBad = 2 };

__device__ __forceinline__ int pages_of(int tokens) { return tokens / kPageTokens + (tokens % kPageTokens != 0); }

// This warp's stretch of the pool's ids: whole rounds of 32, the same for
// every warp of the cluster.
struct Stretch {
    int begin, end;
};
__device__ __forceinline__ Stretch stretch_of(int num_pages, int warps, int w) {
    const int per = (num_pages + warps * 32 - 1) / (warps * 32) * 32;
    const long long b = (long long)per * w;
    return {(int)min(b, (long long)num_pages), (int)min(b + per, (long long)num_pages)};
}

// A stretch's counts, gone over several times in rounds of 32 ids, the loads
// of kAhead rounds together (a load per step would pay the latency once per
// round).  The first of them stay in registers between the passes.
constexpr int kAhead = 4;
struct Counts {
    const int32_t *counts;
    int begin, end;
    int first[kAhead];

    __device__ __forceinline__ void load(int (&c)[kAhead], int p0) const {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int p = p0 + 32 * i + (int)(threadIdx.x & 31);
            c[i] = p < end ? counts[p] : -1;
        }
    }
    // f(id, count) by every lane, with id >= end past the stretch, while f
    // returns true (the same in every lane)
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        for (int p0 = begin; p0 < end; p0 += 32 * kAhead) {
            int c[kAhead];
            if (p0 == begin) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) c[i] = first[i];
            } else {
                load(c, p0);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (p0 + 32 * i < end && !f(p0 + 32 * i + (int)(threadIdx.x & 31), c[i])) return;
        }
    }
};
__device__ __forceinline__ Counts counts_of(const int32_t *counts, Stretch st) {
    Counts c{counts, st.begin, st.end, {}};
    c.load(c.first, st.begin);
    return c;
}

// Sum over the cluster's warps before this one, and over all of them, of a
// warp's count.  Ends with a cluster-wide barrier before the sums are read.
struct ClusterScan {
    int warp_total[kWarps];
    int cta_total[kMaxCtas];
};
__device__ __forceinline__ int2 cluster_scan(cg::cluster_group &cluster, ClusterScan &sm, int count) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) sm.warp_total[warp] = count;
    __syncthreads();
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    int v = sm.warp_total[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, v, 31);
    if ((int)threadIdx.x < C) *cluster.map_shared_rank(&sm.cta_total[me], threadIdx.x) = total;
    cluster.sync();
    int before = 0, all = 0;
    for (int c = 0; c < C; ++c) {
        const int x = sm.cta_total[c];
        all += x;
        if (c < me) before += x;
    }
    const int upto = __shfl_sync(0xFFFFFFFFu, v, warp);
    return make_int2(before + upto - count, all);
}

struct GrantArgs {
    const int32_t *slots, *other;   // extend: slots, new lengths; fork: children, parents
    int n;
    int32_t *block_table;
    int n_slots, max_pages;
    int32_t *seq_lens, *refcount;
    int num_pages;
    int32_t *status;
};

// The entries of one call, one per thread: who asks for how many pages.
// EXTEND: slot s of length len to new_lens[i] tokens.  FORK: child s gets the
// length of its parent and one page for a partly filled last one.
template <bool FORK>
__global__ void __launch_bounds__(kThreads) pages_grant_kernel(const __grid_constant__ GrantArgs a) {
    __shared__ ClusterScan scan;
    __shared__ int upto[kThreads];      // pages wanted by entries 0..i
    __shared__ int32_t slot_of[kThreads];
    __shared__ int first_of[kThreads];  // where in its table row an entry's new pages begin
    __shared__ int keys[kHash], firsts[kHash];
    __shared__ int warp_sum[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    cluster_arrive();
    if (FORK) let_next_start();
    wait_for_last();
    const int i = threadIdx.x, warp = i >> 5, lane = i & 31;

    for (int h = i; h < kHash; h += kThreads) {
        keys[h] = -1;
        firsts[h] = kThreads;
    }
    __syncthreads();
    int s = -1, len = 0, to = 0, need = 0, place = 0;
    bool bad = true;
    if (i < a.n) {
        s = a.slots[i];
        bad = s < 0 || s >= a.n_slots;
        if (!bad) {
            len = a.seq_lens[s];
            if (FORK) {
                const int p = a.other[i];
                bad = p < 0 || p >= a.n_slots || len != 0;
                if (!bad) to = a.seq_lens[p];
            } else {
                to = a.other[i];
            }
            bad = bad || len < 0 || to < len || (long long)to > (long long)a.max_pages * kPageTokens;
            // the first entry that names a slot has it; a later one is refused
            for (place = (unsigned)s * 2654435761u % kHash;; place = (place + 1) % kHash) {
                const int was = atomicCAS(&keys[place], -1, s);
                if (was == -1 || was == s) break;
            }
            atomicMin(&firsts[place], i);
        }
    }
    __syncthreads();
    if (!bad && firsts[place] != i) bad = true;
    if (!bad) {
        need = FORK ? (to % kPageTokens != 0) : pages_of(to) - pages_of(len);
        first_of[i] = FORK ? to / kPageTokens : pages_of(len);
    }
    slot_of[i] = s;
    int v = min(need, kMostWanted);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v = min(v + x, kMostWanted);
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w = min(w + x, kMostWanted);
    }
    const int wanted = __shfl_sync(0xFFFFFFFFu, w, 31);
    v = min(v + (warp == 0 ? 0 : __shfl_sync(0xFFFFFFFFu, w, warp - 1)), kMostWanted);
    upto[i] = v;

    // count the free pages, unless nobody wants one
    const Stretch st = stretch_of(a.num_pages, kWarps * (int)cluster.num_blocks(),
                                  (int)cluster.block_rank() * kWarps + warp);
    int count = 0;
    Counts pages{};
    if (wanted > 0) {
        pages = counts_of(a.refcount, st);
        pages.each([&](int, int c) {
            count += c == 0;
            return true;
        });
    }
    count = __reduce_add_sync(0xFFFFFFFFu, count);
    cluster_wait();
    const int2 free = cluster_scan(cluster, scan, count);   // every length has been read behind its barrier

    // entries in order, while the pages last
    const bool ok = !bad && (need == 0 || v <= free.y);
    if (cluster.block_rank() == 0 && i < a.n) {
        a.status[i] = bad ? kBad : (ok ? kOk : kNoSpace);
        if (ok) a.seq_lens[s] = to;
    }
    // upto is non-decreasing: the pages given are those of the last entry whose sum is covered
    int lo = 0, hi = a.n;   // entries 0..lo-1 are covered
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] <= free.y) lo = mid + 1; else hi = mid;
    }
    const int given = lo > 0 ? upto[lo - 1] : 0;
    int rank = free.x;
    if (rank >= given) return;
    pages.each([&](int p, int c) {
        const unsigned m = __ballot_sync(0xFFFFFFFFu, c == 0);
        const int r = rank + __popc(m & ((1u << lane) - 1u));
        if (c == 0 && r < given) {
            int b = 0, e = a.n - 1;                          // the first entry with upto > r
            while (b < e) {
                const int mid = (b + e) >> 1;
                if (upto[mid] > r) e = mid; else b = mid + 1;
            }
            const int at = first_of[b] + r - (b > 0 ? upto[b - 1] : 0);
            a.block_table[(size_t)slot_of[b] * a.max_pages + at] = p;
            a.refcount[p] = 1;
        }
        rank += __popc(m);
        return rank < given;
    });
}

// ---------------------------------------------------------------------------
// copying pages
// ---------------------------------------------------------------------------

// A page as the caches hold it: each buffer's part in units of 16 bytes, or of
// the largest power of two that divides its page and its address.
struct PageBufs {
    char *base[kPagesMaxBufs];
    unsigned long long page_bytes[kPagesMaxBufs];
    int shift[kPagesMaxBufs];
    int units_end[kPagesMaxBufs];   // units of buffers 0..i
    int units;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 4;                              // units in flight per thread
constexpr int kMoveCtas = 8;                               // CTAs per SM that move pages
constexpr int kPiece = kCopyThreads * kCopyBatch;          // units of one piece of a page

template <typename T>
__device__ __forceinline__ void move_unit(const char *s, char *d) {
    *reinterpret_cast<T *>(d) = *reinterpret_cast<const T *>(s);
}

// Piece `piece` of page src to page dst by one CTA.
__device__ __forceinline__ void copy_piece(const PageBufs &pb, int piece, int src, int dst) {
    uint4 x[kCopyBatch];
    char *to[kCopyBatch];
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i) {
        const int u = piece * kPiece + i * kCopyThreads + threadIdx.x;
        to[i] = nullptr;
        if (u >= pb.units) continue;
        int b = 0;
        while (u >= pb.units_end[b]) ++b;
        const size_t off = (size_t)(u - (b > 0 ? pb.units_end[b - 1] : 0)) << pb.shift[b];
        const char *s = pb.base[b] + (size_t)src * pb.page_bytes[b] + off;
        char *d = pb.base[b] + (size_t)dst * pb.page_bytes[b] + off;
        if (pb.shift[b] == 4) {
            x[i] = *reinterpret_cast<const uint4 *>(s);
            to[i] = d;
        } else if (pb.shift[b] == 3) {
            move_unit<uint2>(s, d);
        } else if (pb.shift[b] == 2) {
            move_unit<unsigned int>(s, d);
        } else if (pb.shift[b] == 1) {
            move_unit<unsigned short>(s, d);
        } else {
            move_unit<unsigned char>(s, d);
        }
    }
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i)
        if (to[i] != nullptr) *reinterpret_cast<uint4 *>(to[i]) = x[i];
}

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PageBufs pb,
                                                                  const int32_t *src, const int32_t *dst, int n,
                                                                  int pieces, int num_pages) {
    wait_for_last();
    for (long long w = blockIdx.x; w < (long long)n * pieces; w += gridDim.x) {
        const int i = (int)(w / pieces);
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= num_pages || d < 0 || d >= num_pages || s == d) continue;
        copy_piece(pb, (int)(w % pieces), s, d);
    }
}

// A granted fork's table row, counts and last page.  One CTA per (entry,
// piece of the page); the first piece's CTA also fills the row.
__global__ void __launch_bounds__(kCopyThreads) pages_fork_kernel(const __grid_constant__ PageBufs pb,
                                                                  const __grid_constant__ GrantArgs a, int pieces) {
    wait_for_last();
    const int i = blockIdx.x / pieces, piece = blockIdx.x % pieces;
    if (a.status[i] != kOk) return;
    const int child = a.slots[i], parent = a.other[i];
    const int len = a.seq_lens[child], full = len / kPageTokens;
    if (child == parent) return;                              // an empty sequence forked to itself
    const int32_t *from = a.block_table + (size_t)parent * a.max_pages;
    int32_t *to = a.block_table + (size_t)child * a.max_pages;
    if (piece == 0)
        for (int j = threadIdx.x; j < full; j += kCopyThreads) {
            const int p = from[j];
            to[j] = p;
            if (p >= 0 && p < a.num_pages) atomicAdd(a.refcount + p, 1);
        }
    if (len % kPageTokens != 0 && pb.units > 0) {
        const int s = from[full], d = to[full];
        if (s >= 0 && s < a.num_pages && d >= 0 && d < a.num_pages) copy_piece(pb, piece, s, d);
    }
}

// One CTA per entry: its pages' counts down by one (never below zero), its
// row empty.  Of entries that name one slot twice the first frees it.
__global__ void __launch_bounds__(256) pages_free_kernel(const int32_t *slots, int n, int32_t *block_table,
                                                         int n_slots, int max_pages, int32_t *seq_lens,
                                                         int32_t *refcount, int num_pages) {
    wait_for_last();
    const int i = blockIdx.x, s = slots[i];
    if (s < 0 || s >= n_slots) return;
    bool again = false;
    for (int j = threadIdx.x; j < i; j += blockDim.x) again = again || slots[j] == s;
    if (__syncthreads_or(again)) return;
    const int len = seq_lens[s];
    __syncthreads();
    if (threadIdx.x == 0) seq_lens[s] = 0;
    int32_t *row = block_table + (size_t)s * max_pages;
    const int used = len > 0 ? min(pages_of(len), max_pages) : 0;
    for (int j = threadIdx.x; j < used; j += blockDim.x) {
        const int p = row[j];
        row[j] = -1;
        if (p >= 0 && p < num_pages && atomicSub(refcount + p, 1) <= 0) atomicAdd(refcount + p, 1);
    }
}

// ---------------------------------------------------------------------------
// compacting
// ---------------------------------------------------------------------------

// Workspace: [moves][pad to 16 bytes][free ids below n_used][used ids from
// n_used on], both ascending; the k-th of the latter moves to the k-th of the
// former, so no page is both read and written by a move.
struct CompactArgs {
    const int32_t *refs_in;
    int32_t *refs_out, *map, *n_used;
    int num_pages;
    int32_t *moves, *lows, *highs;
};

__global__ void __launch_bounds__(kThreads) pages_plan_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ ClusterScan scan0, scan1;
    cg::cluster_group cluster = cg::this_cluster();
    cluster_arrive();
    let_next_start();
    wait_for_last();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const Stretch st = stretch_of(a.num_pages, kWarps * C, me * kWarps + warp);
    int count = 0;
    const Counts pages = counts_of(a.refs_in, st);
    pages.each([&](int p, int c) {
        count += p < st.end && c != 0;
        return true;
    });
    cluster_wait();
    const int2 used = cluster_scan(cluster, scan0, __reduce_add_sync(0xFFFFFFFFu, count));
    const int n_used = used.y;
    // free ids below n_used, by stretch: their total is the number of moves
    int holes = 0;
    if (st.begin < n_used)
        pages.each([&](int p, int c) {
            holes += p < st.end && p < n_used && c == 0;
            return true;
        });
    const int2 low = cluster_scan(cluster, scan1, __reduce_add_sync(0xFFFFFFFFu, holes));
    int lr = low.x, ur = used.x;
    const int below = n_used - low.y;                 // used ids below n_used
    pages.each([&](int p, int ref) {
        const bool in = p < st.end;
        const unsigned mu = __ballot_sync(0xFFFFFFFFu, in && ref != 0);
        const unsigned ml = __ballot_sync(0xFFFFFFFFu, in && ref == 0 && p < n_used);
        const unsigned before = (1u << lane) - 1u;
        if (in) {
            if (ref != 0 && p >= n_used) {
                a.highs[ur + __popc(mu & before) - below] = p;
            } else {
                if (ref == 0 && p < n_used) a.lows[lr + __popc(ml & before)] = p;
                a.map[p] = ref != 0 ? p : -1;
                a.refs_out[p] = ref;
            }
        }
        ur += __popc(mu);
        lr += __popc(ml);
        return true;
    });
    cluster.sync();                                   // both lists are complete
    for (int r = me * kThreads + threadIdx.x; r < low.y; r += C * kThreads) {
        const int h = a.highs[r], l = a.lows[r];
        a.refs_out[l] = a.refs_in[h];                 // read before it is cleared: the counts may be changed in place
        a.refs_out[h] = 0;
        a.map[h] = l;
    }
    if (me == 0 && threadIdx.x == 0) {
        *a.n_used = n_used;
        *a.moves = low.y;
    }
}

// The first `remap` CTAs rewrite the block table, the others move pages, the
// next piece's page ids read ahead.
__global__ void __launch_bounds__(kCopyThreads) pages_move_kernel(const __grid_constant__ PageBufs pb,
                                                                  const __grid_constant__ CompactArgs a, int pieces,
                                                                  const int32_t *table_in, int32_t *table_out,
                                                                  const int32_t *seq_lens, int n_slots,
                                                                  int max_pages, int remap) {
    wait_for_last();
    if ((int)blockIdx.x < remap) {
        const long long entries = (long long)n_slots * max_pages;
        for (long long e = (long long)blockIdx.x * kCopyThreads + threadIdx.x; e < entries;
             e += (long long)remap * kCopyThreads) {
            const int s = (int)(e / max_pages), j = (int)(e % max_pages);
            const int p = table_in[e];
            const bool held = j < pages_of(max(seq_lens[s], 0)) && p >= 0 && p < a.num_pages;
            table_out[e] = held ? a.map[p] : -1;
        }
        return;
    }
    const long long work = (long long)*a.moves * pieces, hop = gridDim.x - remap;
    long long w = blockIdx.x - remap;
    int from = 0, to = 0;
    if (w < work) {
        from = a.highs[w / pieces];
        to = a.lows[w / pieces];
    }
    while (w < work) {
        const int piece = (int)(w % pieces), src = from, dst = to;
        w += hop;
        if (w < work) {
            from = a.highs[w / pieces];
            to = a.lows[w / pieces];
        }
        copy_piece(pb, piece, src, dst);
    }
}

PageBufs page_bufs(void *const *bases, const size_t *bytes, int n) {
    PageBufs pb{};
    for (int i = 0; i < n; ++i) {
        int sh = 4;
        while (sh > 0 && ((reinterpret_cast<uintptr_t>(bases[i]) | bytes[i]) & ((1u << sh) - 1))) --sh;
        pb.base[i] = static_cast<char *>(bases[i]);
        pb.page_bytes[i] = bytes[i];
        pb.shift[i] = sh;
        pb.units += (int)(bytes[i] >> sh);
        pb.units_end[i] = pb.units;
    }
    return pb;
}

int pieces_of(const PageBufs &pb) { return pb.units > kPiece ? (pb.units + kPiece - 1) / kPiece : 1; }

// CTAs of the cluster that reads the pool's counts.
unsigned ctas_of(int num_pages) { return num_pages <= kOneCtaPages ? 1 : kMaxCtas; }

}  // namespace

cudaError_t launch_pages_extend(const int32_t *slots, const int32_t *new_lens, int n, int32_t *block_table,
                                int n_slots, int max_pages, int32_t *seq_lens, int32_t *refcount, int num_pages,
                                int32_t *status, cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const GrantArgs a{slots, new_lens, n, block_table, n_slots, max_pages, seq_lens, refcount, num_pages, status};
    const unsigned ctas = ctas_of(num_pages);
    return EarlyLaunch(ctas, kThreads, 0, stream, ctas)(pages_grant_kernel<false>, a);
}

cudaError_t launch_pages_fork(void *const *bases, const size_t *bytes, int n_bufs, const int32_t *parents,
                              const int32_t *children, int n, int32_t *block_table, int n_slots, int max_pages,
                              int32_t *seq_lens, int32_t *refcount, int num_pages, int32_t *status,
                              cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const GrantArgs a{children, parents, n, block_table, n_slots, max_pages, seq_lens, refcount, num_pages, status};
    const unsigned ctas = ctas_of(num_pages);
    const cudaError_t e = EarlyLaunch(ctas, kThreads, 0, stream, ctas)(pages_grant_kernel<true>, a);
    if (e != cudaSuccess) return e;
    const PageBufs pb = page_bufs(bases, bytes, n_bufs);
    const int pieces = pieces_of(pb);
    return EarlyLaunch((unsigned)n * pieces, kCopyThreads, 0, stream)(pages_fork_kernel, pb, a, pieces);
}

cudaError_t launch_pages_free(const int32_t *slots, int n, int32_t *block_table, int n_slots, int max_pages,
                              int32_t *seq_lens, int32_t *refcount, int num_pages, cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    return EarlyLaunch(n, 256, 0, stream)(pages_free_kernel, slots, n, block_table, n_slots, max_pages, seq_lens,
                                          refcount, num_pages);
}

cudaError_t launch_pages_copy(void *const *bases, const size_t *bytes, int n_bufs, const int32_t *src,
                              const int32_t *dst, int n, int num_pages, cudaStream_t stream) {
    if (n == 0 || n_bufs == 0) return cudaSuccess;
    const PageBufs pb = page_bufs(bases, bytes, n_bufs);
    const int pieces = pieces_of(pb);
    const long long work = (long long)n * pieces;
    const unsigned grid = (unsigned)(work < (1ll << 30) ? work : (1ll << 30));
    return EarlyLaunch(grid, kCopyThreads, 0, stream)(pages_copy_kernel, pb, src, dst, n, pieces, num_pages);
}

size_t pages_compact_workspace_bytes(int num_pages) { return 16 + 2 * ((size_t)num_pages / 2 + 1) * sizeof(int32_t); }

cudaError_t launch_pages_compact(void *const *bases, const size_t *bytes, int n_bufs, const int32_t *table_in,
                                 int32_t *table_out, int n_slots, int max_pages, const int32_t *seq_lens,
                                 const int32_t *refs_in, int32_t *refs_out, int num_pages, int32_t *map,
                                 int32_t *n_used, void *ws, cudaStream_t stream) {
    int32_t *w = static_cast<int32_t *>(ws);
    const CompactArgs a{refs_in, refs_out, map, n_used, num_pages, w, w + 4, w + 4 + num_pages / 2 + 1};
    const unsigned ctas = ctas_of(num_pages);
    const cudaError_t e = EarlyLaunch(ctas, kThreads, 0, stream, ctas)(pages_plan_kernel, a);
    if (e != cudaSuccess) return e;
    const PageBufs pb = page_bufs(bases, bytes, n_bufs);
    const int pieces = pieces_of(pb);
    // one table entry per thread up to a wave's worth of CTAs
    const long long tiles = ((long long)n_slots * max_pages + kCopyThreads - 1) / kCopyThreads;
    const int remap = (int)(tiles < 148 * 4 ? tiles : 148 * 4);
    return EarlyLaunch(remap + 148 * kMoveCtas, kCopyThreads, 0, stream)(
        pages_move_kernel, pb, a, pieces, table_in, table_out, seq_lens, n_slots, max_pages, remap);
}

}  // namespace dsa
