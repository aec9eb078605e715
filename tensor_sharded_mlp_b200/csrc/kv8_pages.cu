// kv8_pages.cu -- the page map of the 8-bit key/value cache: reserving pages
// (with copy on write), forking, cutting and freeing sequences, copying pages
// and compacting the pool.
//
// The only record of a free page is its refcount of 0; "the lowest-numbered
// free pages, in the list's order" is then a prefix sum over the refcounts,
// which makes every result independent of timing.  One cluster of 8 CTAs does
// that sum: each CTA counts the free pages of an eighth of the pool (16-byte
// loads, one or two per thread at 64 Ki pages), the CTAs swap their counts
// through distributed shared memory, and a second walk hands out the ranks (pools
// of up to kMapOneCta pages take one CTA, whose threads keep their pages' bits).
// The data then moves in a second kernel over the whole GPU.
//
// Measured (B200): a compaction that moves 332 pages of 8 layers (697 MB read and
// written), with a saved map put back and a truncation before it, 128 us, 110 of
// them the copy = 6.35 TB/s, 0.97 of the copy rate; the same on a pool of 73
// pages 12.8 us; putting back, a fork and a reserve that copies 32 pages of 4
// layers 20.8 us.  A reserve of one token each, nothing to copy: 1 / 32 / 256 / 1024
// sequences 7.4 / 8.1 / 9.9 / 24 us (pool of 8192 pages; 65536: 8.2 / 9.1 / 11 / 25).
// Each entry's thread looks through the list in front of it for a repeat, and where
// pages are shared through the whole list for their holders: half the list's
// sequences sharing their last page with the other half, 32 / 256 / 1024 entries take
// 12 / 17 / 67 us with the copies.
#include <cuda_runtime.h>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "tc_ptx.cuh"

namespace tpmlp {
namespace {

constexpr int kMapCtas = 8;          // of one cluster, for large pools
constexpr int kMapOneCta = 16384;    // up to so many pages one CTA ranks them (16 a thread)
constexpr int kMapThreads = 1024;
constexpr int kMapWarps = kMapThreads / 32;
constexpr int kMaxList = TP_MLP_KV8_MAX_LIST;
static_assert(kMaxList == kMapThreads, "one thread per list entry");

// Workspace: [header | page pairs to copy | a list of pages | new index of every page]
struct PageWs {
    int *n_pairs;    // pairs that the copy kernel takes
    int *live;       // pages in use (compaction)
    int2 *pairs;     // (source, destination); negative: none
    int *list;
    int *remap;
};
constexpr size_t kHeaderBytes = 256;
size_t pair_slots(const Kv8 &c) { return c.num_pages > kMaxList ? (size_t)c.num_pages : (size_t)kMaxList; }
PageWs page_ws(const Kv8 &c, void *ws) {
    char *p = static_cast<char *>(ws);
    PageWs w;
    w.n_pairs = reinterpret_cast<int *>(p);
    w.live = w.n_pairs + 1;
    w.pairs = reinterpret_cast<int2 *>(p + kHeaderBytes);
    p += kHeaderBytes + align256(pair_slots(c) * sizeof(int2));
    w.list = reinterpret_cast<int *>(p);
    w.remap = reinterpret_cast<int *>(p + align256((size_t)c.num_pages * sizeof(int)));
    return w;
}

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cta_count() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_remote(const int *local, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(tc::cluster_addr(tc::smem_u32(local), rank)) : "memory");
    return v;
}

// The refcounts of pages q .. q + 3 (0 behind the pool's end is not "free":
// the caller masks by the page number).
__device__ __forceinline__ int4 load_refs(const Kv8 &c, int q) {
    if (q + 3 < c.num_pages) return *reinterpret_cast<const int4 *>(c.refcount + q);
    int4 r = make_int4(0, 0, 0, 0);
    if (q < c.num_pages) r.x = c.refcount[q];
    if (q + 1 < c.num_pages) r.y = c.refcount[q + 1];
    if (q + 2 < c.num_pages) r.z = c.refcount[q + 2];
    return r;
}

// The pool is cut into one contiguous span per warp of the cluster (a multiple
// of 128 pages: 32 lanes x 4).
struct Span {
    int lo, hi;
};
__device__ __forceinline__ Span warp_span(const Kv8 &c) {
    const int warps = cta_count() * kMapWarps;
    const int per = ((c.num_pages + warps - 1) / warps + 127) / 128 * 128;
    const long long lo = (long long)per * (cta_rank() * kMapWarps + (threadIdx.x >> 5));
    Span s;
    s.lo = (int)min(lo, (long long)c.num_pages);
    s.hi = (int)min(lo + per, (long long)c.num_pages);
    return s;
}

// Bit k set: page q + k is below `end` and its refcount marks it free (or used).
__device__ __forceinline__ uint32_t free_bits(int4 r, int q, int end) {
    const uint32_t in = q + 3 < end ? 15u : q + 2 < end ? 7u : q + 1 < end ? 3u : q < end ? 1u : 0u;
    return in & ((r.x == 0 ? 1u : 0u) | (r.y == 0 ? 2u : 0u) | (r.z == 0 ? 4u : 0u) | (r.w == 0 ? 8u : 0u));
}

// The first kAhead * 128 pages' bits of a span, loaded before they are needed: all of it for pools of up to
// kAhead * 128 * kMapWarps pages a CTA.
constexpr int kAhead = 4;
struct Ahead {
    uint32_t bits;   // 4 of each round
};
__device__ __forceinline__ Ahead load_ahead(const Kv8 &c, Span s) {
    const int lane = threadIdx.x & 31;
    int4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const long long q = (long long)s.lo + u * 128 + 4 * lane;
        r[u] = q < s.hi ? load_refs(c, (int)q) : make_int4(1, 1, 1, 1);
    }
    Ahead a = {0};
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const long long q = (long long)s.lo + u * 128 + 4 * lane;
        if (q < s.hi) a.bits |= free_bits(r[u], (int)q, s.hi) << (4 * u);
    }
    return a;
}
// This lane's free bits of the span's round u.
__device__ __forceinline__ uint32_t round_bits(const Kv8 &c, Span s, Ahead a, int u) {
    if (u < kAhead) return a.bits >> (4 * u) & 15u;
    const long long q = (long long)s.lo + u * 128LL + 4 * (threadIdx.x & 31);
    return q < s.hi ? free_bits(load_refs(c, (int)q), (int)q, s.hi) : 0u;
}
__device__ __forceinline__ int rounds_of(Span s) { return (s.hi - s.lo + 127) / 128; }

// Free pages in this warp's span, and the sums over the cluster: *before = free
// pages in front of the span, *all = free pages of the pool.  Every thread of
// the cluster calls it; it ends behind a cluster barrier.
__device__ void rank_free(const Kv8 &c, Span s, Ahead a, int *before, int *all) {
    __shared__ int warp_n[kMapWarps];
    __shared__ int cta_n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;
    for (int u = 0; u < rounds_of(s); ++u) n += __popc(round_bits(c, s, a, u));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) warp_n[warp] = n;
    __syncthreads();
    int mine = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kMapWarps; ++w) {
        total += warp_n[w];
        mine += w < warp ? warp_n[w] : 0;
    }
    if (threadIdx.x == 0) cta_n = total;
    cluster_sync();
    const int rank = (int)cta_rank(), ctas = cta_count();
    int sum = 0;
    for (int r = 0; r < ctas; ++r) {
        const int v = ld_remote(&cta_n, (uint32_t)r);
        sum += v;
        mine += r < rank ? v : 0;
    }
    *before = mine;
    *all = sum;
}

// This lane's place in a round: pages free in front of its first one, given those in front of the round.
__device__ __forceinline__ int lane_rank(uint32_t bits, int before, int *in_round) {
    const int lane = threadIdx.x & 31;
    int x = __popc(bits);
    const int mine = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    *in_round = __shfl_sync(0xffffffffu, x, 31);
    return before + x - mine;
}

// take(page, rank) for the free pages of this warp's span whose rank in the pool is below `total`.
template <typename Take>
__device__ __forceinline__ void for_free(const Kv8 &c, Span s, Ahead a, int before, int total, Take take) {
    for (int u = 0; u < rounds_of(s) && before < total; ++u) {
        uint32_t bits = round_bits(c, s, a, u);
        int in_round, rank = lane_rank(bits, before, &in_round);
        const int q = s.lo + u * 128 + 4 * (threadIdx.x & 31);
        for (; bits; bits &= bits - 1, ++rank)
            if (rank < total) take(q + __ffs(bits) - 1, rank);
        before += in_round;
    }
}

// Exclusive prefix sum over the block's threads, and the sum.
__device__ long long block_scan(long long v, long long *sum) {
    __shared__ long long part[kMapWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    long long base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMapWarps; ++w) {
        base += w < warp ? part[w] : 0;
        all += part[w];
    }
    *sum = all;
    return base + x - v;
}

// Entry i of the list belongs to thread i of every CTA: each CTA works out all
// entries' needs by itself (the list is short), so only the pool is shared out.
__global__ void __launch_bounds__(kMapThreads)
    reserve_kernel(Kv8 c, const int *seqs, const int *counts, int n, PageWs ws) {
    __shared__ int s_seq[kMaxList], s_last[kMaxList], s_len[kMaxList], s_slot[kMaxList];
    __shared__ long long s_base[kMaxList];
    const int i = threadIdx.x, lane = threadIdx.x & 31;
    const bool teller = cta_rank() == 0;   // flags and lengths are written once
    pdl_allow_dependents();
    pdl_wait_previous();
    int seq = -1, count = 0, len = 0, bad = 0;
    if (i < n) {
        seq = kv8_seq(seqs, i);
        count = counts[i];
        if (seq < -1 || seq >= c.max_seqs) {
            bad |= TP_MLP_KV8_BAD_SEQUENCE;
            seq = -1;
        }
        if (seq >= 0) len = c.lengths[seq];
    }
    const Span span = warp_span(c);
    const Ahead ahead = load_ahead(c, span);   // (on its way while the entries are worked out)
    s_seq[i] = seq;
    __syncthreads();
    if (seq >= 0 && seqs) {
        bool again = false;
        for (int j = 0; j < i; ++j) again |= s_seq[j] == seq;
        if (again) bad |= TP_MLP_KV8_BAD_SEQUENCE;
    }
    int last = -1, refs = 0;
    bool valid = seq >= 0 && !bad;
    if (valid) {
        if (len < 0 || count < 0 || (long long)len + count > c.capacity()) {
            bad |= TP_MLP_KV8_BAD_LENGTH;
            valid = false;
        } else if (count > 0 && (len & (c.page_size - 1))) {
            last = c.table[(long long)seq * c.max_pages + (len >> c.page_shift)];
            if ((unsigned)last >= (unsigned)c.num_pages) {
                bad |= TP_MLP_KV8_BAD_PAGE;
                valid = false;
                last = -1;
            } else {
                refs = c.refcount[last];
                if (refs <= 1) last = -1;   // the page is the sequence's own
            }
        }
    }
    s_last[i] = last;
    __syncthreads();
    bool own_copy = false;
    if (last >= 0) {   // shared: the first of the holders keeps it if all are here
        int here = 0;
        bool first = true;
        for (int j = 0; j < n; ++j) {
            const bool same = s_last[j] == last;
            here += same;
            first &= !(same && j < i);
        }
        own_copy = !(here == refs && first);
    }
    if (teller && bad) kv8_flag(c, bad);
    const int fresh = valid ? c.pages_of(len + count) - c.pages_of(len) : 0;
    // pages taken in the low 40 bits (at most 2^10 entries of 2^27 pages), copies above
    constexpr long long kPages = (1LL << 40) - 1;
    long long total;
    const long long scan = block_scan(fresh + (own_copy ? (1LL << 40) + 1 : 0), &total);
    const int copies = (int)(total >> 40);
    total &= kPages;
    __syncthreads();   // (s_last is read above)
    s_seq[i] = valid ? seq : -1;
    s_len[i] = len;
    s_base[i] = scan & kPages;
    s_last[i] = own_copy ? last : -1;
    s_slot[i] = (int)(scan >> 40);

    int before, all;
    rank_free(c, span, ahead, &before, &all);
    // (behind the cluster's barrier: every CTA has read the old map)
    const bool enough = total <= all;
    if (teller && i == 0) {
        if (!enough) kv8_flag(c, TP_MLP_KV8_NO_PAGES);
        *ws.n_pairs = enough ? copies : 0;
    }
    if (enough) {
        if (teller && valid) c.lengths[seq] = len + count;
        // the free page of rank r is the (r - base)-th of the entry whose pages start at base: its copy, then its new ones
        for_free(c, span, ahead, before, (int)total, [&](int page, int rank) {
            int lo = 0, hi = kMaxList;   // base(lo) <= rank < base(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_base[mid] <= rank) lo = mid;
                else hi = mid;
            }
            const int s = s_seq[lo], l = s_len[lo], from = s_last[lo], nth = rank - (int)s_base[lo];
            int *row = c.table + (long long)s * c.max_pages;
            c.refcount[page] = 1;
            if (from >= 0 && nth == 0) {
                row[l >> c.page_shift] = page;
                atomicSub(c.refcount + from, 1);   // at least one holder stays: the page is not taken for free
                ws.pairs[s_slot[lo]] = make_int2(from, page);
            } else {
                row[c.pages_of(l) + nth - (from >= 0)] = page;
            }
        });
    }
    cluster_sync();   // no CTA leaves while another may still read its count
}

constexpr int kRowThreads = 128;

// True in all threads if `value` is in list[0 .. n) (`list` NULL: never).
__device__ __forceinline__ bool block_finds(const int *list, int n, int value) {
    bool hit = false;
    if (list)
        for (int j = threadIdx.x; j < n; j += blockDim.x) hit |= list[j] == value;
    return __syncthreads_or(hit);
}

// One CTA per pair.
__global__ void __launch_bounds__(kRowThreads)
    fork_kernel(Kv8 c, const int *parents, const int *children, int n) {
    const int i = blockIdx.x;
    pdl_allow_dependents();
    pdl_wait_previous();
    const int parent = parents[i], child = children[i];
    if (parent == -1 || child == -1) return;
    bool bad = (unsigned)parent >= (unsigned)c.max_seqs || (unsigned)child >= (unsigned)c.max_seqs;
    if (!bad) {   // a child before, or a parent, in a pair that is in use: no CTA sees another's writes
        for (int j = threadIdx.x; j < n; j += kRowThreads) {
            const int p = parents[j], s = children[j];
            bad |= p != -1 && s != -1 && (p == child || (j < i && s == child));
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) kv8_flag(c, TP_MLP_KV8_BAD_SEQUENCE);
        return;
    }
    const int len = c.lengths[parent], was = c.lengths[child];
    __syncthreads();
    if (was != 0 || len < 0 || len > c.capacity()) {
        if (threadIdx.x == 0) kv8_flag(c, TP_MLP_KV8_BAD_LENGTH);
        return;
    }
    const int *from = c.table + (long long)parent * c.max_pages;
    int *to = c.table + (long long)child * c.max_pages;
    for (int k = threadIdx.x; k < c.pages_of(len); k += kRowThreads) {
        const int page = from[k];
        to[k] = page;
        if ((unsigned)page < (unsigned)c.num_pages) atomicAdd(c.refcount + page, 1);
        else kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
    }
    if (threadIdx.x == 0) c.lengths[child] = len;
}

// One CTA per sequence.
__global__ void __launch_bounds__(kRowThreads)
    truncate_kernel(Kv8 c, const int *seqs, const int *new_lengths, int n) {
    const int i = blockIdx.x;
    pdl_allow_dependents();
    pdl_wait_previous();
    const int seq = seqs[i];
    if (seq == -1) return;
    if ((unsigned)seq >= (unsigned)c.max_seqs || block_finds(seqs, i, seq)) {
        if (threadIdx.x == 0) kv8_flag(c, TP_MLP_KV8_BAD_SEQUENCE);
        return;
    }
    const int len = c.lengths[seq], cut = new_lengths ? new_lengths[i] : 0;
    __syncthreads();
    if (cut < 0 || cut > len || len > c.capacity()) {
        if (threadIdx.x == 0) kv8_flag(c, TP_MLP_KV8_BAD_LENGTH);
        return;
    }
    int *row = c.table + (long long)seq * c.max_pages;
    for (int k = c.pages_of(cut) + threadIdx.x; k < c.pages_of(len); k += kRowThreads) {
        const int page = row[k];
        row[k] = -1;
        if ((unsigned)page >= (unsigned)c.num_pages || atomicSub(c.refcount + page, 1) <= 0) {
            if ((unsigned)page < (unsigned)c.num_pages) atomicAdd(c.refcount + page, 1);   // it was free already
            kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
        }
    }
    if (threadIdx.x == 0) c.lengths[seq] = cut;
}

// Which pages move where: the pool's used pages at and behind L = their number,
// in order, to the free pages in front of L, in order.  A free page p < L is
// hole number (free pages before p); a used page p >= L is mover number
// (used pages before p) - (L - H), with H holes.
__global__ void __launch_bounds__(kMapThreads)
    compact_map_kernel(Kv8 c, PageWs ws) {
    __shared__ int warp_holes[kMapWarps];
    __shared__ int cta_holes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_allow_dependents();
    pdl_wait_previous();
    const Span span = warp_span(c);
    const Ahead ahead = load_ahead(c, span);
    int before, all;
    rank_free(c, span, ahead, &before, &all);
    const int live = c.num_pages - all;
    int holes = 0;
    for (int u = 0; u < rounds_of(span); ++u) {
        const long long q = (long long)span.lo + u * 128LL + 4 * lane;
        const uint32_t bits = round_bits(c, span, ahead, u);
        int in_round, rank = lane_rank(bits, before, &in_round);   // free pages before q
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const long long p = q + b;
            if (p >= span.hi) break;
            if (bits >> b & 1) {
                ws.remap[p] = -1;
                if (p < live) {
                    ws.pairs[rank].y = (int)p;
                    ++holes;
                }
                ++rank;
            } else if (p < live) {
                ws.remap[p] = (int)p;
            } else {
                ws.list[p - rank] = (int)p;   // used pages before p
            }
        }
        before += in_round;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) holes += __shfl_xor_sync(0xffffffffu, holes, o);
    if (lane == 0) warp_holes[warp] = holes;
    __syncthreads();
    if (threadIdx.x == 0) {
        int h = 0;
#pragma unroll
        for (int w = 0; w < kMapWarps; ++w) h += warp_holes[w];
        cta_holes = h;
    }
    cluster_sync();   // lists complete, refcounts read
    const int ctas = cta_count();
    int moves = 0;
    for (int r = 0; r < ctas; ++r) moves += ld_remote(&cta_holes, (uint32_t)r);
    for (int r = (int)cta_rank() * kMapThreads + threadIdx.x; r < moves; r += ctas * kMapThreads) {
        const int from = ws.list[live - moves + r], to = ws.pairs[r].y;
        ws.pairs[r].x = from;
        ws.remap[from] = to;
        c.refcount[to] = c.refcount[from];
        c.refcount[from] = 0;
    }
    if (cta_rank() == 0 && threadIdx.x == 0) {
        *ws.n_pairs = moves;
        *ws.live = live;
    }
    cluster_sync();   // no CTA leaves while another may still read its counts
}

// Copies of whole pages over all layers, keys and values and their scales, and
// (compaction) the table's entries brought to the new numbers.  The work is a
// row of tiles of up to kTile 16-byte words, pair-major, cut evenly over the
// grid, so a CTA changes its pair seldom.  HBM-bound: each byte is read and
// written once.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kTile = kCopyThreads * kCopyUnroll;

// `listed` >= 0: that many pairs, from the caller, to be checked; else the
// workspace's own.
__global__ void __launch_bounds__(kCopyThreads)
    page_copy_kernel(Kv8 c, const int2 *pairs, int listed, const int *n_pairs, const int *live, const int *remap) {
    pdl_allow_dependents();
    pdl_wait_previous();
    if (remap) {
        const int first_moved = *live;
        const long long entries = (long long)c.max_seqs * c.max_pages;
        const long long step = (long long)gridDim.x * kCopyThreads;
        for (long long e = (long long)blockIdx.x * kCopyThreads + threadIdx.x; e < entries; e += step) {
            const int p = c.table[e];
            if (p < first_moved) continue;
            const int to = p < c.num_pages ? remap[p] : -1;
            if (to >= 0) c.table[e] = to;
            else kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
        }
    }
    const int n = listed >= 0 ? listed : *n_pairs;
    const long long words = c.page_bytes() / 16, tiles = (words + kTile - 1) / kTile;
    const long long per_pair = tiles * c.layers * 2, total = per_pair * n;
    const long long t1 = total * (blockIdx.x + 1) / gridDim.x;
    int at = -1;
    int2 pair = make_int2(-1, -1);
    for (long long t = total * blockIdx.x / gridDim.x; t < t1; ++t) {
        const int p = (int)(t / per_pair);
        if (p != at) {
            at = p;
            pair = pairs[p];
            bool skip = pair.x < 0 || pair.y < 0 || pair.x == pair.y;
            if (listed >= 0 && !skip) {
                bool clash = false;
                for (int j = threadIdx.x; j < n; j += kCopyThreads) {
                    const int2 o = pairs[j];
                    clash |= o.x == pair.y && o.y >= 0 && o.y != o.x;
                    clash |= j < p && o.y == pair.y && o.x >= 0 && o.x != o.y;
                }
                clash |= pair.x >= c.num_pages || pair.y >= c.num_pages;
                if (__syncthreads_or(clash)) {
                    skip = true;
                    if (threadIdx.x == 0) kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
                }
            }
            if (skip) pair.x = -1;
        }
        if (pair.x < 0) {   // on to the next pair
            t = (long long)(p + 1) * per_pair - 1;
            continue;
        }
        const long long in_pair = t - (long long)p * per_pair;
        const long long item = in_pair / tiles;   // (layer, keys or values)
        const int tile = (int)(in_pair - item * tiles);
        const long long layer_pages = (item >> 1) * c.num_pages;
        uint8_t *pool = item & 1 ? c.v : c.k;
        const uint4 *src = reinterpret_cast<const uint4 *>(pool + (layer_pages + pair.x) * c.page_bytes());
        uint4 *dst = reinterpret_cast<uint4 *>(pool + (layer_pages + pair.y) * c.page_bytes());
        const long long w0 = (long long)tile * kTile + threadIdx.x;
        uint4 v[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (w0 + u * kCopyThreads < words) v[u] = ld_stream_v4(src + w0 + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (w0 + u * kCopyThreads < words) dst[w0 + u * kCopyThreads] = v[u];
        if (tile == 0 && (int)threadIdx.x < c.kv_heads) {
            float *scales = (item & 1 ? c.v_scale : c.k_scale) + layer_pages * c.kv_heads;
            scales[(long long)pair.y * c.kv_heads + threadIdx.x] = scales[(long long)pair.x * c.kv_heads + threadIdx.x];
        }
    }
}

unsigned map_ctas(const Kv8 &c) { return c.num_pages <= kMapOneCta ? 1 : kMapCtas; }

unsigned copy_grid(const Kv8 &c, long long pairs, int num_sms) {
    const long long tiles = (c.page_bytes() / 16 + kTile - 1) / kTile * c.layers * 2 * pairs;
    const long long most = 8LL * num_sms;   // (3 CTAs of 72 registers a thread are resident: 2.7 rounds)
    return (unsigned)(tiles < 1 ? 1 : tiles < most ? tiles : most);
}

}  // namespace

size_t kv8_pages_workspace(const Kv8 &c) {
    return kHeaderBytes + align256(pair_slots(c) * sizeof(int2)) + 2 * align256((size_t)c.num_pages * sizeof(int));
}

cudaError_t launch_kv8_reserve(const Kv8 &c, const int *seqs, const int *counts, int n, void *ws, int num_sms,
                               cudaStream_t st) {
    const PageWs w = page_ws(c, ws);
    const unsigned ctas = map_ctas(c);
    cudaError_t e = launch_pdl_cluster(reserve_kernel, dim3(ctas), dim3(kMapThreads), 0, st, ctas, c, seqs, counts, n, w);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_copy_kernel, dim3(copy_grid(c, n, num_sms)), dim3(kCopyThreads), 0, st, c,
                      static_cast<const int2 *>(w.pairs), -1, static_cast<const int *>(w.n_pairs),
                      static_cast<const int *>(nullptr), static_cast<const int *>(nullptr));
}

cudaError_t launch_kv8_fork(const Kv8 &c, const int *parents, const int *children, int n, cudaStream_t st) {
    return launch_pdl(fork_kernel, dim3((unsigned)n), dim3(kRowThreads), 0, st, c, parents, children, n);
}

cudaError_t launch_kv8_truncate(const Kv8 &c, const int *seqs, const int *new_lengths, int n, cudaStream_t st) {
    return launch_pdl(truncate_kernel, dim3((unsigned)n), dim3(kRowThreads), 0, st, c, seqs, new_lengths, n);
}

cudaError_t launch_kv8_copy_pages(const Kv8 &c, const int *pairs, int n, int num_sms, cudaStream_t st) {
    return launch_pdl(page_copy_kernel, dim3(copy_grid(c, n, num_sms)), dim3(kCopyThreads), 0, st, c,
                      reinterpret_cast<const int2 *>(pairs), n, static_cast<const int *>(nullptr),
                      static_cast<const int *>(nullptr), static_cast<const int *>(nullptr));
}

cudaError_t launch_kv8_compact(const Kv8 &c, int *new_index, void *ws, int num_sms, cudaStream_t st) {
    PageWs w = page_ws(c, ws);
    if (new_index) w.remap = new_index;
    const unsigned ctas = map_ctas(c);
    cudaError_t e = launch_pdl_cluster(compact_map_kernel, dim3(ctas), dim3(kMapThreads), 0, st, ctas, c, w);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_copy_kernel, dim3(copy_grid(c, c.num_pages, num_sms)), dim3(kCopyThreads), 0, st, c,
                      static_cast<const int2 *>(w.pairs), -1, static_cast<const int *>(w.n_pairs),
                      static_cast<const int *>(w.live), static_cast<const int *>(w.remap));
}

}  // namespace tpmlp
