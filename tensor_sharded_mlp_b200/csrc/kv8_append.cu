// kv8_append.cu -- quantising new key/value rows into the pages of the 8-bit cache.
//
// One unit of work is what a call writes into one page for one KV head:
// consecutive slots from slot `a` on.  With amax the largest
// finite magnitude of those rows, the page's scale becomes
//   s = f(amax)                 if a == 0 (the page starts with these rows),
//   s = max(s_old, f(amax))     otherwise,   f(x) = 2^ceil(log2(x / 448)) >= 2^-100,
// and the codes are e4m3(x / s), an exact division before one rounding.  If s
// grows, the codes in slots < a become e4m3(code * s_old / s): a shift of the
// exponent, exact except for results in e4m3's subnormal range.
//
// Keys and values of a unit are read once into registers (as far as kKeep
// vectors a thread hold them; a larger unit is read again, from L2), the two
// maxima are taken, and the codes are written.  Prompts are HBM-bound (2 or 4
// bytes read, 1 written per element): a CTA takes a run of units, so that the
// chain of dependent loads in front of the rows (lists, length, page, refcount)
// is walked once for all of them.  For a decode step that chain is all there
// is: a warp takes a unit, and the rows are loaded beside the page's refcount.
//
// Measured (B200; bf16, 8 KV heads of 128, pages of 64): 8 prompts of 500 to
// 8001 tokens, 191 MB, 37.0 us = 5.2 TB/s, 0.79 of the copy rate: about 5 us of
// dependent loads before the first row, then issue slots (58 % busy) and the
// barrier of each unit's maximum; 256 single tokens 6.4 us.  Tried: two units'
// rows in registers (120 of them, 2 CTAs an SM) 53.6 us; prefetching the next
// unit into L2 41.6 against 39.5; 5 CTAs an SM 54.8.
#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "kv8_run.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;    // vectors of 8 elements of keys (and of values) a thread keeps between the two passes
constexpr int kMaxList = TP_MLP_KV8_MAX_LIST;
constexpr int kMaxSlots = 34;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight consecutive elements as loaded.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = ld_stream_v4(p); }
    // largest magnitude so far, as bits that compare like the numbers (infinities and NaN on top): two at a time
    using Most = uint32_t;
    __device__ __forceinline__ void raise(Most &m) const {
        m = max_u16x2(max_u16x2(m, u.x & 0x7fff7fffu), max_u16x2(u.y & 0x7fff7fffu, u.z & 0x7fff7fffu));
        m = max_u16x2(m, u.w & 0x7fff7fffu);
    }
    static __device__ __forceinline__ uint32_t bits(Most m) { return max(m & 0xffffu, m >> 16) << 16; }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
        f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
    }
};
template <> struct Vec8<float> {
    uint4 u, w;
    __device__ __forceinline__ void load(const float *p) { u = ld_stream_v4(p); w = ld_stream_v4(p + 4); }
    using Most = uint32_t;
    __device__ __forceinline__ void raise(Most &m) const {
        const uint32_t a = max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
        const uint32_t b = max(max(w.x & 0x7fffffffu, w.y & 0x7fffffffu), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
        m = max(m, max(a, b));
    }
    static __device__ __forceinline__ uint32_t bits(Most m) { return m; }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
        f[4] = __uint_as_float(w.x); f[5] = __uint_as_float(w.y); f[6] = __uint_as_float(w.z); f[7] = __uint_as_float(w.w);
    }
};

// 2^ceil(log2(amax / 448)), at least 2^-100, from amax's bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ float step_of(uint32_t b) {
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -100 ? -100 : e;   // (zero and subnormal maxima land here)
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Maxima over the group of G threads that works on one unit; `turn` alternates between the units of a CTA (for_units).
template <int G>
__device__ __forceinline__ uint2 group_max(uint32_t x, uint32_t y, int turn) {
    uint2 m = make_uint2(__reduce_max_sync(0xffffffffu, x), __reduce_max_sync(0xffffffffu, y));
    if (G > 32) {
        __shared__ uint2 part[2][kThreads / 32];   // (two: a warp may be a call ahead of one that still reads)
        if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            m.x = max(m.x, part[turn][w].x);
            m.y = max(m.y, part[turn][w].y);
        }
    }
    return m;
}

// The largest finite magnitude of a vector's elements (the rows hold infinities or NaN).
template <typename T>
__device__ __forceinline__ uint32_t finite_max(const Vec8<T> &r, uint32_t m) {
    float f[8];
    r.widen(f);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t b = __float_as_uint(f[q]) & 0x7fffffffu;
        m = b < 0x7f800000u ? max(m, b) : m;
    }
    return m;
}

template <typename T>
__device__ __forceinline__ void put_codes(uint8_t *dst, const Vec8<T> &r, float inv) {
    float f[8];
    r.widen(f);
    uint2 w;
    w.x = e4m3_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    w.y = e4m3_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    *reinterpret_cast<uint2 *>(dst) = w;
}

// The codes in front of the new rows, brought to a grown scale.
__device__ __forceinline__ void rescale(uint8_t *codes, int bytes, float ratio, int me, int group) {
    uint4 *held = reinterpret_cast<uint4 *>(codes);
    for (int e = me; e < bytes / 16; e += group) {
        const uint4 h = held[e];
        const uint32_t in[4] = {h.x, h.y, h.z, h.w};
        uint32_t out[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 f = e4m3_unpack4(in[q]);
            out[q] = e4m3_pack4(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio);
        }
        held[e] = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

// The rows that a call writes into one page.
struct Slot {
    long long row;   // first input row
    int page;        // -1: nothing to write
    int a, rows;     // first slot of the page, number
};

// Lists of the call, in shared memory.
struct Lists {
    const int *seq, *cu;   // cu NULL: even shares; else ascending within the input, with kBadRows in places
    bool listed;           // the call has a list of sequences (which may repeat itself)
};
constexpr int kBadRows = 1 << 30;   // in cu[i]: entry i is left out

// The slots of a call are pages of its entries.  Without cu, entry i has `each`
// of them; with cu, entry i's start at cu[i] / page_size + 2 i: n rows touch at
// most n / page_size + 2 pages, and floor(a + b) >= floor(a) + floor(b), so the
// ranges do not overlap.  One warp; `teller`: it sets the flags for this slot.
// The page's refcount is checked by the caller, beside the rows' loads.
__device__ __forceinline__ Slot find_slot(const Kv8 &c, Lists l, long long slot, int n, int each, int tokens, bool teller) {
    const int lane = threadIdx.x & 31;
    Slot out = {0, -1, 0, 0};
    teller &= lane == 0;
    int i, row0, count;
    long long j;   // which of the entry's pages
    if (l.cu) {
        // the last entry whose slots start at or before this one: 32 probes a round
        int lo = 0, hi = n;   // start(lo) <= slot < start(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + lane * step;
            const bool in = at < hi && (at == lo || (long long)((l.cu[at] & ~kBadRows) >> c.page_shift) + 2LL * at <= slot);
            const int k_in = 31 - __clz(__ballot_sync(0xffffffffu, in));   // lane 0 is always in
            hi = min(hi, lo + (k_in + 1) * step);
            lo = lo + k_in * step;
        }
        i = lo;
        row0 = l.cu[i];
        if (row0 & kBadRows) return out;   // (flagged with the list)
        j = slot - ((long long)(row0 >> c.page_shift) + 2LL * i);
        count = (l.cu[i + 1] & ~kBadRows) - row0;
    } else {
        i = (int)(slot / each);
        j = slot - (long long)i * each;
        count = tokens / n;
        row0 = i * count;
    }
    const int seq = l.seq[i];
    if (j < 0 || seq == -1) return out;
    if ((unsigned)seq >= (unsigned)c.max_seqs || kv8_repeats(l.listed ? l.seq : nullptr, i, seq)) {
        if (teller && j == 0) kv8_flag(c, TP_MLP_KV8_BAD_SEQUENCE);
        return out;
    }
    const int len = c.lengths[seq], start = len - count;
    if (start < 0 || len > c.capacity()) {
        if (teller && j == 0) kv8_flag(c, TP_MLP_KV8_BAD_LENGTH);
        return out;
    }
    if (count == 0) return out;
    const long long nth = (start >> c.page_shift) + j;
    if (nth > (len - 1) >> c.page_shift) return out;
    const int page = c.table[(long long)seq * c.max_pages + nth];
    const int t0 = j == 0 ? 0 : (int)(nth << c.page_shift) - start;   // the page's first row of the entry
    out.row = row0 + (long long)t0;
    out.a = j == 0 ? start & (c.page_size - 1) : 0;
    out.rows = min(c.page_size - out.a, count - t0);
    if ((unsigned)page < (unsigned)c.num_pages) out.page = page;
    else if (teller) kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
    return out;
}

// One unit, slot (with a page) and head, by a group of G threads.  `checked`: the page is known not to be shared.
template <typename T, int G>
__device__ __forceinline__ void append_unit(const Kv8 &c, const T *k, const T *v, long long row_stride, const Slot &sl,
                                            int head, bool checked, int turn) {
    const int me = threadIdx.x & (G - 1);
    const int D = c.head_dim, per_row = D / 8, vecs = sl.rows * per_row, a = sl.a;
    const int row_shift = 31 - __clz(per_row);   // head_dim is a power of two
    const long long src = sl.row * row_stride + (long long)head * D;
    auto at = [&](int e) { return src + (long long)(e >> row_shift) * row_stride + (e & (per_row - 1)) * 8; };
    Vec8<T> kk[kKeep], kv[kKeep];
#pragma unroll
    for (int x = 0; x < kKeep; ++x) {
        const int e = me + x * G;
        if (e < vecs) {
            kk[x].load(k + at(e));
            kv[x].load(v + at(e));
        }
    }
    if (!checked && c.refcount[sl.page] > 1) {
        if (me == 0 && head == 0) kv8_flag(c, TP_MLP_KV8_SHARED_PAGE);
        return;
    }
    const long long where = (long long)sl.page * c.kv_heads + head;
    // read by all threads before one of them writes it: the maxima's exchange lies between
    const float old_k = a ? c.k_scale[where] : 0.f, old_v = a ? c.v_scale[where] : 0.f;
    typename Vec8<T>::Most most_k = 0, most_v = 0;
#pragma unroll
    for (int x = 0; x < kKeep; ++x)
        if (me + x * G < vecs) {
            kk[x].raise(most_k);
            kv[x].raise(most_v);
        }
    for (int e = me + kKeep * G; e < vecs; e += G) {
        Vec8<T> r, w;
        r.load(k + at(e));
        w.load(v + at(e));
        r.raise(most_k);
        w.raise(most_v);
    }
    uint2 amax = group_max<G>(Vec8<T>::bits(most_k), Vec8<T>::bits(most_v), turn);
    if (max(amax.x, amax.y) >= 0x7f800000u) {   // only the finite ones count (the whole group is here)
        uint32_t fk = 0, fv = 0;
        for (int e = me; e < vecs; e += G) {
            Vec8<T> r, w;
            r.load(k + at(e));
            w.load(v + at(e));
            fk = finite_max(r, fk);
            fv = finite_max(w, fv);
        }
        if (G > 32) __syncthreads();   // (everyone has read the exchange's last values)
        amax = group_max<G>(fk, fv, turn);
    }
    const float scale_k = a ? fmaxf(old_k, step_of(amax.x)) : step_of(amax.x);
    const float scale_v = a ? fmaxf(old_v, step_of(amax.y)) : step_of(amax.y);
    const float inv_k = 1.f / scale_k, inv_v = 1.f / scale_v;   // exact for powers of two
    uint8_t *codes_k = c.k + where * c.page_size * D, *codes_v = c.v + where * c.page_size * D;
    const long long skip = (long long)a * D;   // the slots' rows follow each other
#pragma unroll
    for (int x = 0; x < kKeep; ++x)
        if (me + x * G < vecs) {
            put_codes(codes_k + skip + 8LL * (me + x * G), kk[x], inv_k);
            put_codes(codes_v + skip + 8LL * (me + x * G), kv[x], inv_v);
        }
    for (int e = me + kKeep * G; e < vecs; e += G) {
        Vec8<T> r, w;
        r.load(k + at(e));
        w.load(v + at(e));
        put_codes(codes_k + skip + 8LL * e, r, inv_k);
        put_codes(codes_v + skip + 8LL * e, w, inv_v);
    }
    if (a && scale_k > old_k) rescale(codes_k, a * D, old_k * inv_k, me, G);
    if (a && scale_v > old_v) rescale(codes_v, a * D, old_v * inv_v, me, G);
    if (me == 0) {
        c.k_scale[where] = scale_k;
        c.v_scale[where] = scale_v;
    }
}

// Brings a list of row bounds that is not ascending from 0 on within the input into that order (the search for a slot's
// entry needs it), marks the entries whose own bounds are wrong (they begin before an earlier bound, or end before they
// begin or behind the input), and flags them.  All threads of the block.
__device__ __noinline__ void order_rows(const Kv8 &c, const int *s_seq, int *s_cu, bool listed, int n, int tokens) {
    if (threadIdx.x == 0) {
        int most = 0, at = s_cu[0];
        for (int i = 0; i < n; ++i) {
            const int next = s_cu[i + 1];
            const bool ok = at >= most && next >= at && next <= tokens;
            most = min(max(most, at), tokens);
            s_cu[i] = ok ? most : most | kBadRows;
            at = next;
        }
        s_cu[n] = min(max(most, at), tokens);
    }
    __syncthreads();
    if (blockIdx.x != 0) return;
    for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {
        const int seq = s_seq[i];
        if (!(s_cu[i] & kBadRows) || seq == -1) continue;
        const bool bad_seq = (unsigned)seq >= (unsigned)c.max_seqs || kv8_repeats(listed ? s_seq : nullptr, i, seq);
        if ((threadIdx.x & 31) == 0) kv8_flag(c, bad_seq ? TP_MLP_KV8_BAD_SEQUENCE : TP_MLP_KV8_BAD_LENGTH);
    }
}

__device__ __forceinline__ Lists take_lists(const Kv8 &c, int *s_seq, int *s_cu, const int *seqs, const int *cu, int n,
                                            int tokens) {
    bool off = false;
    for (int x = threadIdx.x; x <= n; x += kThreads) {
        if (x < n) s_seq[x] = kv8_seq(seqs, x);
        if (cu) {
            const int at = cu[x];
            s_cu[x] = at;
            off |= at < 0 || at > tokens || (x < n && cu[x + 1] < at);
        }
    }
    if (__syncthreads_or(off)) order_rows(c, s_seq, s_cu, seqs != nullptr, n, tokens);
    return Lists{s_seq, cu ? s_cu : nullptr, seqs != nullptr};
}

// A warp per unit (slot x kv_heads + head).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    append_few_kernel(Kv8 c, const T *k, const T *v, long long row_stride, int tokens, const int *seqs, const int *cu,
                      int n, int each, long long units) {
    __shared__ int s_seq[kMaxList], s_cu[kMaxList + 1];
    pdl_allow_dependents();
    const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait_previous();
    const Lists l = take_lists(c, s_seq, s_cu, seqs, cu, n, tokens);
    if (unit >= units) return;
    const long long slot = unit / c.kv_heads;
    const int head = (int)(unit - slot * c.kv_heads);
    const Slot sl = find_slot(c, l, slot, n, each, tokens, head == 0);
    if (sl.page >= 0) append_unit<T, 32>(c, k, v, row_stride, sl, head, false, 0);
}

// The CTA works on the units units * b / grid .. units * (b + 1) / grid - 1 one after the other; its slots (at most
// kMaxSlots) are found first, a warp each.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    append_run_kernel(Kv8 c, const T *k, const T *v, long long row_stride, int tokens, const int *seqs, const int *cu,
                      int n, int each, long long units) {
    __shared__ int s_seq[kMaxList], s_cu[kMaxList + 1];
    __shared__ Slot s_slot[kMaxSlots];
    pdl_allow_dependents();
    const long long u0 = units * blockIdx.x / gridDim.x;
    const int run = (int)(units * (blockIdx.x + 1) / gridDim.x - u0);
    const long long slot0 = u0 / c.kv_heads;
    const int head0 = (int)(u0 - slot0 * c.kv_heads);
    pdl_wait_previous();
    const Lists l = take_lists(c, s_seq, s_cu, seqs, cu, n, tokens);
    for (int x = threadIdx.x >> 5; x * c.kv_heads < head0 + run; x += kThreads / 32) {
        const bool teller = x > 0 || head0 == 0;   // the CTA that holds a slot's first unit sets its flags
        Slot sl = find_slot(c, l, slot0 + x, n, each, tokens, teller);
        if (sl.page >= 0 && c.refcount[sl.page] > 1) {
            if (teller && (threadIdx.x & 31) == 0) kv8_flag(c, TP_MLP_KV8_SHARED_PAGE);
            sl.page = -1;
        }
        if ((threadIdx.x & 31) == 0) s_slot[x] = sl;
    }
    __syncthreads();
    for_units(
        run, head0, c.kv_heads, [&](int x) { return s_slot[x].page >= 0; },
        [&](int x, int head, int turn) { append_unit<T, kThreads>(c, k, v, row_stride, s_slot[x], head, true, turn); });
}

template <typename T>
cudaError_t launch_typed(const Kv8 &c, const void *k, const void *v, long long row_stride, int tokens,
                         const int *seqs, const int *cu, int n, int num_sms, cudaStream_t st) {
    const int mean = (tokens + n - 1) / n;   // rows of an entry (with cu: on the mean)
    const int each = mean <= 1 ? 1 : ((mean - 2) >> c.page_shift) + 2;
    const long long slots = cu ? (long long)(tokens >> c.page_shift) + 2LL * n : (long long)each * n;
    const long long units = slots * c.kv_heads;
    const T *tk = static_cast<const T *>(k), *tv = static_cast<const T *>(v);
    // a warp keeps kKeep * 32 vectors: up to there (on the mean) it needs no second read and no barrier
    if (mean * (c.head_dim / 8) <= kKeep * 32) {
        const long long grid = (units + kThreads / 32 - 1) / (kThreads / 32);
        return launch_pdl(append_few_kernel<T>, dim3((unsigned)grid), dim3(kThreads), 0, st, c, tk, tv, row_stride,
                          tokens, seqs, cu, n, each, units);
    }
    // as many CTAs as are resident at once, if their slots fit (a run touches run / kv_heads + 2 slots at most)
    const long long resident = (long long)num_sms * (sizeof(T) == 2 ? 4 : 2);
    const long long most = (long long)(kMaxSlots - 2) * c.kv_heads;
    long long grid = (units + most - 1) / most;
    if (grid < resident) grid = units < resident ? units : resident;
    return launch_pdl(append_run_kernel<T>, dim3((unsigned)grid), dim3(kThreads), 0, st, c, tk, tv, row_stride, tokens,
                      seqs, cu, n, each, units);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8 &c, const void *k, const void *v, long long row_stride, int tokens,
                              const int *seqs, const int *cu, int n, int dtype, int num_sms, cudaStream_t st) {
    if (dtype == TP_MLP_F32) return launch_typed<float>(c, k, v, row_stride, tokens, seqs, cu, n, num_sms, st);
    return launch_typed<__nv_bfloat16>(c, k, v, row_stride, tokens, seqs, cu, n, num_sms, st);
}

}  // namespace tpmlp
