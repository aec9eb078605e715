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
// maxima are taken, and the codes are written: HBM-bound for prompts (2 or 4
// bytes read, 1 written per element).  For a decode step the chain of
// dependent loads is what counts: the lists go to shared memory in one round
// trip (where the entry is searched and checked for repeats), then the length,
// then the table's entry and the rows together.
#include <float.h>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;    // vectors of 8 elements of keys (and of values) a thread keeps between the two passes
constexpr int kMaxList = TP_MLP_KV8_MAX_LIST;

// Eight consecutive elements as loaded.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = ld_stream_v4(p); }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
        f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
    }
};
template <> struct Vec8<float> {
    uint4 u, w;
    __device__ __forceinline__ void load(const float *p) { u = ld_stream_v4(p); w = ld_stream_v4(p + 4); }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
        f[4] = __uint_as_float(w.x); f[5] = __uint_as_float(w.y); f[6] = __uint_as_float(w.z); f[7] = __uint_as_float(w.w);
    }
};

// 2^ceil(log2(amax / 448)), at least 2^-100, from amax's bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ float step_of(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < -100 ? -100 : e;   // (zero and subnormal maxima land here)
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float finite_max(float m, float x) {
    const float a = fabsf(x);
    return a <= FLT_MAX ? fmaxf(m, a) : m;
}

// Maxima over the group of G threads that works on one unit.
template <int G>
__device__ __forceinline__ float2 group_max(float2 m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
        m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
    }
    if (G > 32) {
        __shared__ float2 part[kThreads / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            m.x = fmaxf(m.x, part[w].x);
            m.y = fmaxf(m.y, part[w].y);
        }
    }
    return m;
}

template <typename T>
__device__ __forceinline__ void take_max(const Vec8<T> &r, float &m) {
    float f[8];
    r.widen(f);
#pragma unroll
    for (int q = 0; q < 8; ++q) m = finite_max(m, f[q]);
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

// Units: (sequence and page) x kv_heads + head, keys and values together.
// Without cu, entry i has `slots` page slots; with cu, entry i's slots start at
// cu[i] / page_size + 2 i: n rows touch at most n / page_size + 2 pages, and
// floor(a + b) >= floor(a) + floor(b), so the ranges do not overlap.
// G = 32: a warp per unit; G = kThreads: a CTA per unit.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Kv8 c, const T *k, const T *v, long long row_stride, int tokens, const int *seqs, const int *cu,
                  int n, int slots, long long units) {
    __shared__ int s_seq[kMaxList], s_cu[kMaxList + 1];
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31, me = threadIdx.x & (G - 1);
    const long long unit = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    pdl_wait_previous();
    for (int x = threadIdx.x; x <= n; x += kThreads) {
        if (x < n) s_seq[x] = kv8_seq(seqs, x);
        if (cu) s_cu[x] = cu[x];
    }
    __syncthreads();
    if (unit >= units) return;
    const long long slot = unit / c.kv_heads;
    const int head = (int)(unit - slot * c.kv_heads);
    const bool teller = head == 0 && me == 0;

    int i, row0, count;
    long long j;   // which of the entry's pages
    if (cu) {
        // the last entry whose slots start at or before this one: 32 probes a round
        int lo = 0, hi = n;   // start(lo) <= slot < start(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + lane * step;
            const bool in = at < hi && (at == lo || (long long)(s_cu[at] >> c.page_shift) + 2LL * at <= slot);
            const int k_in = 31 - __clz(__ballot_sync(0xffffffffu, in));   // lane 0 is always in
            hi = min(hi, lo + (k_in + 1) * step);
            lo = lo + k_in * step;
        }
        i = lo;
        row0 = s_cu[i];
        const int end = s_cu[i + 1];
        j = slot - ((long long)(row0 >> c.page_shift) + 2LL * i);
        if (row0 < 0 || end < row0 || end > tokens) {
            if (teller && j == 0) kv8_flag(c, TP_MLP_KV8_BAD_LENGTH);
            return;
        }
        count = end - row0;
    } else {
        i = (int)(slot / slots);
        j = slot - (long long)i * slots;
        count = tokens / n;
        row0 = i * count;
    }
    if (j < 0 || count == 0) return;
    const bool first = teller && j == 0;
    const int seq = s_seq[i];
    if (seq == -1) return;
    if ((unsigned)seq >= (unsigned)c.max_seqs || kv8_repeats(seqs ? s_seq : nullptr, i, seq)) {
        if (first) kv8_flag(c, TP_MLP_KV8_BAD_SEQUENCE);
        return;
    }
    const int len = c.lengths[seq], start = len - count;
    if (start < 0 || len > c.capacity()) {
        if (first) kv8_flag(c, TP_MLP_KV8_BAD_LENGTH);
        return;
    }
    const long long nth = (start >> c.page_shift) + j;
    if (nth > (len - 1) >> c.page_shift) return;
    const int page = c.table[(long long)seq * c.max_pages + nth];
    const int t0 = j == 0 ? 0 : (int)(nth << c.page_shift) - start;   // first row of this page
    const int a = j == 0 ? start & (c.page_size - 1) : 0;
    const int rows = min(c.page_size - a, count - t0);
    const int D = c.head_dim, per_row = D / 8, vecs = rows * per_row;
    const int row_shift = 31 - __clz(per_row);   // head_dim is a power of two
    const long long src = (row0 + (long long)t0) * row_stride + (long long)head * D;
    auto at = [&](int e) { return src + (long long)(e >> row_shift) * row_stride + (e & (per_row - 1)) * 8; };
    Vec8<T> kk[kKeep], kv[kKeep];
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
        const int e = me + u * G;
        if (e < vecs) {
            kk[u].load(k + at(e));
            kv[u].load(v + at(e));
        }
    }
    if ((unsigned)page >= (unsigned)c.num_pages) {
        if (teller) kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
        return;
    }
    if (c.refcount[page] > 1) {
        if (teller) kv8_flag(c, TP_MLP_KV8_SHARED_PAGE);
        return;
    }
    const long long where = (long long)page * c.kv_heads + head;
    // read by all threads before one of them writes it: the maxima's exchange lies between
    const float old_k = a ? c.k_scale[where] : 0.f, old_v = a ? c.v_scale[where] : 0.f;
    float2 amax = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kKeep; ++u)
        if (me + u * G < vecs) {
            take_max(kk[u], amax.x);
            take_max(kv[u], amax.y);
        }
    for (int e = me + kKeep * G; e < vecs; e += G) {
        Vec8<T> r, w;
        r.load(k + at(e));
        w.load(v + at(e));
        take_max(r, amax.x);
        take_max(w, amax.y);
    }
    amax = group_max<G>(amax);
    const float scale_k = a ? fmaxf(old_k, step_of(amax.x)) : step_of(amax.x);
    const float scale_v = a ? fmaxf(old_v, step_of(amax.y)) : step_of(amax.y);
    const float inv_k = 1.f / scale_k, inv_v = 1.f / scale_v;   // exact for powers of two
    uint8_t *codes_k = c.k + where * c.page_size * D, *codes_v = c.v + where * c.page_size * D;
    const long long skip = (long long)a * D;   // the slots' rows follow each other
#pragma unroll
    for (int u = 0; u < kKeep; ++u)
        if (me + u * G < vecs) {
            put_codes(codes_k + skip + 8LL * (me + u * G), kk[u], inv_k);
            put_codes(codes_v + skip + 8LL * (me + u * G), kv[u], inv_v);
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

template <typename T>
cudaError_t launch_typed(const Kv8 &c, const void *k, const void *v, long long row_stride, int tokens,
                         const int *seqs, const int *cu, int n, cudaStream_t st) {
    const int each = (tokens + n - 1) / n;   // rows of an entry; with cu, their mean
    int slots = 0;
    long long all;
    if (cu) {
        all = (long long)(tokens >> c.page_shift) + 2LL * n;
    } else {
        slots = each <= 1 ? 1 : ((each - 2) >> c.page_shift) + 2;
        all = (long long)slots * n;
    }
    const long long units = all * c.kv_heads;
    const T *tk = static_cast<const T *>(k), *tv = static_cast<const T *>(v);
    // a warp keeps kKeep * 32 vectors: up to there (on the mean) it needs no second read and no barrier
    if (each * (c.head_dim / 8) <= kKeep * 32) {
        const long long grid = (units + kThreads / 32 - 1) / (kThreads / 32);
        return launch_pdl(append_kernel<T, 32>, dim3((unsigned)grid), dim3(kThreads), 0, st, c, tk, tv, row_stride,
                          tokens, seqs, cu, n, slots, units);
    }
    return launch_pdl(append_kernel<T, kThreads>, dim3((unsigned)units), dim3(kThreads), 0, st, c, tk, tv, row_stride,
                      tokens, seqs, cu, n, slots, units);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8 &c, const void *k, const void *v, long long row_stride, int tokens,
                              const int *seqs, const int *cu, int n, int dtype, cudaStream_t st) {
    if (dtype == TP_MLP_F32) return launch_typed<float>(c, k, v, row_stride, tokens, seqs, cu, n, st);
    return launch_typed<__nv_bfloat16>(c, k, v, row_stride, tokens, seqs, cu, n, st);
}

}  // namespace tpmlp
