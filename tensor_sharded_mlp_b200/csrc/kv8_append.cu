// kv8_append.cu -- quantising new key/value rows into the pages of the 8-bit cache.
//
// One unit of work is what a call writes into one page for one KV head, keys or
// values: `count` consecutive slots from slot `a` on.  With amax the largest
// finite magnitude of those rows, the page's scale becomes
//   s = f(amax)                 if a == 0 (the page starts with these rows),
//   s = max(s_old, f(amax))     otherwise,   f(x) = 2^ceil(log2(x / 448)) >= 2^-100,
// and the codes are e4m3(x / s), an exact division before one rounding.  If s
// grows, the codes in slots < a become e4m3(code * s_old / s): a shift of the
// exponent, exact except for results in e4m3's subnormal range.
//
// A unit is read once into registers (as far as kKeep vectors a thread hold
// it; a larger one is read again, from L2), its maximum is taken, and the codes
// are written: HBM-bound for prompts (2 or 4 bytes read, 1 written per element).
#include <float.h>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;    // vectors of 8 elements a thread keeps between the two passes

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

// Maximum over the group of G threads that works on one unit.
template <int G>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (G > 32) {
        __shared__ float part[kThreads / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, part[w]);
    }
    return m;
}

// Units: ((sequence and page) x kv_heads + head) x 2 + (keys or values).
// Without cu, entry i has `slots` page slots; with cu, entry i's slots start at
// cu[i] / page_size + 2 i: n rows touch at most n / page_size + 2 pages, and
// floor(a + b) >= floor(a) + floor(b), so the ranges do not overlap.
// G = 32: a warp per unit (few rows); G = kThreads: a CTA per unit.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Kv8 c, const T *k, const T *v, long long row_stride, int tokens, const int *seqs, const int *cu,
                  int n, int slots, long long units) {
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31, me = threadIdx.x & (G - 1);
    const long long unit = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    pdl_wait_previous();
    if (unit >= units) return;
    const int values = (int)(unit & 1);
    const long long slot_head = unit >> 1;
    const long long slot = slot_head / c.kv_heads;
    const int head = (int)(slot_head - slot * c.kv_heads);
    const bool teller = head == 0 && values == 0 && me == 0;

    int i, row0, count;
    long long j;   // which of the entry's pages
    if (cu) {
        // the last entry whose slots start at or before this one: 32 probes a round
        int lo = 0, hi = n;   // start(lo) <= slot < start(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + lane * step;
            const bool in = at < hi && (at == lo || (long long)(cu[at] >> c.page_shift) + 2LL * at <= slot);
            const uint32_t m = __ballot_sync(0xffffffffu, in);
            const int k_in = 31 - __clz(m);   // lane 0 is always in
            hi = min(hi, lo + (k_in + 1) * step);
            lo = lo + k_in * step;
        }
        i = lo;
        row0 = cu[i];
        const int end = cu[i + 1];
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
    const int seq = kv8_seq(seqs, i);
    if (seq == -1) return;
    if ((unsigned)seq >= (unsigned)c.max_seqs || kv8_repeats(seqs, i, seq)) {
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
    if ((unsigned)page >= (unsigned)c.num_pages) {
        if (teller) kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
        return;
    }
    if (c.refcount[page] > 1) {
        if (teller) kv8_flag(c, TP_MLP_KV8_SHARED_PAGE);
        return;
    }
    const int t0 = j == 0 ? 0 : (int)(nth << c.page_shift) - start;   // first row of this page
    const int a = j == 0 ? start & (c.page_size - 1) : 0;
    const int rows = min(c.page_size - a, count - t0);
    const int D = c.head_dim, per_row = D / 8, vecs = rows * per_row;
    const T *x = (values ? v : k) + (row0 + (long long)t0) * row_stride + (long long)head * D;
    uint8_t *codes = (values ? c.v : c.k) + ((long long)page * c.kv_heads + head) * c.page_size * D;
    float *scale = (values ? c.v_scale : c.k_scale) + (long long)page * c.kv_heads + head;

    const float old = a ? *scale : 0.f;   // read by all before anyone writes it (the maximum's exchange is between)
    Vec8<T> kept[kKeep];
    float amax = 0.f;
    const int row_shift = 31 - __clz(per_row);   // head_dim is a power of two
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
        const int e = me + u * G;
        if (e < vecs) kept[u].load(x + (long long)(e >> row_shift) * row_stride + (e & (per_row - 1)) * 8);
    }
#pragma unroll
    for (int u = 0; u < kKeep; ++u)
        if (me + u * G < vecs) {
            float f[8];
            kept[u].widen(f);
#pragma unroll
            for (int q = 0; q < 8; ++q) amax = finite_max(amax, f[q]);
        }
    for (int e = me + kKeep * G; e < vecs; e += G) {
        Vec8<T> r;
        r.load(x + (long long)(e >> row_shift) * row_stride + (e & (per_row - 1)) * 8);
        float f[8];
        r.widen(f);
#pragma unroll
        for (int q = 0; q < 8; ++q) amax = finite_max(amax, f[q]);
    }
    amax = group_max<G>(amax);
    const float s = a ? fmaxf(old, step_of(amax)) : step_of(amax);
    const float inv = 1.f / s;   // exact for a power of two
    auto put = [&](const Vec8<T> &r, int e) {
        float f[8];
        r.widen(f);
        uint2 w;
        w.x = e4m3_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        w.y = e4m3_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
        *reinterpret_cast<uint2 *>(codes + (long long)a * D + 8LL * e) = w;   // the slots' rows follow each other
    };
#pragma unroll
    for (int u = 0; u < kKeep; ++u)
        if (me + u * G < vecs) put(kept[u], me + u * G);
    for (int e = me + kKeep * G; e < vecs; e += G) {
        Vec8<T> r;
        r.load(x + (long long)(e >> row_shift) * row_stride + (e & (per_row - 1)) * 8);
        put(r, e);
    }
    if (a && s > old) {
        const float ratio = old * inv;
        uint4 *held = reinterpret_cast<uint4 *>(codes);
        for (int e = me; e < a * D / 16; e += G) {
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
    if (me == 0) *scale = s;
}

template <typename T>
cudaError_t launch_typed(const Kv8 &c, const void *k, const void *v, long long row_stride, int tokens,
                         const int *seqs, const int *cu, int n, cudaStream_t st) {
    int slots = 0;
    long long all;
    int rows;   // rows of one page that a call writes at most
    if (cu) {
        all = (long long)(tokens >> c.page_shift) + 2LL * n;
        rows = tokens < c.page_size ? tokens : c.page_size;
    } else {
        const int each = tokens / n;
        slots = each <= 1 ? 1 : ((each - 2) >> c.page_shift) + 2;
        all = (long long)slots * n;
        rows = each < c.page_size ? each : c.page_size;
    }
    const long long units = all * c.kv_heads * 2;
    const T *tk = static_cast<const T *>(k), *tv = static_cast<const T *>(v);
    // a warp holds kKeep * 32 vectors: up to there it needs no second read and no barrier
    if (rows * (c.head_dim / 8) <= kKeep * 32) {
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
