// kv8_attention.cuh -- what the attention kernels over the paged 8-bit cache share: the call's entries and their prefix
// sums, register-level instructions, a row's result, and the kernel that joins what several CTAs share.
#pragma once

#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"
#include "tc_ptx.cuh"
#include "vec_io.cuh"

namespace tpmlp {
namespace {

constexpr int kStep = 16;            // tokens of one step
// A row's reference is set kLift (base-2 logs) below its largest s_t + log2(v_scale's binade), and stays until one exceeds
// it by kSlack.  So the weights that multiply values reach from 2^6 .. 2^15, in the upper range of fp16, and have its full
// precision down to 2^-14; one that is 2^-31 of the largest still counts (2^-25 is half of fp16's smallest number).
constexpr float kLift = 7.f, kSlack = 15.f;
constexpr int kLeastLog = -81;       // smallest binade of a value scale in R: 2^31 weights of 2^(15 + 81) have a finite sum
// fp32 results: what fp16 cuts off a weight is held this much larger, in fp16 too (at most 2^3 * 2^12 there).
constexpr float kLow = 4096.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxList = TP_MLP_KV8_MAX_LIST;
constexpr int kWideRows = 128;         // query rows of a tile of the kernel for many rows

// Workspace: [a segment to join per CTA | two pieces per CTA].  CTA i's is the segment that begins in it and goes on in
// the next ones: {entry, unit, CTAs that share it, -}, with a count of 0 for none.
struct Split {
    int4 *shared;
    float *pieces;
};

struct Entry {             // one entry of the call's list
    int seq, len;          // seq -1: passed over
    int first;             // position of its query 0, brought to [-128, len]: no token's visibility changes
    __device__ __forceinline__ int seen(int query) const { return max(0, min(len, first + query + 1)); }
};

// An entry as loaded (len and first only if seq is in the table) made safe: seq -1 and no tokens if it cannot be used.
__device__ __forceinline__ void check_entry(const Kv8 &c, Entry &e, int *bad) {
    if (e.seq != -1 && (unsigned)e.seq >= (unsigned)c.max_seqs) {
        *bad |= TP_MLP_KV8_BAD_SEQUENCE;
        e.seq = -1;
    } else if (e.seq >= 0 && (e.len < 0 || e.len > c.capacity())) {
        *bad |= TP_MLP_KV8_BAD_LENGTH;
        e.seq = -1;
    }
    if (e.seq < 0) e.len = 0;
    e.first = max(-TP_MLP_KV8_MAX_QUERIES, min(e.len, e.first));
}

// a / b for a >= 0, b > 0, by the short division where it can be.
__device__ __forceinline__ long long quotient(long long a, int b) {
    return a <= 0x7fffffffLL ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The entry that holds step x < prefix[n]: the last with prefix <= x (one warp, 32 probes a round).
__device__ __forceinline__ int entry_of(const long long *prefix, int n, long long x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int in = 31 - __clz(__ballot_sync(0xffffffffu, at < hi && prefix[at] <= x));   // (lane 0 always is)
        hi = min(hi, lo + (in + 1) * step);
        lo += in * step;
    }
    return lo;
}

// --- register-level pieces ------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool take) {
    const int bytes = take ? 16 : 0;   // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t p, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(p), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
    return v;
}
// four e4m3 bytes -> two f16x2 (bytes 0,1 and 2,3), exact
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 widen_f16x2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A sum of weights brought from its reference to one that is `d` <= 0 away; turn = 2^d.  Pages of zeros (the smallest scale)
// beside pages of large values put references more than 126 apart, and then the sum at the lower one is as much larger.
__device__ __forceinline__ float turn_sum(float sum, float turn, float d) {
    const float half = exp2_fast(0.5f * d);
    return turn >= FLT_MIN ? sum * turn : sum * half * half;
}
// Bytes of w that are e4m3 NaN, as 0xff each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Eight query elements as loaded.
template <typename T> struct RawQuery;
template <> struct RawQuery<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void widen(float *f) const {
        f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
        f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
    }
};
template <> struct RawQuery<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void widen(float *f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// A query row is brought to [2^14, 2^15) by a power of two (`down`), which the scores get back (`up`): the upper end of
// fp16, so that elements far below the row's largest (which may meet keys near zero) keep their bits too.  Rows below
// 2^-112 are brought up by 2^126 only, the largest power of two that has an inverse among normal numbers.
struct QueryScale {
    float down, up;
};
__device__ __forceinline__ QueryScale query_scale(float amax) {
    const int ex = max((int)(__float_as_uint(amax) >> 23) - 127, -112) - 14;   // -126 .. 113
    const float down = amax > FLT_MAX ? NAN   // an infinity in a row makes its scores, and so its result, NaN
                                      : __uint_as_float((uint32_t)(127 - ex) << 23);   // 2^-ex
    return {down, __uint_as_float((uint32_t)(ex + 127) << 23)};
}

// Where row r (0 .. q_len * group - 1) of (entry, KV head) is in q and the outputs.
struct RowMap {
    int entry, kv_head, group, q_len, heads;
    __device__ __forceinline__ int query(int r) const { return r / group; }
    __device__ __forceinline__ long long out_row(int r) const {
        const int j = r / group;
        return ((long long)entry * q_len + j) * heads + kv_head * group + (r - j * group);
    }
};

// A row's statistics in the result's terms.  ref: reference R, sum: sum of
// 2^(s - R), top: the row's true maximum score (base-2 logs).
struct RowResult {
    float factor;          // what the accumulated outputs are multiplied with
    float maximum, exp_sum;
};
__device__ __forceinline__ RowResult row_result(float ref, float sum, float top, bool partial) {
    RowResult r;
    if (!partial) {
        r.factor = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // nothing seen: zeros; NaN stays
        return r;
    }
    if (top == -INFINITY && sum == 0.f) {
        r.factor = 0.f;
        r.maximum = -INFINITY;
        r.exp_sum = 0.f;
        return r;
    }
    r.factor = exp2f(ref - top);
    r.exp_sum = sum * r.factor;
    r.maximum = isnan(sum) && top != INFINITY ? sum : top * kLn2;
    return r;
}

// Writes a joined row of the result (one warp).
template <typename T, int D>
__device__ __forceinline__ void write_row(const Kv8Query &a, long long orow, float ref, float sum, float top,
                                          const float4 (&v)[(D + 127) / 128]) {
    const int lane = threadIdx.x & 31;
    const RowResult res = row_result(ref, sum, top, a.maximum != nullptr);
#pragma unroll
    for (int x = 0; x < (D + 127) / 128; ++x) {
        if (D == 64 && lane >= 16) continue;
        store4(static_cast<T *>(a.o) + orow * D + 4 * (lane + 32 * x),
               make_float4(v[x].x * res.factor, v[x].y * res.factor, v[x].z * res.factor, v[x].w * res.factor));
    }
    if (a.maximum && lane == 0) {
        a.maximum[orow] = res.maximum;
        a.exp_sum[orow] = res.exp_sum;
    }
}

// The call's entries, each one's steps of `step` tokens, and the prefix sums of prefix[0 .. n] of units_per_entry * (steps +
// open) each (0 for an entry without steps), in shared memory; the caller's next barrier publishes them.
struct Entries {
    long long *prefix;
    int *seq, *len, *first, *steps;
};
template <int kThreads>
__device__ __forceinline__ void list_entries(const Kv8 &c, const Kv8Query &a, int units_per_entry, int step, int open,
                                             const Entries &out, long long *scan_part) {
    const int n = a.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kMost = (kMaxList + kThreads - 1) / kThreads;
    const int per = n <= kThreads ? 1 : kMost;   // consecutive entries of a thread
    long long mine[kMost], sum = 0;
    int bad = 0;
    Entry en[kMost];
    // (the loads of all entries before the first use)
#pragma unroll
    for (int u = 0; u < kMost; ++u) en[u].seq = u < per && tid * per + u < n ? kv8_seq(a.seqs, tid * per + u) : -1;
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const bool ok = (unsigned)en[u].seq < (unsigned)c.max_seqs;
        en[u].len = ok ? c.lengths[en[u].seq] : 0;
        en[u].first = ok && a.positions ? a.positions[tid * per + u] : en[u].len - a.q_len;
    }
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int i = tid * per + u;
        mine[u] = sum;
        if (u < per && i < n) {
            check_entry(c, en[u], &bad);
            const int steps = (en[u].seen(a.q_len - 1) + step - 1) / step;
            out.seq[i] = en[u].seq;
            out.len[i] = en[u].len;
            out.first[i] = en[u].first;
            out.steps[i] = steps;
            sum += (long long)(steps ? steps + open : 0) * units_per_entry;
        }
    }
    if (bad && blockIdx.x == 0) kv8_flag(c, bad);
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scan_part[warp] = x;
    __syncthreads();
    long long base = x - sum;
#pragma unroll
    for (int w = 0; w < (kThreads / 32); ++w) base += w < warp ? scan_part[w] : 0;
#pragma unroll
    for (int u = 0; u < kMost; ++u)
        if (u < per && tid * per + u <= n) out.prefix[tid * per + u] = base + mine[u];
    if (n == per * kThreads && tid == kThreads - 1) out.prefix[n] = base + sum;
}

// Entries that see nothing: their rows are written by the CTAs in turn (a few, if any).
template <typename T, int D, int kThreads>
__device__ __forceinline__ void write_unseen(const Kv8Query &a, const Entries &en) {
    for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
        if (en.steps[i] > 0 || en.seq[i] < 0) continue;
        const long long row0 = (long long)i * a.q_len * a.heads, row_n = (long long)a.q_len * a.heads;
        for (long long x = threadIdx.x; x < row_n * (D / 4); x += kThreads)
            store4(static_cast<T *>(a.o) + row0 * D + 4 * x, make_float4(0.f, 0.f, 0.f, 0.f));
        if (a.maximum)
            for (long long x = threadIdx.x; x < row_n; x += kThreads) {
                a.maximum[row0 + x] = -INFINITY;
                a.exp_sum[row0 + x] = 0.f;
            }
    }
}

// Joins the pieces of the segments that several CTAs share.  kJoinWarps warps take a row: warp w the pieces w, w +
// kJoinWarps, ...; their sums meet in shared memory.  A CTA has kJoinThreads / 32 / kJoinWarps rows.
constexpr int kJoinThreads = 256;

template <typename T, int D, int kRows, int kJoinWarps>
__global__ void __launch_bounds__(kJoinThreads)
    combine_kernel(Kv8 c, Kv8Query a, Split ws, int row_tiles) {
    constexpr int kCols = (D + 127) / 128, kJoinRows = kJoinThreads / 32 / kJoinWarps;
    __shared__ float4 part[kJoinRows][kJoinWarps][kCols * 32];
    __shared__ float4 part_stat[kJoinRows][kJoinWarps];
    pdl_allow_dependents();
    pdl_wait_previous();
    const int4 d = ws.shared[blockIdx.x];
    const int count = d.z;
    if (count == 0) return;
    const int kv_head = d.y / row_tiles, tile = d.y - kv_head * row_tiles;
    const RowMap map = {d.x, kv_head, a.heads / c.kv_heads, a.q_len, a.heads};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, my_row = warp / kJoinWarps, w = warp % kJoinWarps;
    const int in_tile = blockIdx.y * kJoinRows + my_row, r = tile * kRows + in_tile;
    float ref = -INFINITY, sum = 0.f, top = -INFINITY;
    float4 v[kCols];
#pragma unroll
    for (int x = 0; x < kCols; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = w; p < count; p += kJoinWarps) {
        const float *pc = ws.pieces + ((size_t)(blockIdx.x + p) * 2 + (p == 0 ? 1 : 0)) * (kRows * (D + 4));
        const float4 stat = *reinterpret_cast<const float4 *>(pc + kRows * D + in_tile * 4);
        const float m = fmaxf(ref, stat.x);
        const float f0 = ref == m ? 1.f : exp2f(ref - m), f1 = stat.x == m ? 1.f : exp2f(stat.x - m);
        sum = turn_sum(sum, f0, ref - m) + turn_sum(stat.y, f1, stat.x - m);
        ref = m;
        top = fmaxf(top, stat.z);
#pragma unroll
        for (int x = 0; x < kCols; ++x)
            if (D != 64 || lane < 16) {
                const float4 y = *reinterpret_cast<const float4 *>(pc + in_tile * D + 4 * (lane + 32 * x));
                v[x].x = v[x].x * f0 + y.x * f1;
                v[x].y = v[x].y * f0 + y.y * f1;
                v[x].z = v[x].z * f0 + y.z * f1;
                v[x].w = v[x].w * f0 + y.w * f1;
            }
    }
#pragma unroll
    for (int x = 0; x < kCols; ++x) part[my_row][w][lane + 32 * x] = v[x];
    if (lane == 0) part_stat[my_row][w] = make_float4(ref, sum, top, 0.f);
    __syncthreads();
    if (w != 0 || r >= a.q_len * map.group) return;
    float m = ref;
#pragma unroll
    for (int p = 1; p < kJoinWarps; ++p) {
        m = fmaxf(m, part_stat[my_row][p].x);
        top = fmaxf(top, part_stat[my_row][p].z);
    }
    sum = 0.f;
#pragma unroll
    for (int x = 0; x < kCols; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kJoinWarps; ++p) {
        const float4 stat = part_stat[my_row][p];
        const float f = stat.x == m ? 1.f : exp2f(stat.x - m);
        sum += turn_sum(stat.y, f, stat.x - m);
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
            const float4 y = part[my_row][p][lane + 32 * x];
            v[x].x += y.x * f;
            v[x].y += y.y * f;
            v[x].z += y.z * f;
            v[x].w += y.w * f;
        }
    }
    write_row<T, D>(a, map.out_row(r), m, sum, top, v);
}

// Eight warps a row where a segment has many pieces, four (half as many CTAs) otherwise: one sequence of 200000 tokens with
// one KV head 26.3 against 30.8 us, of 20000 with two 14.5 / 17.2, of 4099 with eight 12.0 / 12.3; 16 sequences of 4000 with
// eight (128 segments) 32.7 / 31.9, 32 ragged ones 44.8 / 44.0.  One warp a row of the wide tiles, where the rows are many
// (128 rows of head_dim 128; 1 / 2 / 4 warps a row): 16 sequences of 4000 tokens 98 / 101 / 109 us, one 28.2 / 27.4 / 29.9.
template <typename T, int D, int kRows>
cudaError_t launch_combine(const Kv8 &c, const Kv8Query &a, const Split &s, int row_tiles, int num_sms, cudaStream_t st) {
    const int join_rows = min(kRows, (a.q_len * (a.heads / c.kv_heads) + 7) / 8 * 8);
    if constexpr (kRows == kWideRows) {
        return launch_pdl(combine_kernel<T, D, kRows, 1>, dim3((unsigned)num_sms, join_rows / 8), dim3(kJoinThreads), 0, st, c,
                          a, s, row_tiles);
    } else {
        if ((long long)a.n * c.kv_heads * row_tiles * 8 <= num_sms)
            return launch_pdl(combine_kernel<T, D, kRows, 8>, dim3((unsigned)num_sms, join_rows), dim3(kJoinThreads), 0, st, c,
                              a, s, row_tiles);
        return launch_pdl(combine_kernel<T, D, kRows, 4>, dim3((unsigned)num_sms, join_rows / 2), dim3(kJoinThreads), 0, st, c,
                          a, s, row_tiles);
    }
}

inline Split split_of(void *ws, int num_sms) {
    char *p = static_cast<char *>(ws);
    return Split{reinterpret_cast<int4 *>(p), reinterpret_cast<float *>(p + align256((size_t)num_sms * sizeof(int4)))};
}

}  // namespace
}  // namespace tpmlp
