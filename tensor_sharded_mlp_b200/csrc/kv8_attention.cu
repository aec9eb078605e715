// kv8_attention.cu -- attention over the paged 8-bit key/value cache.
//
// For a query row (query j of an entry, head h) and the tokens t that it sees:
//   s_t = scale * k_scale * (q . k_t),   m = max s_t,   p_t = exp(s_t - m),
//   out = sum p_t v_scale v_t / sum p_t.
//
// A decode step reads every cached byte once and does 4 * rows flops with it,
// rows = q_len * heads / kv_heads: HBM-bound.  The kernel's shape follows from
// keeping the loads going:
//
// * The work is a row of steps of 16 tokens -- entry by entry, KV head by KV
//   head, tile of query rows by tile -- cut evenly over all warps of the GPU
//   (prefix sums over the lengths, on the device: the lengths are not known to
//   the host).  A warp owns its steps: it streams their keys and values through
//   a ring of its own in shared memory (cp.async, no block-wide barrier) and
//   keeps running maxima, sums and outputs in registers.
// * Both products are mma.m16n8k16 with the tokens (or the value columns) as
//   the M side and 8 query rows as N, so a group of up to 8 heads fills the
//   tile.  e4m3 to fp16 is exact.  Keys: a thread's 16 loaded bytes are the
//   k-elements of four mma steps (the head dimension may be taken in any order,
//   the same one for the queries).  Values: two tokens' bytes are interleaved
//   (prmt) into the (token, token + 1) pairs that the A operand holds, and a
//   thread ends up with head_dim / 8 consecutive output columns.  The weights
//   turn from the first product's C layout to the second's B layout by
//   movmatrix; nothing passes through shared memory between the products.
// * The scales are constant over a step (a step lies in one page): the key
//   scale multiplies the scores, the value scale the weights.
//
// Precision.  Queries are brought to [2^14, 2^15) by a power of two per row and
// held in fp16, exactly for bf16 input (but for elements 2^-31 below the row's
// largest, whose error is 2^-39 of it); fp32 input is held as two fp16 parts
// (22 bits of an element, 2^-39 of the largest at worst).  The running reference
// R is the maximum of s_t + log2(v_scale's binade), in base-2 logs, less 7, so
// that the largest weight that multiplies the values, w_t = 2^(s_t - R) v_scale,
// lies between 2^6 and 2^15 whatever the pages' scales.  It is rounded to fp16
// for bf16 results (2^-11 of it, under the result's 2^-8; below 2^-20 of the
// largest weight an absolute 2^-31 of that) and held as two parts for fp32, the
// lower 2^12 times as large (2^-22 of it; 2^-43 of the largest).  R moves only
// when a score exceeds it by 2^15 (one vote a step; the sums are rescaled then).
// Scores, sums and outputs are fp32; the mma's own sum, which cuts what it
// shifts out, carries bf16 outputs over a warp's share (at most 2^-23 a step of
// 16 tokens, so 2^-11 at 64 Ki tokens).  2^(s_t - R) is 2^6 / v_scale at the
// largest score, so above a v_scale of 2^90 the exp2, which ends at 2^-126, loses
// weights of 2^-132 v_scale of the largest and less; one that does not took a
// third longer for 128 rows.  Below a v_scale of 2^-81 (kLeastLog) the largest
// weight is lower than 2^6, and what counts ends at 2^-112 / v_scale of it.
//
// Warps whose pieces meet in one segment (entry, KV head, row tile) join them
// in shared memory; pieces of a segment that CTAs share go to the workspace (at
// most two per CTA) and a second kernel joins them, in order, so the result
// does not depend on timing.  Masked places: bytes behind a sequence's end are
// never loaded (zero-filled), a masked score is -inf before it is used, and a
// NaN value that only some rows see is taken out of the product and put into
// just their outputs.
//
// Measured (B200; 64 heads on 8 KV heads of 128, bf16): 32 sequences of 20001
// to 36001 tokens, 1.84 GB, 285-290 us = 6.3-6.5 TB/s, 0.97-0.99 of the copy
// rate (295-310 us in thousands of calls in a row, under the power cap); 32 of
// 300 to 6000 tokens 44.7 us, of which a kernel that loads the same and computes
// nothing takes 42.5: lists, first loads, joins and the second launch are some
// 10 us; one sequence of 4099 tokens 12.2 us.  fp32, 16 sequences of 4000 tokens,
// 8 / 16 / 32 / 64 / 128 rows a KV head: 29 / 37 / 62 / 101 / 186 us for head_dim 64,
// 37 / 57 / 94 / 172 / 321 for 128, 59 / 98 / 178 / 340 / 680-750 for 256 (21 us of bytes at
// 128): every row tile reads and converts the history again; of it the lower parts'
// scaling is 3-5 %.  What was tried beside this form:
//   12 or 16 warps a CTA: more pieces to join, 1.04-1.1 times as long;
//   one step at a time instead of two: 332 against 309 us under the power cap;
//   the score product on the 8-bit mma with the query as two e4m3 parts: 279
//     against 288 us in short runs, 328 against 295 under the cap (twice the
//     multiplies), and 2-4 us more where segments are short;
//   the last CTA to arrive joining a segment in the same kernel: 13.8 -> 17.9 us
//     for one sequence, 44.7 -> 46.5 for 32.
#include <type_traits>

#include "kv8_attention.cuh"

namespace tpmlp {
namespace {

constexpr int kOpen = 3;             // steps that a segment's start and end cost beside its own, about

// Shared memory: [ring of every warp | first piece of every warp | scales of every ring place | where joined rows go |
// prefix of the entries' steps | entries | piece table].  A warp leaves at most two pieces, at the start and at the end
// of its steps; the second lies in its ring, which is idle then.
template <int D, int NT>
struct Cfg {
    static constexpr int kWarps = 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = 8 * NT;
    static constexpr int kStage = 2 * kStep * D;                       // keys and values of one step
    // steps whose products are worked on together
    static constexpr int kPair = D * NT <= 128 ? 2 : 1;
    static constexpr int kStages = D == 256 ? 2 : D == 64 ? 6 : NT == 1 ? 5 : 4;
    static constexpr int kRing = kStage * kStages;
    static constexpr int kPad = D + 4;                                  // floats a piece's row takes
    static constexpr int kPiece = kRows * (kPad + 4) * 4;               // outputs, reference, sum, maximum
    static_assert(kPiece <= kRing, "the second piece lies in the ring");
    static constexpr size_t kScaleOff = (size_t)kWarps * (kRing + kPiece);
    static constexpr size_t kJoinOff = kScaleOff + kWarps * kStages * 8;
    static constexpr size_t kPrefixOff = kJoinOff + 2 * kWarps * kRows * 8;
    static constexpr size_t smem(int n) { return kPrefixOff + (size_t)(n + 1) * 8 + (size_t)n * 16 + kWarps * 2 * 4; }
};

// Byte offset of 16-byte chunk ch of row `row` in a stage's keys or values.  For
// rows of 128 bytes and more the chunks are swizzled so that the 8 lanes of a
// load phase (two neighbouring rows of keys with chunks 2t + const, or four
// even rows of values with two chunks) touch 8 different 16-byte banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
    return (uint32_t)(row * D + ((D >= 128 ? ch ^ (row & 7) : ch) << 4));
}
// The chunk of a key row that thread t of a quad takes as its i-th.
template <int D>
__device__ __forceinline__ int key_chunk(int t, int i) {
    return D == 64 ? t : 8 * (i >> 1) + 2 * t + (i & 1);
}

// --- the streaming kernel ----------------------------------------------------------
template <typename T, int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1)
    attention_kernel(Kv8 c, Kv8Query a, Split ws, int row_tiles) {
    using C = Cfg<D, NT>;
    constexpr bool kExact = sizeof(T) == 4;       // two fp16 parts for queries and weights
    constexpr int kParts = kExact ? 2 : 1;
    constexpr int kKs = D / 16;                   // mma steps of the score product
    constexpr int kMt = D / 16;                   // 16-column tiles of the output product
    extern __shared__ __align__(128) unsigned char smem[];
    const int n = a.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = a.heads / c.kv_heads, rows = a.q_len * group;
    const int units_per_entry = c.kv_heads * row_tiles;
    const uint32_t ring = tc::smem_u32(smem) + warp * C::kRing;
    const uint32_t scales = tc::smem_u32(smem) + (uint32_t)C::kScaleOff + warp * C::kStages * 8;
    auto piece_at = [&](int w, int p) {
        return reinterpret_cast<float *>(smem + (p ? (size_t)w * C::kRing : (size_t)C::kWarps * C::kRing + (size_t)w * C::kPiece));
    };
    long long *prefix = reinterpret_cast<long long *>(smem + C::kPrefixOff);
    int *e_seq = reinterpret_cast<int *>(prefix + n + 1), *e_len = e_seq + n, *e_first = e_len + n;
    int *e_steps = e_first + n;       // of one segment of the entry
    int *piece_seg = e_steps + n;
    uintptr_t *join_to = reinterpret_cast<uintptr_t *>(smem + C::kJoinOff);
    __shared__ long long scan_part[C::kWarps];

    pdl_allow_dependents();
    pdl_wait_previous();

    // 1. the entries, the steps of each, and their prefix sums.  A segment takes kOpen places in front of its steps, so
    // that many short ones are not a warp's lot.
    list_entries<C::kThreads>(c, a, units_per_entry, kStep, kOpen, {prefix, e_seq, e_len, e_first, e_steps}, scan_part);
    if (lane < 2) piece_seg[warp * 2 + lane] = -1;
    __syncthreads();
    const long long total = prefix[n];
    const int ctas = (int)max(1LL, min((long long)gridDim.x, (total + C::kWarps - 1) / C::kWarps));
    // CTA i takes steps first_step(i) .. first_step(i + 1) - 1: equal shares, the first `extra` one step more
    const long long share = quotient(total, ctas);
    const int extra = (int)(total - share * ctas);
    auto first_step = [&](int i) { return share * i + min(i, extra); };
    write_unseen<T, D, C::kThreads>(a, {prefix, e_seq, e_len, e_first, e_steps});
    if (blockIdx.x >= ctas || total == 0) {
        if (tid == 0) ws.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    const long long c0 = first_step(blockIdx.x), c1 = first_step(blockIdx.x + 1);
    const long long w0 = c0 + (c1 - c0) * warp / C::kWarps, w1 = c0 + (c1 - c0) * (warp + 1) / C::kWarps;

    // 2. this warp's steps, segment by segment.  The loads run a ring ahead of the products, across segments.
    int e = 0, unit = 0, n_pieces = 0;
    if (w0 < w1) e = entry_of(prefix, n, w0);
    const int page_steps = c.page_shift - 4;            // log2(steps of a page)

    // The loading side: its segment (first step at lseg; steps ls .. lend - 1 are this warp's), and the pages of its batch
    // of 32 (lane x holds the x-th); the next batch's page numbers (of this segment, or the next one's first) are loaded
    // while this one is in use.  key_ptr and scale_ptr move on from step to step within a page.
    int le = e, lunit = 0, ls = 0, lend = 0, lbatch = 0, lpage = 0, npage = 0, llen = 0, lhead = 0;
    long long lseg = w1;
    const uint8_t *key_ptr = nullptr;
    const float *scale_ptr = nullptr;
    const long long to_values = c.v - c.k;
    uint32_t chunk[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) chunk[i] = chunk_at<D>((i * 32 + lane) / (D / 16), (i * 32 + lane) % (D / 16));
    auto load_pages = [&](int i, int b) {
        const int x = b * 32 + lane;
        return x < c.pages_of(e_len[i]) ? c.table[(long long)e_seq[i] * c.max_pages + x] : -1;
    };
    auto take_batch = [&]() {   // npage becomes the batch in use
        const bool ok = (unsigned)npage < (unsigned)c.num_pages;
        if (!ok && lbatch * 32 + lane <= (lend - 1) >> page_steps) kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
        lpage = ok ? npage : -1;
        if ((lend - 1) >> (page_steps + 5) > lbatch) {
            npage = load_pages(le, lbatch + 1);
        } else if (lseg + lend + kOpen < w1) {
            int i = le;
            if (lunit + 1 == units_per_entry)
                do ++i;
                while (e_steps[i] == 0);
            npage = load_pages(i, 0);
        }
    };
    bool work = w0 < w1;
    if (work) {
        const int steps = e_steps[e];
        unit = lunit = (int)quotient(w0 - prefix[e], steps + kOpen);
        lhead = lunit / row_tiles;
        llen = e_len[e];
        lseg = prefix[e] + (long long)lunit * (steps + kOpen) + kOpen;
        work = lseg < w1;
    }
    if (work) {
        ls = (int)max(0LL, w0 - lseg);
        lend = (int)min((long long)e_steps[e], w1 - lseg);
        lbatch = ls >> (page_steps + 5);
        npage = load_pages(e, lbatch);
    }
    bool turn_page = true;
    auto fetch = [&](int place) {
        if (ls == lend) {                                  // the next segment
            if (lseg + lend + kOpen >= w1) return;
            lseg += lend + kOpen;
            if (++lunit == units_per_entry) {
                lunit = 0;
                do ++le;
                while (e_steps[le] == 0);
                llen = e_len[le];
            }
            lhead = lunit / row_tiles;
            ls = 0;
            lend = (int)min((long long)e_steps[le], w1 - lseg);
            lbatch = 0;
            take_batch();
            turn_page = true;
        } else if (ls >> (page_steps + 5) != lbatch) {
            lbatch = ls >> (page_steps + 5);
            take_batch();
        }
        if (turn_page) {
            const int p = __shfl_sync(0xffffffffu, lpage, (ls >> page_steps) & 31);
            const long long head = (long long)(p < 0 ? 0 : p) * c.kv_heads + lhead;
            key_ptr = p < 0 ? nullptr : c.k + (head * c.page_size + ((ls * kStep) & (c.page_size - 1))) * D + 16 * lane;
            scale_ptr = (lane ? c.v_scale : c.k_scale) + head;
        }
        const uint32_t dst = ring + place * C::kStage;
        const int live = key_ptr ? llen - ls * kStep : 0;      // rows behind the end are zeros
        if (live >= kStep) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                cp_async16(dst + chunk[i], key_ptr + 512 * i);
                cp_async16(dst + kStep * D + chunk[i], key_ptr + to_values + 512 * i);
            }
        } else {
            const uint8_t *src = key_ptr ? key_ptr : c.k;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const bool take = (i * 32 + lane) / (D / 16) < live;
                cp_async16_or_zero(dst + chunk[i], src + 512 * i, take);
                cp_async16_or_zero(dst + kStep * D + chunk[i], src + to_values + 512 * i, take);
            }
        }
        if (!key_ptr) {
            if (lane == 0) sts64(scales + place * 8, 0.f, -1.f);   // negative: not a page of the pool
        } else if (lane < 2) {
            cp_async4(scales + place * 8 + lane * 4, scale_ptr);
        }
        ++ls;
        turn_page = (ls & ((1 << page_steps) - 1)) == 0;
        if (key_ptr) key_ptr += kStep * D;
    };
    // The products' side: segment (e, unit), of which this warp has steps s0 .. s1 - 1 and is at s.
    constexpr bool kAhead = NT == 1 && (!kExact || D == 64);   // queries are loaded ahead where the registers hold them
    RawQuery<T> raw[NT][D / 32];
    auto load_queries = [&]() {
        const int kv_head = unit / row_tiles, tile = unit - kv_head * row_tiles;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = (tile * NT + nt) * 8 + g, rr = r < rows ? r : 0, j = rr / group;
            const T *src = static_cast<const T *>(a.q) + ((long long)e * a.q_len + j) * a.row_stride +
                           (long long)(kv_head * group + rr - j * group) * D;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                raw[nt][2 * i].load(src + key_chunk<D>(t, i) * 16);
                raw[nt][2 * i + 1].load(src + key_chunk<D>(t, i) * 16 + 8);
            }
        }
    };
    uint32_t q[kParts][NT][kKs][2];
    float fac[NT][2];
    int limit[NT][2];      // tokens that the column's row sees
    int plain = 0;
    float o[NT][kMt][4], ref[NT][2], sum[NT][2], top[NT][2];
    int steps = 0, s0 = 0, s1 = 0, s = 0;
    long long first = lseg;   // where the segment's steps begin
    if (work) {
        if (kAhead) load_queries();
        steps = e_steps[e];
        s = s0 = ls;
        s1 = lend;
        take_batch();
    }
    // One step's products (kUnits = 1), or two unmasked ones' together: the two chains of dependent instructions
    // overlap.
    auto products = [&](auto units, const uint32_t *stage, const float *kscale, const float *vscale) {
        constexpr int kUnits = decltype(units)::value;
        // scores: 16 tokens x 8 rows a tile
        float sc[kUnits][NT][4], sc2[kUnits][NT][4];      // two sums: half as long a chain of dependent products
#pragma unroll
        for (int y = 0; y < kUnits; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[y][nt][k] = sc2[y][nt][k] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int y = 0; y < kUnits; ++y) {
                const uint4 lo4 = lds128(stage[y] + chunk_at<D>(g, key_chunk<D>(t, i)));
                const uint4 hi4 = lds128(stage[y] + chunk_at<D>(g + 8, key_chunk<D>(t, i)));
                const uint32_t lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a0, a1, a2, a3;
                    e4m3_to_f16(lo[w], a0, a2);
                    e4m3_to_f16(hi[w], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int pt = 0; pt < kParts; ++pt)
                            mma(w & 1 ? sc2[y][nt] : sc[y][nt], a0, a1, a2, a3, q[pt][nt][4 * i + w][0],
                                q[pt][nt][4 * i + w][1]);
                }
            }
        // base-2 scores; vlog: the binade above the value scale
        float vlog[kUnits];
        const bool masked = kUnits == 1 && s >= plain;
        bool rise = false;
#pragma unroll
        for (int y = 0; y < kUnits; ++y) {
            vlog[y] = (float)max((int)(__float_as_uint(vscale[y]) >> 23) - 126, kLeastLog);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x = (sc[y][nt][k] + sc2[y][nt][k]) * (fac[nt][k & 1] * kscale[y]);
                    if (masked && s * kStep + g + 8 * (k >> 1) >= limit[nt][k & 1]) x = -INFINITY;
                    sc[y][nt][k] = x;
                    rise |= x - ref[nt][k & 1] > kSlack - vlog[y];   // (a difference: exact however large the scores)
                    top[nt][k & 1] = fmaxf(top[nt][k & 1], x);
                }
        }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float m = -INFINITY;
#pragma unroll
                    for (int y = 0; y < kUnits; ++y) m = fmaxf(m, fmaxf(sc[y][nt][x], sc[y][nt][x + 2]) + (vlog[y] - kLift));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    m = fmaxf(ref[nt][x], m);
                    const float turn = m == ref[nt][x] ? 1.f : exp2_fast(ref[nt][x] - m);
                    sum[nt][x] = turn_sum(sum[nt][x], turn, ref[nt][x] - m);
                    ref[nt][x] = m;
#pragma unroll
                    for (int mt = 0; mt < kMt; ++mt) {
                        o[nt][mt][x] *= turn;
                        o[nt][mt][x + 2] *= turn;
                    }
                }
        }
        uint32_t w[kUnits][kParts][NT][2];      // weights as the second product's B operand
#pragma unroll
        for (int y = 0; y < kUnits; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[k] = exp2_fast(sc[y][nt][k] - ref[nt][k & 1]);
                    sum[nt][k & 1] += p[k];
                    p[k] *= vscale[y];
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t h = f16x2(p[2 * x], p[2 * x + 1]);
                    w[y][0][nt][x] = transpose8x8(h);
                    if (kExact) {
                        const float2 b = widen_f16x2(h);
                        w[y][kParts - 1][nt][x] = transpose8x8(f16x2((p[2 * x] - b.x) * kLow, (p[2 * x + 1] - b.y) * kLow));
                    }
                }
            }

        // outputs: tokens 2t, 2t+1, 2t+8, 2t+9 of this thread, D / 8 columns from g on
#pragma unroll
        for (int y = 0; y < kUnits; ++y) {
            const uint32_t vals = stage[y] + kStep * D;
            uint32_t v[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 2 * t + (k & 1) + 8 * (k >> 1);
                if (D == 64) {
                    const uint2 x = lds64(vals + r * D + g * 8);
                    v[k][0] = x.x;
                    v[k][1] = x.y;
                } else {
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {
                        const uint4 x = lds128(vals + chunk_at<D>(r, g + 8 * i));
                        v[k][4 * i] = x.x;
                        v[k][4 * i + 1] = x.y;
                        v[k][4 * i + 2] = x.z;
                        v[k][4 * i + 3] = x.w;
                    }
                }
            }
            if (masked) {   // a NaN value must not reach rows that do not see its token (0 * NaN)
                uint32_t any = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) any |= nan_bytes(v[k][i]);
                if (__any_sync(0xffffffffu, any != 0)) {
                    uint32_t see[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int tok = s * kStep + g + 8 * x;
                            see[nt][x] = transpose8x8(f16x2(tok < limit[nt][0] ? 1.f : 0.f, tok < limit[nt][1] ? 1.f : 0.f));
                        }
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t nb[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            nb[k] = nan_bytes(v[k][i]);
                            v[k][i] &= ~nb[k];
                            nb[k] &= 0x38383838u;           // e4m3's 1
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t sel = h ? 0x7362u : 0x5140u;
                            uint32_t a0, a1, a2, a3;
                            e4m3_to_f16(__byte_perm(nb[0], nb[1], sel), a0, a1);
                            e4m3_to_f16(__byte_perm(nb[2], nb[3], sel), a2, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                mma(hit, a0, a1, a2, a3, see[nt][0], see[nt][1]);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (hit[k] > 0.f) o[nt][2 * i + h][k] = NAN;
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7362u : 0x5140u;   // (token, token + 1) pairs of two columns
                    uint32_t a0, a1, a2, a3;
                    e4m3_to_f16(__byte_perm(v[0][i], v[1][i], sel), a0, a1);
                    e4m3_to_f16(__byte_perm(v[2][i], v[3][i], sel), a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (!kExact) {
                            mma(o[nt][2 * i + h], a0, a1, a2, a3, w[y][0][nt][0], w[y][0][nt][1]);
                        } else {
                            // the mma's own sum cuts what it shifts out: over thousands of steps that adds up, so for
                            // fp32 results a step's sum is added by an instruction that rounds
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
                            mma(d, a0, a1, a2, a3, w[y][kParts - 1][nt][0], w[y][kParts - 1][nt][1]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) d[k] *= 1.f / kLow;
                            mma(d, a0, a1, a2, a3, w[y][0][nt][0], w[y][0][nt][1]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[nt][2 * i + h][k] += d[k];
                        }
                    }
                }
        }
    };
    // The ring: the products read at `place`, the next fetch goes to next_place; n_free places were read since the last
    // fetch.  Fetches fill the whole ring, so kStages - kPair groups may be open when the oldest kPair are needed.
    int place = 0, next_place = 0, n_free = C::kStages;
    while (work) {
        {
            const int kv_head = unit / row_tiles, tile = unit - kv_head * row_tiles;
            if (!kAhead) load_queries();
            const Entry en = {e_seq[e], e_len[e], e_first[e]};
            const RowMap map = {e, kv_head, group, a.q_len, a.heads};
            // queries: row g of each n-tile, this thread's columns of every k-step
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = (tile * NT + nt) * 8 + g;
                const bool have = r < rows;
                float f[D / 4];
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) raw[nt][i].widen(f + 8 * i);
#pragma unroll
                for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(f[i]));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const QueryScale qs = query_scale(amax);
#pragma unroll
                for (int k = 0; k < kKs; ++k) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float v0 = have ? f[4 * k + 2 * x] * qs.down : 0.f;
                        const float v1 = have ? f[4 * k + 2 * x + 1] * qs.down : 0.f;
                        q[0][nt][k][x] = f16x2(v0, v1);
                        if (kExact) {
                            const float2 h = widen_f16x2(q[0][nt][k][x]);
                            q[kParts - 1][nt][k][x] = f16x2(v0 - h.x, v1 - h.y);
                        }
                    }
                }
                const float up = have ? a.scale * kLog2e * qs.up : 0.f;
                const int lim = have ? en.seen(map.query(r)) : 0x7fffffff;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    fac[nt][x] = __shfl_sync(0xffffffffu, up, (2 * t + x) * 4);
                    limit[nt][x] = __shfl_sync(0xffffffffu, lim, (2 * t + x) * 4);
                }
            }
            // steps below `plain` need no mask: the tile's first row sees the fewest tokens
            plain = en.seen(map.query(tile * C::kRows)) / kStep;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int m = 0; m < kMt; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[nt][m][k] = 0.f;
                ref[nt][0] = ref[nt][1] = -FLT_MAX;   // finite: a masked score minus it is -inf, never NaN
                top[nt][0] = top[nt][1] = -INFINITY;
                sum[nt][0] = sum[nt][1] = 0.f;
            }
        }
        while (s < s1) {
            __syncwarp();   // every lane is done with the places that these fetches refill
            for (; n_free > 0; --n_free) {
                fetch(next_place);
                cp_commit();
                next_place = next_place + 1 == C::kStages ? 0 : next_place + 1;
            }
            cp_wait<C::kStages - C::kPair>();
            __syncwarp();
            const int place1 = place + 1 == C::kStages ? 0 : place + 1;
            const uint2 pair0 = lds64(scales + place * 8);
            if (C::kPair == 2 && s + 2 <= s1 && s + 2 <= plain) {
                const uint2 pair1 = lds64(scales + place1 * 8);
                const uint32_t at2[2] = {ring + place * C::kStage, ring + place1 * C::kStage};
                const float ks[2] = {__uint_as_float(pair0.x), __uint_as_float(pair1.x)};
                const float vs[2] = {__uint_as_float(pair0.y), __uint_as_float(pair1.y)};
                if (fminf(vs[0], vs[1]) >= 0.f) {
                    products(std::integral_constant<int, C::kPair>{}, at2, ks, vs);
                    s += 2;
                    n_free = 2;
                    place = place1 + 1 == C::kStages ? 0 : place1 + 1;
                    continue;
                }
            }
            const uint32_t at1[1] = {ring + place * C::kStage};
            const float ks[1] = {__uint_as_float(pair0.x)}, vs[1] = {__uint_as_float(pair0.y)};
            // (a negative value scale: not a page of the pool, nothing is seen)
            if (!(vs[0] < 0.f)) products(std::integral_constant<int, 1>{}, at1, ks, vs);
            ++s;
            n_free = 1;
            place = place1;
        }

        // the segment's end: its rows, or a piece of them
        const int done_e = e, done_unit = unit;
        const bool whole = s0 == 0 && s1 == steps;
        first += s1 + kOpen;
        work = first < w1;
        if (work) {
            if (++unit == units_per_entry) {
                unit = 0;
                do ++e;
                while (e_steps[e] == 0);
                steps = e_steps[e];
            }
            s = s0 = 0;
            s1 = (int)min((long long)steps, w1 - first);
            if (kAhead) load_queries();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) {
                    sum[nt][x] += __shfl_xor_sync(0xffffffffu, sum[nt][x], m);
                    top[nt][x] = fmaxf(top[nt][x], __shfl_xor_sync(0xffffffffu, top[nt][x], m));
                }
        __syncwarp();   // (a second piece overwrites the ring)
        const int kv_head = done_unit / row_tiles, tile = done_unit - kv_head * row_tiles;
        const RowMap map = {done_e, kv_head, group, a.q_len, a.heads};
        // (a whole segment is written, a piece of one goes to shared memory.  The thread's column of output
        // product 2 i + h, element pair (x, x + 2), is column(i) + 2 h (+ 1).)
        float *piece = piece_at(warp, n_pieces);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int in_tile = nt * 8 + 2 * t + x, r = tile * C::kRows + in_tile;
                float factor = 1.f;
                T *dst = nullptr;
                if (whole) {
                    if (r >= rows) continue;
                    const long long orow = map.out_row(r);
                    const RowResult res = row_result(ref[nt][x], sum[nt][x], top[nt][x], a.maximum != nullptr);
                    factor = res.factor;
                    dst = static_cast<T *>(a.o) + orow * D;
                    if (a.maximum && g == 0) {
                        a.maximum[orow] = res.maximum;
                        a.exp_sum[orow] = res.exp_sum;
                    }
                } else if (g == 0) {
                    float *stat = piece + C::kRows * C::kPad + in_tile * 4;
                    stat[0] = ref[nt][x];
                    stat[1] = sum[nt][x];
                    stat[2] = top[nt][x];
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int col = D == 64 ? g * 8 + 4 * i : 128 * (i >> 2) + g * 16 + 4 * (i & 3);
                    const float4 v4 = make_float4(o[nt][2 * i][x] * factor, o[nt][2 * i][x + 2] * factor,
                                                  o[nt][2 * i + 1][x] * factor, o[nt][2 * i + 1][x + 2] * factor);
                    if (whole) store4(dst + col, v4);
                    else *reinterpret_cast<float4 *>(piece + in_tile * C::kPad + col) = v4;
                }
            }
        if (!whole) {
            if (lane == 0) piece_seg[warp * 2 + n_pieces] = done_e * units_per_entry + done_unit;
            ++n_pieces;
        }
    }
    __syncthreads();

    // 3. join the pieces of each segment, in order; those of a segment that other CTAs share go to the workspace.  First a
    // thread per (piece, row) works out what the piece's row is multiplied with (and, for the segment's first piece,
    // where the result goes) ...
    constexpr int kPieces = 2 * C::kWarps;
    static_assert(kPieces < 32, "a lane per piece");
    const int seg = lane < kPieces ? piece_seg[lane] : -1;
    const uint32_t live = __ballot_sync(0xffffffffu, seg >= 0);
    const uint32_t before = live & ((1u << lane) - 1);
    const int seg_before = __shfl_sync(0xffffffffu, seg, before ? 31 - __clz(before) : lane);
    const uint32_t starts = __ballot_sync(0xffffffffu, seg >= 0 && (!before || seg_before != seg));
    // the pieces of the segment whose first piece is p0
    auto pieces_from = [&](int p0) {
        const uint32_t later = starts & ~((2u << p0) - 1);
        return live & ~((1u << p0) - 1) & (later ? (later & -later) - 1 : 0xffffffffu);
    };
    for (int x = tid; x < kPieces * C::kRows; x += C::kThreads) {
        const int p = x / C::kRows, in_tile = x % C::kRows;
        if (!(live >> p & 1)) continue;
        auto stat_of = [&](int i) {
            return reinterpret_cast<float4 *>(piece_at(i >> 1, i & 1) + C::kRows * C::kPad) + in_tile;
        };
        const int first = 31 - __clz(starts & ((2u << p) - 1)), sg = piece_seg[p];
        const uint32_t mine = pieces_from(first);
        const float own = stat_of(p)->x;
        float ref = own, l = 0.f, tp = -INFINITY;
        for (uint32_t m = mine; m; m &= m - 1) ref = fmaxf(ref, stat_of(__ffs(m) - 1)->x);
        for (uint32_t m = mine; m; m &= m - 1) {
            const float4 st = *stat_of(__ffs(m) - 1);
            l += turn_sum(st.y, st.x == ref ? 1.f : exp2f(st.x - ref), st.x - ref);
            tp = fmaxf(tp, st.z);
        }
        float f = own == ref ? 1.f : exp2f(own - ref);
        const int se = sg / units_per_entry, su = sg - se * units_per_entry, n_steps = e_steps[se];
        const long long seg0 = prefix[se] + (long long)su * (n_steps + kOpen) + kOpen;
        const int kv_head = su / row_tiles, row = (su - kv_head * row_tiles) * C::kRows + in_tile;
        uintptr_t to = 0;
        if (seg0 >= c0 && seg0 + n_steps <= c1) {
            const RowResult res = row_result(ref, l, tp, a.maximum != nullptr);
            f *= res.factor;
            if (row < rows && first == p) {
                const RowMap map = {se, kv_head, group, a.q_len, a.heads};
                const long long orow = map.out_row(row);
                to = reinterpret_cast<uintptr_t>(static_cast<T *>(a.o) + orow * D);
                if (a.maximum) {
                    a.maximum[orow] = res.maximum;
                    a.exp_sum[orow] = res.exp_sum;
                }
            }
        } else if (first == p) {
            float *out = ws.pieces + ((size_t)blockIdx.x * 2 + (seg0 < c0 ? 0 : 1)) * (C::kRows * (D + 4));
            *reinterpret_cast<float4 *>(out + C::kRows * D + in_tile * 4) = make_float4(ref, l, tp, 0.f);
            to = reinterpret_cast<uintptr_t>(out + in_tile * D) | 1;   // odd: fp32, not T
        }
        reinterpret_cast<float *>(stat_of(p))[3] = f;                   // (the others read only the first three)
        join_to[x] = first == p ? to : 0;
    }
    __syncthreads();
    // ... then a warp takes kRowsPer rows of a segment, a lane their columns.
    constexpr int kCols = (D + 127) / 128, kRowsPer = 4, kGroups = C::kRows / kRowsPer;
    const int tasks = __popc(starts) * kGroups;
    for (int task = warp; task < tasks; task += C::kWarps) {
        uint32_t left = starts;
        for (int i = task / kGroups; i > 0; --i) left &= left - 1;
        const int p0 = __ffs(left) - 1, row0 = task % kGroups * kRowsPer;
        const uint32_t mine = pieces_from(p0);
        float4 v[kRowsPer][kCols];
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k)
#pragma unroll
            for (int x = 0; x < kCols; ++x) v[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t m = mine; m; m &= m - 1) {
            const int p = __ffs(m) - 1;
            const float *pc = piece_at(p >> 1, p & 1);
#pragma unroll
            for (int k = 0; k < kRowsPer; ++k) {
                const float w = pc[C::kRows * C::kPad + (row0 + k) * 4 + 3];
#pragma unroll
                for (int x = 0; x < kCols; ++x)
                    if (D != 64 || lane < 16) {
                        const float4 y = *reinterpret_cast<const float4 *>(pc + (row0 + k) * C::kPad + 4 * (lane + 32 * x));
                        v[k][x].x += y.x * w;
                        v[k][x].y += y.y * w;
                        v[k][x].z += y.z * w;
                        v[k][x].w += y.w * w;
                    }
            }
        }
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) {
            const uintptr_t to = join_to[p0 * C::kRows + row0 + k];
#pragma unroll
            for (int x = 0; x < kCols; ++x) {
                if ((D == 64 && lane >= 16) || to == 0) continue;
                if (to & 1) reinterpret_cast<float4 *>(to - 1)[lane + 32 * x] = v[k][x];
                else store4(reinterpret_cast<T *>(to) + 4 * (lane + 32 * x), v[k][x]);
            }
        }
    }
    // the segment that goes on in the next CTAs, if it began in this one
    if (warp == C::kWarps - 1) {
        int4 d = make_int4(0, 0, 0, 0);
        const int lo = entry_of(prefix, n, c1 - 1);
        const int n_steps = e_steps[lo], su = (int)quotient(c1 - 1 - prefix[lo], n_steps + kOpen);
        const long long seg0 = prefix[lo] + (long long)su * (n_steps + kOpen) + kOpen, seg1 = seg0 + n_steps;
        if (seg0 >= c0 && seg0 < c1 && seg1 > c1) {
            int last = blockIdx.x + 1;
            while (first_step(last + 1) < seg1) ++last;
            d = make_int4(lo, su, last - (int)blockIdx.x + 1, 0);
        }
        if (lane == 0) ws.shared[blockIdx.x] = d;
    }
}

template <typename T, int D, int NT>
cudaError_t launch_tile(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    using C = Cfg<D, NT>;
    static_assert(C::smem(kMaxList) <= 227 * 1024 - 256, "shared memory of an SM");
    const int rows = a.q_len * (a.heads / c.kv_heads), row_tiles = (rows + C::kRows - 1) / C::kRows;
    const Split s = split_of(ws, num_sms);
    auto kern = attention_kernel<T, D, NT>;
    cudaError_t e = ensure_smem_attr(kern, C::smem(kMaxList));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)num_sms), dim3(C::kThreads), C::smem(a.n), st, c, a, s, row_tiles);
    if (e != cudaSuccess) return e;
    return launch_combine<T, D, C::kRows>(c, a, s, row_tiles, num_sms, st);
}

// Row tiles of 8 while a group's rows fit one, else as wide as the registers hold.
template <int D> constexpr int wide_tiles() { return D == 64 ? 4 : D == 128 ? 2 : 1; }

template <typename T, int D>
cudaError_t launch_dim(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    const int rows = a.q_len * (a.heads / c.kv_heads);
    if (rows <= 8 || wide_tiles<D>() == 1) return launch_tile<T, D, 1>(c, a, ws, num_sms, st);
    if (rows <= 16 || wide_tiles<D>() == 2) return launch_tile<T, D, (wide_tiles<D>() > 1 ? 2 : 1)>(c, a, ws, num_sms, st);
    return launch_tile<T, D, wide_tiles<D>()>(c, a, ws, num_sms, st);
}

template <typename T>
cudaError_t launch_typed(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    if (c.head_dim == 64) return launch_dim<T, 64>(c, a, ws, num_sms, st);
    if (c.head_dim == 128) return launch_dim<T, 128>(c, a, ws, num_sms, st);
    return launch_dim<T, 256>(c, a, ws, num_sms, st);
}

}  // namespace

// Two pieces per CTA of the widest row tile.
size_t kv8_attention_workspace(const Kv8 &c, int q_len, int heads, int num_sms) {
    int rows = 8 * (c.head_dim == 64 ? wide_tiles<64>() : c.head_dim == 128 ? wide_tiles<128>() : wide_tiles<256>());
    if (kv8_may_be_wide(c, q_len, heads)) rows = kWideRows;
    return align256((size_t)num_sms * sizeof(int4)) + align256((size_t)num_sms * 2 * rows * (c.head_dim + 4) * sizeof(float));
}

cudaError_t launch_kv8_attention(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    if (a.dtype == TP_MLP_F32) return launch_typed<float>(c, a, ws, num_sms, st);
    if (kv8_wide_rows(c, a.n, a.q_len, a.heads)) return launch_kv8_attention_wide(c, a, ws, num_sms, st);
    return launch_typed<__nv_bfloat16>(c, a, ws, num_sms, st);
}

}  // namespace tpmlp
