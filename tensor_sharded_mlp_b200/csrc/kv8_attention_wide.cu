// kv8_attention_wide.cu -- attention over the paged 8-bit cache where many query rows share a KV head (a prompt's chunk on
// a long history, drafted tokens of wide groups), bf16.  The mathematics, the precision and what a call means are
// kv8_attention.cu's.
//
// With R query rows a cached byte takes 2 R flops: from some tens of rows on the warp-level products, not the loads, bound
// that kernel, and every tile of 8 to 32 rows reads the cache again.  Here a CTA takes 128 rows at once and both products
// are tcgen05.mma (M = 128 rows, fp16, accumulators in TMEM):
//
//   S = Q K^T   (N = tokens of a tile, K = head_dim)     O += W V   (N = head_dim, K = tokens, W from TMEM)
//
// * Eight warps load a tile's codes (into registers, two tiles ahead), turn them into fp16 once (exact) and store them
//   in the swizzled layout of the operands: keys K-major, values MN-major, so neither is transposed.
// * Four warps do the softmax, a thread a row: it reads its scores from TMEM and writes its weights (fp16; the value
//   scale and the reference R as in kv8_attention.cu) back to TMEM as the second product's A operand.  A tile is worked
//   through once against the reference so far; only if a score exceeds that by 2^15 the reference moves, the outputs in
//   TMEM are rescaled and the tile is done again.
// * One thread issues the products: the next tile's scores before this tile's outputs.
// A value that is NaN would reach every row through 0 * NaN: the loaders take it out and mark the tile, and each row's
// thread looks up the marked tile's codes for the tokens that it sees.
//
// The tiles of all segments are cut evenly over the CTAs as in kv8_attention.cu, and the same kernel joins pieces.  Every
// wait is bounded; one that gives up ends the CTA and sets TP_MLP_KV8_TIMEOUT.
//
// Measured (B200, bf16, 8 KV heads, 16 sequences of 4000 tokens; kv8_attention.cu's kernel -> this one, us):
//   rows            72            128            256           1024
//   head_dim 64   103 -> 76     132 -> 82      244 -> 144     914 -> 515
//   head_dim 128  144 -> 92     220 -> 98      429 -> 173    1652 -> 617
//   head_dim 256  294 -> 155    606 -> 166    1243 -> 300    4912 -> 1082
// What bounds it: a tile's way through the two places of keys and values (some 4300 cycles for 128 tokens of 128 columns:
// codes to operands 1700, scores 1000, softmax 3300, outputs 1000, each behind a barrier; two tiles are on it at a time).
// The tensor pipe is busy 19 % of the time.  Tried beside this form (64 rows of head_dim 128, 95 us): weights through shared
// memory 105; keys' and values' places freed separately 99-153, the more the longer the unrolled code; two threads a row
// 113; 16 loading warps 99-113.
#include "kv8_attention.cuh"

namespace tpmlp {
namespace {

constexpr int kWideOpen = 1;         // tiles that a segment's start and end cost beside its own, about

template <int D>
struct WideCfg {
    static constexpr int kTok = D == 256 ? 64 : 128;
    static constexpr int kLoaders = 256;
    static constexpr int kThreads = 128 + kLoaders + 32;
    static constexpr int kTile = kTok * D * 2;                           // fp16 keys (or values) of a tile
    static constexpr int kScores = 0, kOut = 2 * kTok, kWeights = kOut + D, kColumns = 512;   // TMEM
    static constexpr int kKeys = 0, kValues = 2 * kTile, kQuery = 4 * kTile;
    static constexpr int kScales = kQuery + kWideRows * D * 2, kPrefix = kScales + 2 * (kTok / 16) * 8;
    static constexpr size_t smem(int n) { return 1024 + (size_t)kPrefix + (size_t)(n + 1) * 8 + (size_t)n * 16; }
    static_assert(kWeights + kTok <= kColumns, "TMEM of an SM");
    static_assert(smem(kMaxList) <= 226 * 1024, "shared memory of an SM; the static part beside it is below 1 KB");
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
// Waits for the TMEM loads so far; v's values are only there after it.
__device__ __forceinline__ void tmem_ld_wait_for(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc], fp16 inputs, fp32 accumulator.
__device__ __forceinline__ void mma_f16_from_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t p, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(p), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Where a CTA is in its tiles: segment (entry, unit) of `steps` tiles from place seg0 on, of which it has t0 .. t1 - 1.
struct Walk {
    int e, unit, steps, t, t0, t1;
    long long seg0;
    bool live;
};

// kStalls: the form for the test of the waits, in which a role stops (Kv8Stall).
template <int D, bool kStalls>
__global__ void __launch_bounds__(WideCfg<D>::kThreads, 1)
    attention_wide_kernel(Kv8 c, Kv8Query a, Split ws, int row_tiles) {
    using C = WideCfg<D>;
    using T = __nv_bfloat16;
    constexpr int kTok = C::kTok;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t base = tc::smem_u32(smem);
    const int n = a.n, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.heads / c.kv_heads, rows = a.q_len * group, units_per_entry = c.kv_heads * row_tiles;
    long long *prefix = reinterpret_cast<long long *>(smem + C::kPrefix);
    int *e_seq = reinterpret_cast<int *>(prefix + n + 1), *e_len = e_seq + n, *e_first = e_len + n, *e_steps = e_first + n;
    float2 *scales = reinterpret_cast<float2 *>(smem + C::kScales);
    __shared__ long long scan_part[C::kThreads / 32];
    __shared__ __align__(8) unsigned long long bars[12];
    __shared__ uint32_t tmem_base;
    __shared__ int nan_tile[2];      // 1 + the number of the last tile in this place that held a NaN value
    __shared__ volatile int gave_up;
    const uint32_t bar0 = tc::smem_u32(bars);
    const uint32_t kv_full = bar0, kv_empty = bar0 + 16, s_full = bar0 + 32, p_full = bar0 + 48, o_full = bar0 + 64,
                   q_full = bar0 + 80, done = bar0 + 88;
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(kv_full + 8 * x, C::kLoaders / 32);
            tc::mbar_init(kv_empty + 8 * x, 1);
            tc::mbar_init(s_full + 8 * x, 1);
            tc::mbar_init(p_full + 8 * x, 4);
            tc::mbar_init(o_full + 8 * x, 1);
            nan_tile[x] = 0;
        }
        tc::mbar_init(q_full, 4);
        tc::mbar_init(done, 1);
        gave_up = 0;
        tc::fence_barrier_init();
    }
    pdl_allow_dependents();
    pdl_wait_previous();
    const Entries entries = {prefix, e_seq, e_len, e_first, e_steps};
    list_entries<C::kThreads>(c, a, units_per_entry, kTok, kWideOpen, entries, scan_part);
    __syncthreads();
    const long long total = prefix[n];
    const int ctas = (int)max(1LL, min((long long)gridDim.x, total));
    const long long share = quotient(total, ctas);
    const int extra = (int)(total - share * ctas);
    auto first_place = [&](int i) { return share * i + min(i, extra); };
    write_unseen<T, D, C::kThreads>(a, entries);
    if (blockIdx.x >= ctas || total == 0) {
        if (tid == 0) ws.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    const long long c0 = first_place(blockIdx.x), c1 = first_place(blockIdx.x + 1);
    if (warp == 12) tc::tmem_alloc(tc::smem_u32(&tmem_base), C::kColumns);
    if (warp == 0) {   // the segment that goes on in the next CTAs, if it begins in this one
        int4 d = make_int4(0, 0, 0, 0);
        const int lo = entry_of(prefix, n, c1 - 1);
        const int n_steps = e_steps[lo], su = (int)quotient(c1 - 1 - prefix[lo], n_steps + kWideOpen);
        const long long seg0 = prefix[lo] + (long long)su * (n_steps + kWideOpen) + kWideOpen, seg1 = seg0 + n_steps;
        if (seg0 >= c0 && seg0 < c1 && seg1 > c1) {
            int last = blockIdx.x + 1;
            while (first_place(last + 1) < seg1) ++last;
            d = make_int4(lo, su, last - (int)blockIdx.x + 1, 0);
        }
        if (lane == 0) ws.shared[blockIdx.x] = d;
    }
    Walk w;
    auto open_segment = [&]() {
        w.live = w.seg0 < c1;
        w.t = w.t0 = (int)max(0LL, c0 - w.seg0);
        w.t1 = (int)min((long long)w.steps, c1 - w.seg0);
    };
    auto next_segment = [&]() {
        w.seg0 += w.steps + kWideOpen;
        if (w.seg0 >= c1) {
            w.live = false;
            return;
        }
        if (++w.unit == units_per_entry) {
            w.unit = 0;
            do ++w.e;
            while (e_steps[w.e] == 0);
            w.steps = e_steps[w.e];
        }
        open_segment();
    };
    w.e = entry_of(prefix, n, c0);
    w.steps = e_steps[w.e];
    w.unit = (int)quotient(c0 - prefix[w.e], w.steps + kWideOpen);
    w.seg0 = prefix[w.e] + (long long)w.unit * (w.steps + kWideOpen) + kWideOpen;
    open_segment();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base;
    auto wait = [&](uint32_t bar, int phase) {
        return tc::mbar_wait(bar, phase & 1, &gave_up, kStalls ? a.stall.wait_us * 1000ull : tc::kWaitLimitNs);
    };

    if (warp >= 4 && warp < 12) {
        // --- loads: codes of two tiles in registers, the pages of the tile behind them ----------------------------
        constexpr int kChunks = kTok * D / 16 / C::kLoaders;
        const int lt = tid - 128;
        struct Raw {
            uint4 k[kChunks], v[kChunks];
            float2 sc;
        };
        Raw ra, rb;
        int page[kChunks], scale_page = -2;     // -2: no token there
        auto token_of = [&](int i) { return w.t * kTok + (i * C::kLoaders + lt) / (D / 16); };
        auto find_pages = [&]() {
            if (!w.live) return;
            const Entry en = {e_seq[w.e], e_len[w.e], e_first[w.e]};
            const int need = en.seen(a.q_len - 1);
            const int *row = c.table + (long long)en.seq * c.max_pages;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) page[i] = token_of(i) < need ? row[token_of(i) >> c.page_shift] : -2;
            const int s_tok = w.t * kTok + 16 * lt;
            scale_page = lt < kTok / 16 && s_tok < need ? row[s_tok >> c.page_shift] : -2;
        };
        auto load = [&](Raw &r) {
            const int head = w.unit / row_tiles;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const bool ok = (unsigned)page[i] < (unsigned)c.num_pages;
                bad |= !ok && page[i] != -2;
                r.k[i] = r.v[i] = make_uint4(0, 0, 0, 0);
                if (ok) {
                    const long long at = (((long long)page[i] * c.kv_heads + head) * c.page_size +
                                          (token_of(i) & (c.page_size - 1))) * D + (i * C::kLoaders + lt) % (D / 16) * 16;
                    r.k[i] = *reinterpret_cast<const uint4 *>(c.k + at);
                    r.v[i] = *reinterpret_cast<const uint4 *>(c.v + at);
                }
            }
            if (bad) kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
            r.sc = make_float2(0.f, scale_page == -2 ? 0.f : -1.f);   // negative: not a page of the pool
            if ((unsigned)scale_page < (unsigned)c.num_pages) {
                const long long at = (long long)scale_page * c.kv_heads + head;
                r.sc = make_float2(c.k_scale[at], c.v_scale[at]);
            }
            if (++w.t == w.t1) next_segment();
            find_pages();
        };
        auto store = [&](Raw &r, int i) {
            const int slot = i & 1;
            if (i >= 2 && !__all_sync(0xffffffffu, wait(kv_empty + 8 * slot, (i >> 1) - 1))) return false;
            if (kStalls && i >= a.stall.loads) return false;
            uint32_t any = 0;
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
                any |= nan_bytes(r.v[x].x) | nan_bytes(r.v[x].y) | nan_bytes(r.v[x].z) | nan_bytes(r.v[x].w);
            if (any) {
                nan_tile[slot] = i + 1;
#pragma unroll
                for (int x = 0; x < kChunks; ++x) {
                    r.v[x].x &= ~nan_bytes(r.v[x].x);
                    r.v[x].y &= ~nan_bytes(r.v[x].y);
                    r.v[x].z &= ~nan_bytes(r.v[x].z);
                    r.v[x].w &= ~nan_bytes(r.v[x].w);
                }
            }
            const uint32_t keys = base + C::kKeys + slot * C::kTile, values = base + C::kValues + slot * C::kTile;
#pragma unroll
            for (int x = 0; x < kChunks; ++x) {
                const int at = x * C::kLoaders + lt, tok = at / (D / 16), ch = at % (D / 16), block = ch >> 2;
                // columns 64 block + 16 (ch & 3) ..: 16-byte pieces j, j + 1 of the token's 128 bytes in the block
                const int j = (ch & 3) * 2, odd = block & 1;   // (odd blocks' threads store the second one first: banks)
                const uint32_t kp = keys + block * (kTok * 128) + tok * 128;
                const uint32_t vp = values + (tok >> 6) * (D / 64 * 8192) + block * 8192 + (tok & 63) * 128;
                const uint32_t p0 = ((j + odd) ^ (tok & 7)) << 4, p1 = ((j + 1 - odd) ^ (tok & 7)) << 4;
                uint32_t h[8];
                e4m3_to_f16(r.k[x].x, h[0], h[1]);
                e4m3_to_f16(r.k[x].y, h[2], h[3]);
                e4m3_to_f16(r.k[x].z, h[4], h[5]);
                e4m3_to_f16(r.k[x].w, h[6], h[7]);
                sts128(kp + p0, odd ? h[4] : h[0], odd ? h[5] : h[1], odd ? h[6] : h[2], odd ? h[7] : h[3]);
                sts128(kp + p1, odd ? h[0] : h[4], odd ? h[1] : h[5], odd ? h[2] : h[6], odd ? h[3] : h[7]);
                e4m3_to_f16(r.v[x].x, h[0], h[1]);
                e4m3_to_f16(r.v[x].y, h[2], h[3]);
                e4m3_to_f16(r.v[x].z, h[4], h[5]);
                e4m3_to_f16(r.v[x].w, h[6], h[7]);
                sts128(vp + p0, odd ? h[4] : h[0], odd ? h[5] : h[1], odd ? h[6] : h[2], odd ? h[7] : h[3]);
                sts128(vp + p1, odd ? h[0] : h[4], odd ? h[1] : h[5], odd ? h[2] : h[6], odd ? h[3] : h[7]);
            }
            if (lt < kTok / 16) scales[slot * (kTok / 16) + lt] = r.sc;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(kv_full + 8 * slot);   // (arrivals on one word go one by one)
            return true;
        };
        find_pages();
        bool ha = w.live, hb = false;
        if (ha) load(ra);
        if (ha && (hb = w.live)) load(rb);
        for (int i = 0; ha; i += 2) {
            if (!store(ra, i)) break;
            if ((ha = w.live)) load(ra);
            if (!hb || !store(rb, i + 1)) break;
            if ((hb = w.live)) load(rb);
        }
    } else if (warp < 4) {
        // --- softmax: thread = row -----------------------------------------------------------------------------
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16), out = lanes + C::kOut;
        int i = 0;
        bool ok = true;
        auto outputs_done = [&]() { return __all_sync(0xffffffffu, wait(o_full + 8 * ((i - 1) & 1), (i - 1) >> 1)); };
        while (ok && w.live) {
            const Entry en = {e_seq[w.e], e_len[w.e], e_first[w.e]};
            const int kv_head = w.unit / row_tiles, tile = w.unit - kv_head * row_tiles;
            const RowMap map = {w.e, kv_head, group, a.q_len, a.heads};
            const int r = tile * kWideRows + tid;
            const bool have = r < rows, busy = tile * kWideRows + warp * 32 < rows;
            float fac = 0.f, ref = -FLT_MAX, sum = 0.f, top = -INFINITY;
            int limit = 0x7fffffff;
            uint32_t nan_cols[D / 32];
#pragma unroll
            for (int x = 0; x < D / 32; ++x) nan_cols[x] = 0;
            if (busy) {
                const int rr = have ? r : 0, j = rr / group;
                const T *src = static_cast<const T *>(a.q) + ((long long)w.e * a.q_len + j) * a.row_stride +
                               (long long)(kv_head * group + rr - j * group) * D;
                float amax = 0.f;
#pragma unroll 4
                for (int x = 0; x < D; x += 8) {
                    RawQuery<T> raw;
                    float f[8];
                    raw.load(src + x);
                    raw.widen(f);
#pragma unroll
                    for (int y = 0; y < 8; ++y) amax = fmaxf(amax, fabsf(f[y]));
                }
                const QueryScale qs = query_scale(amax);
#pragma unroll 4
                for (int x = 0; x < D; x += 8) {
                    RawQuery<T> raw;
                    float f[8];
                    raw.load(src + x);
                    raw.widen(f);
                    uint32_t h[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        h[y] = have ? f16x2(f[2 * y] * qs.down, f[2 * y + 1] * qs.down) : 0u;
                    sts128(base + C::kQuery + (x >> 6) * (kWideRows * 128) + tid * 128 + ((((x >> 3) & 7) ^ (tid & 7)) << 4),
                           h[0], h[1], h[2], h[3]);
                }
                if (have) {
                    fac = a.scale * kLog2e * qs.up;
                    limit = en.seen(map.query(r));
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(q_full);
            for (; w.t < w.t1; ++w.t, ++i) {
                const int slot = i & 1;
                ok = __all_sync(0xffffffffu, wait(kv_full + 8 * slot, i >> 1) && wait(s_full + 8 * slot, i >> 1));
                if (!ok) break;
                if (busy) {
                    tc::tc_fence_after();
                    const uint32_t scores = lanes + C::kScores + slot * kTok;
                    const int tok0 = w.t * kTok;
                    const bool plain = __all_sync(0xffffffffu, limit >= tok0 + kTok);
                    const float2 *sc = scales + slot * (kTok / 16);
                    // 16 base-2 scores, in place; returns the binade above the value scale
                    auto base2 = [&](int gr, float (&s)[16], float2 ks) {
                        const float f = fac * ks.x;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            s[k] *= f;
                            if (!plain && tok0 + 16 * gr + k >= limit) s[k] = -INFINITY;
                            if (ks.y < 0.f) s[k] = -INFINITY;
                        }
                        return (float)max((int)((__float_as_uint(ks.y) & 0x7fffffffu) >> 23) - 126, kLeastLog);
                    };
                    // the reference that this tile's scores ask for
                    auto tile_ref = [&]() {
                        float m = -INFINITY;
#pragma unroll 2
                        for (int gr = 0; gr < kTok / 16; ++gr) {
                            float s[16];
                            tc::tmem_ld16(scores + 16 * gr, s);
                            tmem_ld_wait_for(s);
                            const float vlog = base2(gr, s, sc[gr]);
                            float x = s[0];
#pragma unroll
                            for (int k = 1; k < 16; ++k) x = fmaxf(x, s[k]);
                            m = fmaxf(m, x + (vlog - kLift));
                        }
                        return fmaxf(ref, m);
                    };
                    if (w.t == w.t0) ref = tile_ref();
                    float part, above;   // above: how far a score lies above the reference (a difference: exact however large)
                    auto weights = [&]() {
                        part = 0.f;
                        above = -INFINITY;
#pragma unroll 2
                        for (int gr = 0; gr < kTok / 16; ++gr) {
                            float s[16];
                            tc::tmem_ld16(scores + 16 * gr, s);
                            tmem_ld_wait_for(s);
                            const float2 ks = sc[gr];
                            const float vlog = base2(gr, s, ks), vs = ks.y < 0.f ? 0.f : ks.y;
                            float x = s[0], l0 = 0.f, l1 = 0.f;
                            uint32_t h[8];
#pragma unroll
                            for (int k = 1; k < 16; ++k) x = fmaxf(x, s[k]);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float p0 = exp2_fast(s[2 * k] - ref), p1 = exp2_fast(s[2 * k + 1] - ref);
                                l0 += p0;
                                l1 += p1;
                                h[k] = f16x2(p0 * vs, p1 * vs);
                            }
                            part += l0 + l1;
                            top = fmaxf(top, x);
                            above = fmaxf(above, (x - ref) + vlog);
                            tmem_st8(lanes + C::kWeights + slot * (kTok / 2) + 8 * gr, h);
                        }
                    };
                    weights();
                    if (__any_sync(0xffffffffu, above > kSlack)) {
                        const float up = tile_ref(), turn = up == ref ? 1.f : exp2_fast(ref - up);
                        sum = turn_sum(sum, turn, ref - up);
                        ref = up;
                        if (w.t > w.t0) {
                            if (!(ok = outputs_done())) break;
                            tc::tc_fence_after();
#pragma unroll 1
                            for (int x = 0; x < D / 16; ++x) {
                                float v[16];
                                tc::tmem_ld16(out + 16 * x, v);
                                tmem_ld_wait_for(v);
#pragma unroll
                                for (int k = 0; k < 16; ++k) v[k] *= turn;
                                tmem_st16(out + 16 * x, v);
                            }
                        }
                        weights();
                    }
                    tmem_st_wait();
                    sum += part;
                    if (nan_tile[slot] == i + 1 && have) {
                        const int end = min(limit, tok0 + kTok);
                        const int *row = c.table + (long long)en.seq * c.max_pages;
                        for (int tok = tok0; tok < end; ++tok) {
                            const int p = row[tok >> c.page_shift];
                            if ((unsigned)p >= (unsigned)c.num_pages) continue;
                            const uint32_t *v = reinterpret_cast<const uint32_t *>(
                                c.v + (((long long)p * c.kv_heads + kv_head) * c.page_size + (tok & (c.page_size - 1))) * D);
#pragma unroll
                            for (int x = 0; x < D / 32; ++x)
                                for (int y = 0; y < 8; ++y) {
                                    const uint32_t nb = nan_bytes(v[8 * x + y]) & 0x08040201u;
                                    nan_cols[x] |= ((nb | nb >> 8 | nb >> 16 | nb >> 24) & 15u) << (4 * y);
                                }
                        }
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0 && !(kStalls && i >= a.stall.weights)) tc::mbar_arrive(p_full + 8 * slot);
            }
            if (!ok || !(ok = outputs_done())) break;
            tc::tc_fence_after();
            if (busy) {
                const bool whole = w.t0 == 0 && w.t1 == w.steps;
                float factor = 1.f;
                float *piece = ws.pieces + ((size_t)blockIdx.x * 2 + (w.seg0 < c0 ? 0 : 1)) * (kWideRows * (D + 4));
                T *dst = nullptr;
                if (whole && have) {
                    const long long orow = map.out_row(r);
                    const RowResult res = row_result(ref, sum, top, a.maximum != nullptr);
                    factor = res.factor;
                    dst = static_cast<T *>(a.o) + orow * D;
                    if (a.maximum) {
                        a.maximum[orow] = res.maximum;
                        a.exp_sum[orow] = res.exp_sum;
                    }
                } else if (!whole) {
                    *reinterpret_cast<float4 *>(piece + kWideRows * D + tid * 4) = make_float4(ref, sum, top, 0.f);
                }
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    float v[16];
                    tc::tmem_ld16(out + 16 * x, v);
                    tmem_ld_wait_for(v);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        v[k] = nan_cols[x >> 1] >> ((x & 1) * 16 + k) & 1 ? NAN : v[k] * factor;
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 v4 = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                        if (!whole) *reinterpret_cast<float4 *>(piece + tid * D + 16 * x + k) = v4;
                        else if (have) store4(dst + 16 * x + k, v4);
                    }
                }
            }
            next_segment();
        }
        if (!ok) tmem_st_wait();   // (weights on their way when a wait gave up)
    } else if (lane == 0) {
        // --- products -------------------------------------------------------------------------------------------
        constexpr uint32_t kF16 = (1u << 4) | ((uint32_t)(kWideRows >> 4) << 24);      // f16 x f16 -> f32, M = 128
        constexpr uint32_t kScoreDesc = kF16 | ((uint32_t)(kTok >> 3) << 17);
        constexpr uint32_t kOutDesc = kF16 | ((uint32_t)(D >> 3) << 17) | tc::kIdescBMajorMN;
        int i = 0, seg = 0;
        bool ok = true, open = false, open_first = false;   // open: tile i - 1's output product is still to come
        auto outputs = [&]() {
            const int j = i - 1, slot = j & 1;
            if (!(ok = wait(p_full + 8 * slot, j >> 1))) return;
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kTok / 16; ++k)
                mma_f16_from_tmem(tmem + C::kOut, tmem + C::kWeights + slot * (kTok / 2) + 8 * k,
                             tc::smem_desc_mnmajor_sw128(base + C::kValues + slot * C::kTile + (k >> 2) * (D / 64 * 8192) +
                                                         (k & 3) * 2048),
                             kOutDesc, !(open_first && k == 0));
            tc::mma_commit(kv_empty + 8 * slot);
            tc::mma_commit(o_full + 8 * slot);
            open = false;
        };
        while (ok && w.live) {
            const bool first = w.t == w.t0;
            const int slot = i & 1;
            if (kStalls && i >= a.stall.products) break;
            if (first) {       // (the row threads turn to the next segment once this one's outputs are there)
                if (open) outputs();
                if (!ok || !(ok = wait(q_full, seg))) break;
                ++seg;
            }
            if (!(ok = wait(kv_full + 8 * slot, i >> 1))) break;
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                tc::mma_bf16(tmem + C::kScores + slot * kTok,
                             tc::smem_desc_kmajor_sw128(base + C::kQuery + (k >> 2) * (kWideRows * 128) + (k & 3) * 32),
                             tc::smem_desc_kmajor_sw128(base + C::kKeys + slot * C::kTile + (k >> 2) * (kTok * 128) +
                                                        (k & 3) * 32),
                             kScoreDesc, k > 0);
            tc::mma_commit(s_full + 8 * slot);
            if (open) outputs();
            ++i;
            open = true;
            open_first = first;
            if (++w.t == w.t1) next_segment();
        }
        if (ok && open) outputs();
        // products in flight end before the memory is given back, whichever role's wait gave up
        volatile int none = 0;
        tc::mma_commit(done);
        tc::mbar_wait(done, 0, &none);
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 12) {
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, C::kColumns);
    }
    if (tid == 0 && gave_up) kv8_flag(c, TP_MLP_KV8_TIMEOUT);
}

template <int D, bool kStalls>
cudaError_t launch_wide(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    using C = WideCfg<D>;
    const int row_tiles = (a.q_len * (a.heads / c.kv_heads) + kWideRows - 1) / kWideRows;
    const Split s = split_of(ws, num_sms);
    auto kern = attention_wide_kernel<D, kStalls>;
    cudaError_t e = ensure_smem_attr(kern, C::smem(kMaxList));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)num_sms), dim3(C::kThreads), C::smem(a.n), st, c, a, s, row_tiles);
    if (e != cudaSuccess) return e;
    return launch_combine<__nv_bfloat16, D, kWideRows>(c, a, s, row_tiles, num_sms, st);
}

template <int D>
cudaError_t launch_either(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    return a.stall.wait_us ? launch_wide<D, true>(c, a, ws, num_sms, st) : launch_wide<D, false>(c, a, ws, num_sms, st);
}

}  // namespace

// From so many rows on the products bound the other kernel, whose row tiles (32, 16 or 8 rows for head_dim 64, 128, 256)
// each read the history again; but it cuts a short history finer, and a segment's queries, outputs and join cost less there.
// Both in us, 8 KV heads, other kernel / this one:
//                                 16 x 4000 tokens  32 x 1000    64 x 200     8 x 100-300  1 x 4000
//   head_dim 256, 24 rows           107 / 147         61 / 105     37 / 100    15 / 25      19 / 35
//                 33                195 / 148         93 / 108     51 / 103    16 / 26      23 / 38
//                 64                288 / 150        144 / 110     77 / 107    19 / 28      28 / 38
//   head_dim 128, 48 rows            92 / 90          55 / 64      36 / 58     15 / 18      17 / 23
//                 64                119 / 91          69 / 65      44 / 58     16 / 18      18 / 24
//   head_dim 64,  33-64 rows         76 / 73-74       49-50 / 50   38 / 43     18 / 15      22 / 21
// The lengths are the device's to know.  The host has a bound of the tokens that a call can see, and up to 64 rows this
// kernel is taken only where those of all KV heads may be 2^18 (16 x 4000 x 8 are 2^19, 32 x 1000 x 8 are 2^18).  Above 64
// rows it always is, for the table at the head of this file; what that costs short histories (head_dim 64, 128, 256): one
// sequence of 4000 tokens, 72 rows 22 -> 22, 20 -> 25, 38 -> 40, 128 rows 24 -> 25, 25 -> 28, 45 -> 48; 8 of 100 to 300 tokens,
// 128 rows 21 -> 18, 20 -> 22, 29 -> 36.
namespace {
constexpr int kAlwaysWide = 64;
int wide_rows_from(int head_dim) { return head_dim == 256 ? 32 : head_dim == 128 ? 48 : kAlwaysWide; }
}  // namespace

bool kv8_may_be_wide(const Kv8 &c, int q_len, int heads) {
    return q_len * (heads / c.kv_heads) > wide_rows_from(c.head_dim);
}

bool kv8_wide_rows(const Kv8 &c, int n, int q_len, int heads) {
    const long long pages = (long long)n * c.max_pages < c.num_pages ? (long long)n * c.max_pages : c.num_pages;
    return kv8_may_be_wide(c, q_len, heads) &&
           (q_len * (heads / c.kv_heads) > kAlwaysWide || pages * c.page_size * c.kv_heads >= 1LL << 18);
}

cudaError_t launch_kv8_attention_wide(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st) {
    if (c.head_dim == 64) return launch_either<64>(c, a, ws, num_sms, st);
    if (c.head_dim == 128) return launch_either<128>(c, a, ws, num_sms, st);
    return launch_either<256>(c, a, ws, num_sms, st);
}

}  // namespace tpmlp
