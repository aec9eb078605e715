// kv8_attention.cu -- attention over the paged 8-bit key/value cache.
//
// For query row r (query j of an entry, head h) and the tokens t that it sees:
//   s_t = scale * k_scale * (q . k_t),  m = max s_t,  p_t = exp(s_t - m),
//   out = sum p_t v_scale v_t / sum p_t.
// One CTA per query row walks the sequence 128 tokens at a time with a running
// maximum and sum: a thread scores one token, then owns output columns.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace tpmlp {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxDim = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) attention_rows_kernel(Kv8 c, Kv8Query a) {
    __shared__ float qs[kMaxDim], ps[kThreads], red[kThreads];
    __shared__ int pages[kThreads / 16];
    pdl_allow_dependents();
    pdl_wait_previous();
    const int tid = threadIdx.x, D = c.head_dim;
    const int h = blockIdx.x % a.heads, j = blockIdx.x / a.heads % a.q_len, i = blockIdx.x / a.heads / a.q_len;
    const int seq = kv8_seq(a.seqs, i);
    if (seq == -1) return;
    if ((unsigned)seq >= (unsigned)c.max_seqs) {
        if (tid == 0) kv8_flag(c, TP_MLP_KV8_BAD_SEQUENCE);
        return;
    }
    const int len = c.lengths[seq];
    if (len < 0 || len > c.capacity()) {
        if (tid == 0) kv8_flag(c, TP_MLP_KV8_BAD_LENGTH);
        return;
    }
    const long long pos = (a.positions ? (long long)a.positions[i] : (long long)len - a.q_len) + j;
    const int end = (int)max(0LL, min((long long)len, pos + 1));
    const int kvh = h / (a.heads / c.kv_heads);
    const T *q = static_cast<const T *>(a.q) + ((long long)i * a.q_len + j) * a.row_stride + (long long)h * D;
    for (int d = tid; d < D; d += kThreads) qs[d] = to_f32(q[d]) * a.scale;
    float m = -INFINITY, l = 0.f, o[kMaxDim / kThreads] = {0.f, 0.f};
    for (int t0 = 0; t0 < end; t0 += kThreads) {
        __syncthreads();
        if (tid < kThreads / 16) {
            const int t = t0 + tid * 16;
            int p = -1;
            if (t < end) {
                p = c.table[(long long)seq * c.max_pages + (t >> c.page_shift)];
                if ((unsigned)p >= (unsigned)c.num_pages) {
                    kv8_flag(c, TP_MLP_KV8_BAD_PAGE);
                    p = -1;
                }
            }
            pages[tid] = p;
        }
        __syncthreads();
        const int t = t0 + tid, p = pages[tid >> 4];
        float s = -INFINITY;
        if (t < end && p >= 0) {
            const long long head = (long long)p * c.kv_heads + kvh;
            const uint32_t *k = reinterpret_cast<const uint32_t *>(c.k + (head * c.page_size + (t & (c.page_size - 1))) * D);
            float acc = 0.f;
            for (int d = 0; d < D / 4; ++d) {
                const float4 f = e4m3_unpack4(k[d]);
                acc += f.x * qs[4 * d] + f.y * qs[4 * d + 1] + f.z * qs[4 * d + 2] + f.w * qs[4 * d + 3];
            }
            s = acc * c.k_scale[head];
        }
        red[tid] = s;
        __syncthreads();
        for (int w = kThreads / 2; w > 0; w >>= 1) {
            if (tid < w) red[tid] = fmaxf(red[tid], red[tid + w]);
            __syncthreads();
        }
        const float top = fmaxf(m, red[0]);
        const float base = top == -INFINITY ? 0.f : top;
        const float turn = expf(m - base);
        m = top;
        ps[tid] = expf(s - base);
        __syncthreads();
        l *= turn;
        for (int x = 0; x < kThreads; ++x) l += ps[x];
        for (int u = 0; u < kMaxDim / kThreads; ++u) {
            const int d = tid + u * kThreads;
            if (d >= D) break;
            float acc = o[u] * turn;
            for (int x = 0; x < kThreads && t0 + x < end; ++x) {
                const int pg = pages[x >> 4];
                if (pg < 0) continue;
                const long long head = (long long)pg * c.kv_heads + kvh;
                const uint8_t code = c.v[(head * c.page_size + ((t0 + x) & (c.page_size - 1))) * D + d];
                const float v = __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
                acc += ps[x] * c.v_scale[head] * v;
            }
            o[u] = acc;
        }
    }
    const long long row = ((long long)i * a.q_len + j) * a.heads + h;
    const float inv = a.maximum ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN;
    for (int u = 0; u < kMaxDim / kThreads; ++u) {
        const int d = tid + u * kThreads;
        if (d < D) static_cast<T *>(a.o)[row * D + d] = from_f32<T>(o[u] * inv);
    }
    if (a.maximum && tid == 0) {
        a.maximum[row] = isnan(l) && m != INFINITY ? l : m;   // (fmaxf passes over a NaN score)
        a.exp_sum[row] = l;
    }
}

}  // namespace

size_t kv8_attention_workspace(const Kv8 &, int, int, int, int) { return 256; }

cudaError_t launch_kv8_attention(const Kv8 &c, const Kv8Query &a, void *, int, cudaStream_t st) {
    const dim3 grid((unsigned)((long long)a.n * a.q_len * a.heads));
    if (a.dtype == TP_MLP_F32) return launch_pdl(attention_rows_kernel<float>, grid, dim3(kThreads), 0, st, c, a);
    return launch_pdl(attention_rows_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, c, a);
}

}  // namespace tpmlp
