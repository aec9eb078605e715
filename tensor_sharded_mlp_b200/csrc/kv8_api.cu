// kv8_api.cu -- the C entry points of the paged 8-bit key/value cache: host-side
// argument checks (sizes, enums, alignment, every buffer inside its device
// allocation) and the launches.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

using namespace tpmlp;

namespace {

int from_cuda(cudaError_t e) { return e == cudaSuccess ? TP_MLP_OK : TP_MLP_ERR_CUDA; }

bool pow2_between(int v, int lo, int hi) { return v >= lo && v <= hi && (v & (v - 1)) == 0; }

// Sizes alone (no pointer is looked at), and the kernels' view of the first layer.
int view_of(const tp_mlp_kv8_cache *cache, Kv8 *c) {
    if (!cache) return TP_MLP_ERR_INVALID_ARG;
    if (cache->layers < 1 || cache->num_pages < 1 || cache->max_seqs < 1 || cache->max_pages < 1)
        return TP_MLP_ERR_SHAPE;
    if (cache->kv_heads < 1 || cache->kv_heads > 256 || !pow2_between(cache->page_size, 16, 256) ||
        !pow2_between(cache->head_dim, 64, 256))
        return TP_MLP_ERR_SHAPE;
    if (cache->num_pages > (1 << 30)) return TP_MLP_ERR_SHAPE;
    // token counts are 32-bit; the table's entries are indexed in 64 bits
    if ((long long)cache->max_pages * cache->page_size > 0x7fffff00LL) return TP_MLP_ERR_SHAPE;
    c->k = static_cast<uint8_t *>(cache->k);
    c->v = static_cast<uint8_t *>(cache->v);
    c->k_scale = cache->k_scale;
    c->v_scale = cache->v_scale;
    c->table = cache->table;
    c->lengths = cache->lengths;
    c->refcount = cache->refcount;
    c->status = cache->status;
    c->layers = cache->layers;
    c->num_pages = cache->num_pages;
    c->kv_heads = cache->kv_heads;
    c->page_size = cache->page_size;
    c->page_shift = 4;
    while ((1 << c->page_shift) < c->page_size) ++c->page_shift;
    c->head_dim = cache->head_dim;
    c->max_seqs = cache->max_seqs;
    c->max_pages = cache->max_pages;
    return TP_MLP_OK;
}

int check_map(const Kv8 &c) {
    int s;
    if ((s = check_dev(c.table, (size_t)c.max_seqs * c.max_pages * sizeof(int)))) return s;
    if ((s = check_dev(c.lengths, (size_t)c.max_seqs * sizeof(int)))) return s;
    if ((s = check_dev(c.refcount, (size_t)c.num_pages * sizeof(int)))) return s;
    return check_dev(c.status, sizeof(int));
}

int check_pool(const Kv8 &c) {
    const size_t pages = (size_t)c.layers * c.num_pages;
    int s;
    if ((s = check_dev(c.k, pages * c.page_bytes()))) return s;
    if ((s = check_dev(c.v, pages * c.page_bytes()))) return s;
    if ((s = check_dev(c.k_scale, pages * c.kv_heads * sizeof(float)))) return s;
    return check_dev(c.v_scale, pages * c.kv_heads * sizeof(float));
}

void to_layer(Kv8 *c, int layer) {
    const long long pages = (long long)layer * c->num_pages;
    c->k += pages * c->page_bytes();
    c->v += pages * c->page_bytes();
    c->k_scale += pages * c->kv_heads;
    c->v_scale += pages * c->kv_heads;
}

int check_list(const int *list, int n, bool optional = false) {
    if (!list) return optional ? TP_MLP_OK : TP_MLP_ERR_INVALID_ARG;
    return check_dev(list, (size_t)n * sizeof(int));
}

int sm_count(int *sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || *sms < 1)
        return TP_MLP_ERR_CUDA;
    return TP_MLP_OK;
}

size_t elem_bytes(int dtype) { return dtype == TP_MLP_F32 ? 4 : 2; }

// `rows` rows of `width` elements, one every `stride` elements, each starting
// on a 16-byte boundary.
int check_rows(const void *p, long long rows, long long width, long long stride, int dtype) {
    const size_t e = elem_bytes(dtype);
    return check_dev(p, (size_t)((rows - 1) * stride + width) * e);
}

int attention_sizes(const Kv8 &c, int n, int q_len, int heads) {
    if (n < 0 || n > TP_MLP_KV8_MAX_LIST || q_len < 1 || q_len > TP_MLP_KV8_MAX_QUERIES || heads < 1) return TP_MLP_ERR_SHAPE;
    if (heads % c.kv_heads != 0 || heads / c.kv_heads > 128) return TP_MLP_ERR_SHAPE;
    return TP_MLP_OK;
}

int attention(const tp_mlp_kv8_cache *cache, int layer, const Kv8Query &a, bool partial, void *ws, size_t ws_bytes,
              tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if ((s = attention_sizes(c, a.n, a.q_len, a.heads))) return s;
    if (layer < 0 || layer >= c.layers) return TP_MLP_ERR_SHAPE;
    if (a.dtype != TP_MLP_F32 && a.dtype != TP_MLP_BF16) return TP_MLP_ERR_INVALID_ARG;
    if (!std::isfinite(a.scale)) return TP_MLP_ERR_INVALID_ARG;
    const size_t e = elem_bytes(a.dtype);
    const long long width = (long long)a.heads * c.head_dim, rows = (long long)a.n * a.q_len;
    if (a.row_stride < width || a.row_stride > (1LL << 40)) return TP_MLP_ERR_SHAPE;
    if (a.row_stride * (long long)e % 16 != 0) return TP_MLP_ERR_ALIGNMENT;
    if (a.n == 0) return TP_MLP_OK;   // empty tensors may carry null pointers
    if (!a.q || !a.o || (partial && (!a.maximum || !a.exp_sum))) return TP_MLP_ERR_INVALID_ARG;
    if (!a.seqs && a.n > c.max_seqs) return TP_MLP_ERR_SHAPE;
    if ((s = check_map(c)) || (s = check_pool(c))) return s;
    if ((s = check_rows(a.q, rows, width, a.row_stride, a.dtype))) return s;
    if ((s = check_dev(a.o, (size_t)(rows * width) * e))) return s;
    if (partial) {
        if ((s = check_dev(a.maximum, (size_t)rows * a.heads * sizeof(float)))) return s;
        if ((s = check_dev(a.exp_sum, (size_t)rows * a.heads * sizeof(float)))) return s;
    }
    if ((s = check_list(a.seqs, a.n, true)) || (s = check_list(a.positions, a.n, true))) return s;
    int sms = 0;
    if ((s = sm_count(&sms))) return s;
    const size_t need = kv8_attention_workspace(c, a.q_len, a.heads, sms);
    if (!ws || ws_bytes < need) return TP_MLP_ERR_WORKSPACE;
    if ((s = check_dev(ws, need))) return s;
    to_layer(&c, layer);
    return from_cuda(launch_kv8_attention(c, a, ws, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int tp_mlp_kv8_get_status(const tp_mlp_kv8_cache *cache, int *flags) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if (!flags) return TP_MLP_ERR_INVALID_ARG;
    if ((s = check_dev(c.status, sizeof(int)))) return s;
    int bits = 0;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&bits, c.status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(c.status, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
        return TP_MLP_ERR_CUDA;
    *flags = bits;
    return TP_MLP_OK;
}

size_t tp_mlp_kv8_pages_workspace_bytes(const tp_mlp_kv8_cache *cache) {
    Kv8 c;
    return view_of(cache, &c) ? 0 : kv8_pages_workspace(c);
}

int tp_mlp_kv8_reserve(const tp_mlp_kv8_cache *cache, const int *seqs, const int *counts, int n, void *workspace,
                       size_t workspace_bytes, tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if (n < 0 || n > TP_MLP_KV8_MAX_LIST || (!seqs && n > c.max_seqs)) return TP_MLP_ERR_SHAPE;
    if (n == 0) return TP_MLP_OK;
    if (!counts) return TP_MLP_ERR_INVALID_ARG;
    if ((s = check_map(c)) || (s = check_pool(c))) return s;
    if ((s = check_list(seqs, n, true)) || (s = check_list(counts, n))) return s;
    const size_t need = kv8_pages_workspace(c);
    if (!workspace || workspace_bytes < need) return TP_MLP_ERR_WORKSPACE;
    if ((s = check_dev(workspace, need))) return s;
    int sms = 0;
    if ((s = sm_count(&sms))) return s;
    return from_cuda(launch_kv8_reserve(c, seqs, counts, n, workspace, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int tp_mlp_kv8_fork(const tp_mlp_kv8_cache *cache, const int *parents, const int *children, int n,
                    tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if (n < 0 || n > TP_MLP_KV8_MAX_LIST) return TP_MLP_ERR_SHAPE;
    if (n == 0) return TP_MLP_OK;
    if ((s = check_map(c)) || (s = check_list(parents, n)) || (s = check_list(children, n))) return s;
    return from_cuda(launch_kv8_fork(c, parents, children, n, reinterpret_cast<cudaStream_t>(stream)));
}

int tp_mlp_kv8_truncate(const tp_mlp_kv8_cache *cache, const int *seqs, const int *new_lengths, int n,
                        tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if (n < 0 || n > TP_MLP_KV8_MAX_LIST) return TP_MLP_ERR_SHAPE;
    if (n == 0) return TP_MLP_OK;
    if ((s = check_map(c)) || (s = check_list(seqs, n)) || (s = check_list(new_lengths, n, true))) return s;
    return from_cuda(launch_kv8_truncate(c, seqs, new_lengths, n, reinterpret_cast<cudaStream_t>(stream)));
}

int tp_mlp_kv8_copy_pages(const tp_mlp_kv8_cache *cache, const int *pairs, int n, tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if (n < 0 || n > TP_MLP_KV8_MAX_LIST) return TP_MLP_ERR_SHAPE;
    if (n == 0) return TP_MLP_OK;
    if ((s = check_map(c)) || (s = check_pool(c)) || (s = check_list(pairs, 2 * n))) return s;
    int sms = 0;
    if ((s = sm_count(&sms))) return s;
    return from_cuda(launch_kv8_copy_pages(c, pairs, n, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int tp_mlp_kv8_compact(const tp_mlp_kv8_cache *cache, int *new_index, void *workspace, size_t workspace_bytes,
                       tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if ((s = check_map(c)) || (s = check_pool(c))) return s;
    if (new_index && (s = check_dev(new_index, (size_t)c.num_pages * sizeof(int)))) return s;
    const size_t need = kv8_pages_workspace(c);
    if (!workspace || workspace_bytes < need) return TP_MLP_ERR_WORKSPACE;
    if ((s = check_dev(workspace, need))) return s;
    int sms = 0;
    if ((s = sm_count(&sms))) return s;
    return from_cuda(launch_kv8_compact(c, new_index, workspace, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int tp_mlp_kv8_append(const tp_mlp_kv8_cache *cache, int layer, const void *k, const void *v, long long row_stride,
                      int tokens, const int *seqs, const int *cu_tokens, int n, int dtype, tp_mlp_stream_t stream) {
    Kv8 c;
    int s = view_of(cache, &c);
    if (s) return s;
    if (layer < 0 || layer >= c.layers) return TP_MLP_ERR_SHAPE;
    if (n < 0 || n > TP_MLP_KV8_MAX_LIST || tokens < 0 || tokens > (1 << 22) || (!seqs && n > c.max_seqs))
        return TP_MLP_ERR_SHAPE;
    if (dtype != TP_MLP_F32 && dtype != TP_MLP_BF16) return TP_MLP_ERR_INVALID_ARG;
    const long long width = (long long)c.kv_heads * c.head_dim;
    if (row_stride < width || row_stride > (1LL << 40)) return TP_MLP_ERR_SHAPE;
    if (row_stride * (long long)elem_bytes(dtype) % 16 != 0) return TP_MLP_ERR_ALIGNMENT;
    if (n == 0 || tokens == 0) return TP_MLP_OK;
    if (!cu_tokens && tokens % n != 0) return TP_MLP_ERR_SHAPE;
    if ((s = check_map(c)) || (s = check_pool(c))) return s;
    if ((s = check_rows(k, tokens, width, row_stride, dtype)) || (s = check_rows(v, tokens, width, row_stride, dtype)))
        return s;
    if ((s = check_list(seqs, n, true)) || (s = check_list(cu_tokens, n + 1, true))) return s;
    int sms = 0;
    if ((s = sm_count(&sms))) return s;
    to_layer(&c, layer);
    return from_cuda(launch_kv8_append(c, k, v, row_stride, tokens, seqs, cu_tokens, n, dtype, sms,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

size_t tp_mlp_kv8_attention_workspace_bytes(const tp_mlp_kv8_cache *cache, int n, int q_len, int heads) {
    Kv8 c;
    if (view_of(cache, &c) || attention_sizes(c, n, q_len, heads)) return 0;
    int sms = 0;
    if (sm_count(&sms)) {
        cudaGetLastError();
        sms = 148;   // B200
    }
    return kv8_attention_workspace(c, q_len, heads, sms);
}

int tp_mlp_kv8_attention(const tp_mlp_kv8_cache *cache, int layer, const void *q, long long row_stride,
                         const int *seqs, const int *positions, int n, int q_len, int heads, float scale, int dtype,
                         void *out, void *workspace, size_t workspace_bytes, tp_mlp_stream_t stream) {
    const Kv8Query a = {q, row_stride, seqs, positions, n, q_len, heads, scale, dtype, out, nullptr, nullptr, {}};
    return attention(cache, layer, a, false, workspace, workspace_bytes, stream);
}

int tp_mlp_kv8_attention_partials(const tp_mlp_kv8_cache *cache, int layer, const void *q, long long row_stride,
                                  const int *seqs, const int *positions, int n, int q_len, int heads, float scale,
                                  int dtype, float *maximum, float *exp_sum, void *weighted, void *workspace,
                                  size_t workspace_bytes, tp_mlp_stream_t stream) {
    const Kv8Query a = {q, row_stride, seqs, positions, n, q_len, heads, scale, dtype, weighted, maximum, exp_sum, {}};
    return attention(cache, layer, a, true, workspace, workspace_bytes, stream);
}

int tp_mlp_kv8_selftest_stalled_attention(const tp_mlp_kv8_cache *cache, int layer, const void *q, int n, int q_len,
                                          int heads, void *out, void *workspace, size_t workspace_bytes, int role,
                                          int tile, unsigned wait_us, tp_mlp_stream_t stream) {
    Kv8 c;
    const int s = view_of(cache, &c);
    if (s) return s;
    if (attention_sizes(c, n, q_len, heads)) return TP_MLP_ERR_SHAPE;
    if (role < 0 || role > 2 || tile < 0 || wait_us == 0 || wait_us > 100000) return TP_MLP_ERR_INVALID_ARG;
    if (!kv8_wide_rows(c, n, q_len, heads)) return TP_MLP_ERR_UNSUPPORTED;
    Kv8Query a = {q, (long long)heads * c.head_dim, nullptr, nullptr, n, q_len, heads, 1.f, TP_MLP_BF16, out, nullptr,
                  nullptr, {}};
    (role == 0 ? a.stall.loads : role == 1 ? a.stall.weights : a.stall.products) = tile;
    a.stall.wait_us = wait_us;
    return attention(cache, layer, a, false, workspace, workspace_bytes, stream);
}

}  // extern "C"
