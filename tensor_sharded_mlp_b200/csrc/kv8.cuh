// kv8.cuh -- the paged 8-bit key/value cache as its kernels see it.
//
// One layer's codes and scales (value = e4m3(code) * scale of its page and
// head), the page map that all layers share, and the checks of what the host
// cannot see: every sequence number, length and page number is checked before
// it becomes an address; a bad one is flagged in the status word and left out.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"

namespace tpmlp {

struct Kv8 {
    uint8_t *k, *v;              // first layer, or the call's layer
    float *k_scale, *v_scale;
    int *table, *lengths, *refcount, *status;
    int layers, num_pages, kv_heads, page_size, page_shift, head_dim, max_seqs, max_pages;

    __host__ __device__ long long page_bytes() const { return (long long)kv_heads * page_size * head_dim; }
    __host__ __device__ long long capacity() const { return (long long)max_pages << page_shift; }
    __host__ __device__ int pages_of(int tokens) const { return (tokens + page_size - 1) >> page_shift; }
};

// Bits of the status word: the header's tp_mlp_kv8_flag.
__device__ __forceinline__ void kv8_flag(const Kv8 &c, int bits) { atomicOr(c.status, bits); }

// Entry i of a list of sequences; NULL lists sequence i.
__device__ __forceinline__ int kv8_seq(const int *seqs, int i) { return seqs ? seqs[i] : i; }

// Whether an entry at `i` repeats an earlier one of the list (one warp, all
// lanes; `list` NULL never repeats).
__device__ __forceinline__ bool kv8_repeats(const int *list, int i, int value) {
    if (!list) return false;
    bool hit = false;
    for (int j = (int)(threadIdx.x & 31); j < i; j += 32) hit |= list[j] == value;
    return __any_sync(0xffffffffu, hit);
}

// Four e4m3 codes <-> four floats.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ float4 e4m3_unpack4(uint32_t w) {
    const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
    const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    return make_float4(a.x, a.y, b.x, b.y);
}

// kv8_append.cu
cudaError_t launch_kv8_append(const Kv8 &c, const void *k, const void *v, long long row_stride, int tokens,
                              const int *seqs, const int *cu, int n, int dtype, int num_sms, cudaStream_t st);

// For the test of the bounded waits: from which tile of a CTA on a role of the many-rows kernel delivers nothing, and
// after how long waits give up (0: an ordinary call).
struct Kv8Stall {
    int loads = 0x7fffffff, weights = 0x7fffffff, products = 0x7fffffff;
    unsigned wait_us = 0;
};

// kv8_attention.cu.  maximum != nullptr: the partial form (o = weighted).
struct Kv8Query {
    const void *q;
    long long row_stride;
    const int *seqs, *positions;
    int n, q_len, heads;
    float scale;
    int dtype;
    void *o;
    float *maximum, *exp_sum;
    Kv8Stall stall;
};
// kv8_attention_wide.cu: the form for many query rows a KV head
bool kv8_wide_rows(const Kv8 &c, int n, int q_len, int heads);     // whether a call takes it
bool kv8_may_be_wide(const Kv8 &c, int q_len, int heads);          // whether a call of any number of entries does
cudaError_t launch_kv8_attention_wide(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st);
size_t kv8_attention_workspace(const Kv8 &c, int q_len, int heads, int num_sms);
cudaError_t launch_kv8_attention(const Kv8 &c, const Kv8Query &a, void *ws, int num_sms, cudaStream_t st);

// kv8_pages.cu
size_t kv8_pages_workspace(const Kv8 &c);
cudaError_t launch_kv8_reserve(const Kv8 &c, const int *seqs, const int *counts, int n, void *ws, int num_sms,
                               cudaStream_t st);
cudaError_t launch_kv8_fork(const Kv8 &c, const int *parents, const int *children, int n, cudaStream_t st);
cudaError_t launch_kv8_truncate(const Kv8 &c, const int *seqs, const int *new_lengths, int n, cudaStream_t st);
cudaError_t launch_kv8_copy_pages(const Kv8 &c, const int *pairs, int n, int num_sms, cudaStream_t st);
cudaError_t launch_kv8_compact(const Kv8 &c, int *new_index, void *ws, int num_sms, cudaStream_t st);

}  // namespace tpmlp
