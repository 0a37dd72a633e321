// The paged cache as the kernels see it: sequences of tokens over pools of
// pages (include/ecco.h, ecco_paged).  Everything read from the device-side
// arrays is bounded here, so that no index leaves its buffer whatever they hold.
#pragma once

#include "ecco_internal.cuh"

namespace ecco {

// Tokens that a page_table row can hold.
__host__ __device__ __forceinline__ int64_t paged_capacity(const ecco_paged& p)
{
    return (int64_t)p.max_pages * p.page_size;
}

// Keys of sequence b, at most `bound`.
__device__ __forceinline__ int paged_kv_len(const ecco_paged& p, int b, int bound)
{
    const int cap = (int)min(paged_capacity(p), (int64_t)bound);
    return min(max(p.kv_lens[b], 0), cap);
}

// Block index (within a pool) of head h of token t of sequence b, or -1 where
// the table names no page.  0 <= t < paged_capacity.
__device__ __forceinline__ int64_t paged_block(const ecco_paged& p, int b, int h, int t)
{
    const int pi = t / p.page_size;
    const int page = __ldg(p.page_table + (int64_t)b * p.table_stride + pi);
    if ((uint32_t)page >= (uint64_t)p.n_pages) return -1;
    return ((int64_t)page * p.kv_heads + h) * p.page_size + (t - pi * p.page_size);
}

// ------------------------------------------------------------ launchers
cudaError_t launch_rope_table(const double* inv_freq, int n_freq, double magnitude, int64_t n_positions, float* table,
                              cudaStream_t s);

struct RopeArgs {
    const void* x;
    void* y;
    int64_t x_token, x_head, y_token, y_head;  // strides in elements
    int64_t tokens, n_positions;
    const float* table;
    const int32_t* positions;
    int heads, dim, rotary, interleaved, inverse, copy_rest;  // copy_rest: y is not x
};
cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t s);

struct AppendArgs {
    ecco_paged p;
    const DevTables* tb[2];  // K, V
    const uint16_t* x[2];
    int64_t token_stride[2], head_stride[2];
    uint8_t* pages[2];
    int64_t tokens;
    const float* rope;  // null: keys as they are
    int64_t n_positions;
    const int32_t* positions;
    int rotary, interleaved, inverse;
    ecco_stats* stats;
};
cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t s);

struct PagedAttnArgs {
    ecco_paged p;
    const DevTables* tb[2];
    const uint8_t* pages[2];
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    int64_t q_token, q_head, out_token, out_head;
    int64_t tokens;
    int group, max_q, max_kv, window;
    float scale;
};
size_t paged_attention_bytes(int batch, int kv_heads, int group, int max_q, int max_kv);
cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* workspace, cudaStream_t s);

cudaError_t launch_copy_pages(uint8_t* k, uint8_t* v, int64_t page_bytes, const int32_t* src, const int32_t* dst,
                              int64_t n, cudaStream_t s);

struct CompactArgs {
    ecco_paged p;
    uint8_t* pages[2];
    const uint8_t* keep;
    int64_t keep_stride;
    const int32_t* dst_table;
    int64_t dst_stride;
    int dst_max_pages;
    int32_t* new_lens;
};
cudaError_t launch_compact_pages(const CompactArgs& a, cudaStream_t s);

}  // namespace ecco
