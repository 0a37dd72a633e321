// Page copies and token compaction: 64-byte blocks moved as they are.
#include <algorithm>

#include "ecco_paged.cuh"

namespace ecco {
namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 3840;                // pairs a launch takes as kernel parameters (30 KB)
constexpr int64_t kPiece = kThreads * 64;   // bytes a CTA moves: 4 16-byte pieces a thread

struct CopyParams {
    uint8_t* pages[2];
    int64_t page_bytes;
    int32_t src[kPairs], dst[kPairs];
};

// grid (pieces of a page, pairs, pools); the page numbers are the launch's parameters, checked on the host
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyParams P)
{
    uint8_t* pool = P.pages[blockIdx.z];
    const uint8_t* src = pool + P.src[blockIdx.y] * P.page_bytes;
    uint8_t* dst = pool + P.dst[blockIdx.y] * P.page_bytes;
    const int64_t at = blockIdx.x * kPiece + threadIdx.x * 16;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (at + k * kThreads * 16 < P.page_bytes) v[k] = *reinterpret_cast<const uint4*>(src + at + k * kThreads * 16);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (at + k * kThreads * 16 < P.page_bytes) *reinterpret_cast<uint4*>(dst + at + k * kThreads * 16) = v[k];
}

constexpr int kChunk = 1024;  // tokens of a CTA

// grid (chunks of tokens, KV heads, batch).  A CTA counts the kept tokens
// before its chunk (the mask's bytes come from L2), scans its own, and moves
// their blocks of one head, K and V.
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactArgs A)
{
    __shared__ int s_sum[kThreads / 32], s_from[kChunk], s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.z, h = blockIdx.y;
    const int n = (int)min((int64_t)paged_kv_len(A.p, b, 0x7fffffff), A.keep_stride);
    const int t0 = blockIdx.x * kChunk;
    if (t0 >= n && blockIdx.x > 0) return;
    const uint8_t* keep = A.keep + b * A.keep_stride;
    const int64_t cap = (int64_t)A.dst_max_pages * A.p.page_size;

    auto block_sum = [&](int v) {
        v = __reduce_add_sync(0xffffffffu, v);
        __syncthreads();
        if (lane == 0) s_sum[warp] = v;
        __syncthreads();
        int r = 0;
        for (int w = 0; w < kThreads / 32; ++w) r += s_sum[w];
        return r;
    };
    int before = 0;
    for (int t = tid; t < t0; t += kThreads) before += keep[t] != 0;
    before = block_sum(before);

    if (tid == 0) s_n = 0;
    __syncthreads();
    for (int base = 0; base < kChunk; base += kThreads) {  // the chunk's kept tokens, in order
        const int t = t0 + base + tid;
        const bool k = t < n && keep[t] != 0;
        const uint32_t m = __ballot_sync(0xffffffffu, k);
        if (lane == 0) s_sum[warp] = __popc(m);
        __syncthreads();
        int at = s_n, all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += s_sum[w];
            all += s_sum[w];
        }
        if (k) s_from[at + __popc(m & ((1u << lane) - 1u))] = t;
        __syncthreads();
        if (tid == 0) s_n += all;
        __syncthreads();
    }
    const int mine = s_n;
    if (h == 0 && t0 + kChunk >= n && tid == 0) A.new_lens[b] = (int)min((int64_t)before + mine, cap);

    for (int i = tid; i < mine * 8; i += kThreads) {  // 16 bytes each: K then V of a token
        const int j = i >> 3, part = i & 3;
        const int64_t to = (int64_t)before + j;
        if (to >= cap) continue;
        const int64_t sb = paged_block(A.p, b, h, s_from[j]);
        const int pi = (int)(to / A.p.page_size);
        const int page = __ldg(A.dst_table + b * A.dst_stride + pi);
        if (sb < 0 || (uint32_t)page >= (uint64_t)A.p.n_pages) continue;
        const int64_t db = ((int64_t)page * A.p.kv_heads + h) * A.p.page_size + (to - (int64_t)pi * A.p.page_size);
        uint8_t* pool = A.pages[(i >> 2) & 1];
        *reinterpret_cast<uint4*>(pool + db * ECCO_BLOCK_BYTES + part * 16) =
            *reinterpret_cast<const uint4*>(pool + sb * ECCO_BLOCK_BYTES + part * 16);
    }
}

}  // namespace

cudaError_t launch_copy_pages(uint8_t* k, uint8_t* v, int64_t page_bytes, const int32_t* src, const int32_t* dst,
                              int64_t n, cudaStream_t s)
{
    for (int64_t i = 0; i < n; i += kPairs) {
        CopyParams P;
        const int m = (int)std::min<int64_t>(kPairs, n - i);
        P.pages[0] = k;
        P.pages[1] = v;
        P.page_bytes = page_bytes;
        std::copy(src + i, src + i + m, P.src);
        std::copy(dst + i, dst + i + m, P.dst);
        copy_pages_kernel<<<dim3((unsigned)((page_bytes + kPiece - 1) / kPiece), m, 2), kThreads, 0, s>>>(P);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_compact_pages(const CompactArgs& a, cudaStream_t s)
{
    const int64_t chunks = std::max<int64_t>(1, (paged_capacity(a.p) + kChunk - 1) / kChunk);
    compact_kernel<<<dim3((unsigned)chunks, a.p.kv_heads, a.p.batch), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ecco
