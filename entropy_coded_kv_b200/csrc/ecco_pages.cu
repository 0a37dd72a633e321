// Page copies and token compaction: 64-byte blocks moved as they are, both
// bound by HBM.  On one B200: 6000 page pairs of 32 KB, K and V, in 127 us
// (6.2 TB/s read and written, two launches); half of 3 x 100000 tokens of 8
// heads kept in 71 us -- 4.3 TB/s of the blocks moved, 5.2 TB/s of DRAM
// traffic: 231 MB are read for the 154 MB kept, 3/4 of all blocks, which is what
// a random half costs when memory is fetched 128 bytes (two tokens) at a time.
// Loads that ask for 64 were not tried.
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

constexpr int kChunk = 256;  // tokens of a CTA: one a thread

// Bytes of p[0 .. n) that are not zero, this thread's share: 16 bytes at a time
// between the ends that are not aligned.
__device__ __forceinline__ int count_kept(const uint8_t* p, int n, int tid)
{
    const int head = min(n, (int)(-reinterpret_cast<uintptr_t>(p) & 15u)), body = (n - head) / 16;
    int c = 0;
    for (int i = tid; i < body; i += kThreads) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + head) + i);
        c += __popc(__vcmpne4(v.x, 0u)) + __popc(__vcmpne4(v.y, 0u)) + __popc(__vcmpne4(v.z, 0u)) +
             __popc(__vcmpne4(v.w, 0u));
    }
    c >>= 3;  // eight bits a byte
    for (int i = tid; i < head; i += kThreads) c += p[i] != 0;
    for (int i = head + 16 * body + tid; i < n; i += kThreads) c += p[i] != 0;
    return c;
}

// grid (chunks of tokens, batch).  A CTA counts the kept tokens before its
// chunk (at most one byte a token, from L2), ranks its own, and moves their
// blocks of every head, K and V: four threads a block, neighbours in the
// destination next to each other.
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactArgs A)
{
    __shared__ int s_before[kThreads / 32], s_own[kThreads / 32];
    __shared__ int64_t s_src[kChunk], s_dst[kChunk];  // block of head 0, or -1: not moved
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y, ps = A.p.page_size;
    const int n = (int)min((int64_t)paged_kv_len(A.p, b, 0x7fffffff), A.keep_stride);
    const int t0 = blockIdx.x * kChunk;
    if (t0 >= n && blockIdx.x > 0) return;
    const uint8_t* keep = A.keep + b * A.keep_stride;
    const int64_t cap = (int64_t)A.dst_max_pages * ps;

    const int t = t0 + tid;
    const bool kept = t < n && keep[t] != 0;
    const int64_t src = kept ? paged_block(A.p, b, 0, t) : -1;
    const int before = __reduce_add_sync(0xffffffffu, count_kept(keep, t0, tid));
    const uint32_t m = __ballot_sync(0xffffffffu, kept);
    if (lane == 0) {
        s_before[warp] = before;
        s_own[warp] = __popc(m);
    }
    __syncthreads();
    int first = 0, rank = __popc(m & ((1u << lane) - 1u)), mine = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        first += s_before[w];
        if (w < warp) rank += s_own[w];
        mine += s_own[w];
    }
    if (kept) {
        const int64_t to = (int64_t)first + rank;
        int64_t dst = -1;
        if (to < cap && src >= 0) {
            const int pi = (int)(to / ps);
            const int page = __ldg(A.dst_table + b * A.dst_stride + pi);
            if ((uint32_t)page < (uint64_t)A.p.n_pages) dst = (int64_t)page * A.p.kv_heads * ps + (to - (int64_t)pi * ps);
        }
        s_src[rank] = src;
        s_dst[rank] = dst;
    }
    if (tid == 0 && t0 + kChunk >= n) A.new_lens[b] = (int)min((int64_t)first + mine, cap);
    __syncthreads();

    // K and V of kBatch heads in flight (all in one pool: the compiler cannot
    // move a load over a store)
    constexpr int kBatch = 4;
    const int part = (tid & 3) * 16;
    const int64_t head = (int64_t)ps * ECCO_BLOCK_BYTES;
    for (int j = tid >> 2; j < mine; j += kThreads / 4) {
        if (s_dst[j] < 0) continue;
        const int64_t from = s_src[j] * ECCO_BLOCK_BYTES + part, to = s_dst[j] * ECCO_BLOCK_BYTES + part;
        for (int h = 0; h < A.p.kv_heads; h += kBatch) {
            uint4 v[2][kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int kv = 0; kv < 2; ++kv)
                    if (h + k < A.p.kv_heads) v[kv][k] = __ldcs(reinterpret_cast<const uint4*>(A.pages[kv] + from + (h + k) * head));
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int kv = 0; kv < 2; ++kv)
                    if (h + k < A.p.kv_heads) __stcs(reinterpret_cast<uint4*>(A.pages[kv] + to + (h + k) * head), v[kv][k]);
        }
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
    compact_kernel<<<dim3((unsigned)chunks, a.p.batch), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ecco
