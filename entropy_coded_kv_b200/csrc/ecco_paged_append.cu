// New tokens into a paged cache: keys turned by their positions, keys and
// values encoded (ecco_encode.cuh), each block written straight to its page.
//
// 16 lanes hold a group of 128 values, 8 each.  A turned pair lies in one lane
// (interleaved) or rotary / 16 lanes apart (halves), so the turn costs four
// shuffles and the cos / sin of 8 or 4 pairs, and the turned key never leaves
// the registers.
//
// Bound by the encoder's instructions (issue 68%, integer pipe 55% busy, as
// ecco_encode.cu): 53 us for 4,489 tokens of 8 heads (72 k groups, 1.36 G groups
// a second; HBM alone would take 4 us), 8 us for 8 tokens.  The division-free
// walk over (token, head) that the descriptors of ecco_encode.cu use made no
// difference here.
#include <algorithm>

#include "ecco_encode.cuh"
#include "ecco_paged.cuh"
#include "ecco_rope.cuh"

namespace ecco {
namespace {

constexpr int kWarps = 8;
constexpr int kCtasPerSm = 4;

// The lane's 8 values of a key turned to position `pos`.
__device__ __forceinline__ uint4 turn_key(const AppendArgs& A, uint4 q, int64_t pos, int hl, uint32_t gmask)
{
    pos = min(max(pos, (int64_t)0), A.n_positions - 1);
    const float* row = A.rope + pos * A.rotary;
    const int pairs8 = A.rotary / 16;  // lanes of a half
    __nv_bfloat16* e = reinterpret_cast<__nv_bfloat16*>(&q);
    if (A.interleaved) {
        if (hl < 2 * pairs8) {
            const float4* cs = reinterpret_cast<const float4*>(row + 8 * hl);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 c = __ldg(cs + k);
                rope_turn(e[4 * k], e[4 * k + 1], c.x, A.inverse ? -c.y : c.y);
                rope_turn(e[4 * k + 2], e[4 * k + 3], c.z, A.inverse ? -c.w : c.w);
            }
        }
        return q;
    }
    const bool first = hl < pairs8, turned = hl < 2 * pairs8;
    const int from = turned ? (first ? hl + pairs8 : hl - pairs8) : hl;
    uint4 o;  // the partner lane's values
    o.x = __shfl_sync(gmask, q.x, from, 16);
    o.y = __shfl_sync(gmask, q.y, from, 16);
    o.z = __shfl_sync(gmask, q.z, from, 16);
    o.w = __shfl_sync(gmask, q.w, from, 16);
    if (turned) {
        __nv_bfloat16* f = reinterpret_cast<__nv_bfloat16*>(&o);
        const float4* cs = reinterpret_cast<const float4*>(row + 16 * (first ? hl : hl - pairs8));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 c = __ldg(cs + k);
            const float s0 = A.inverse ? -c.y : c.y, s1 = A.inverse ? -c.w : c.w;
            if (first) {
                rope_turn(e[2 * k], f[2 * k], c.x, s0);
                rope_turn(e[2 * k + 1], f[2 * k + 1], c.z, s1);
            } else {
                rope_turn(f[2 * k], e[2 * k], c.x, s0);
                rope_turn(f[2 * k + 1], e[2 * k + 1], c.z, s1);
            }
        }
    }
    return q;
}

// Groups in the order K [token][head], V [token][head]; each CTA encodes one
// contiguous, equal share and stages a tensor's tables when it enters it.
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) paged_append_kernel(const __grid_constant__ AppendArgs A)
{
    __shared__ uint32_t rows[kNPat * kRow];
    __shared__ __align__(256) uint8_t qlo[kNPat * 256];
    __shared__ float4 qmap[kNPat];
    __shared__ uint32_t bufs[2 * kWarps][20];
    __shared__ uint32_t tops[2 * kWarps][kMaxRec];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t QL = (uint32_t)__cvta_generic_to_shared(qlo);
    for (int i = tid; i < 2 * kWarps * 20; i += kWarps * 32) (&bufs[0][0])[i] = 0u;
    const int sub = lane >> 4, hl = lane & 15;
    const uint32_t gmask = 0xffffu << (16 * sub);
    Counters cnt = {0, 0, 0, 0, 0, 0, 0ull};

    const int H = A.p.kv_heads;
    const int64_t each = A.tokens * H, total = 2 * each, share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t begin = (int64_t)blockIdx.x * share, end = min(total, begin + share);
    const int q0 = A.p.cu_q[0], q1 = A.p.cu_q[A.p.batch];
    for (int kv = 0; kv < 2; ++kv) {
        const int64_t lo = max(begin, kv * each) - kv * each, hi = min(end, (kv + 1) * each) - kv * each;
        if (lo >= hi) continue;
        const DevTables* tb = A.tb[kv];
        __syncthreads();  // the keys' rows are no longer read
        stage_pattern_rows<kWarps * 32>(tb, rows, qlo, qmap, tid);
        float2 ends[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ends[k] = __ldg(&tb->ends[hl + 16 * k]);
        __syncthreads();
        for (int64_t i = lo + 2 * warp + sub; i < hi; i += 2 * kWarps) {
            const int64_t t = i / H;
            const int h = (int)(i - t * H);
            if (t < q0 || t >= q1) continue;
            int b = 0, top = A.p.batch - 1;  // the last sequence that begins at or before row t
            while (b < top) {
                const int mid = (b + top + 1) >> 1;
                if (__ldg(A.p.cu_q + mid) <= t)
                    b = mid;
                else
                    top = mid - 1;
            }
            const int64_t pos = (int64_t)A.p.kv_lens[b] - ((int64_t)__ldg(A.p.cu_q + b + 1) - t);
            if (pos < 0 || pos >= paged_capacity(A.p)) continue;
            const int64_t blk = paged_block(A.p, b, h, (int)pos);
            if (blk < 0) continue;
            uint4 q = __ldg(reinterpret_cast<const uint4*>(A.x[kv] + t * A.token_stride[kv] + h * A.head_stride[kv]) + hl);
            if (kv == 0 && A.rope) q = turn_key(A, q, A.positions ? (int64_t)A.positions[t] : pos, hl, gmask);
            encode_group<0, kG>(tb, rows, QL, qmap, nullptr, bufs[2 * warp + sub], tops[2 * warp + sub], ends, q,
                                A.pages[kv] + blk * ECCO_BLOCK_BYTES, hl, gmask, kNPat, cnt);
        }
    }
    if (hl == 0) add_counters(A.stats, cnt);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t s)
{
    const int64_t total = 2 * a.tokens * a.p.kv_heads;
    const int64_t want = std::max<int64_t>(2, (total + 2 * kWarps - 1) / (2 * kWarps));
    const int64_t cap = (int64_t)device_sm_count() * kCtasPerSm;
    paged_append_kernel<<<(int)std::min(want, cap), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ecco
