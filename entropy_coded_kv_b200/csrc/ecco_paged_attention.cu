// Attention of new tokens over a paged compressed cache.
//
// Two launches a round of KV heads: the visible keys' and values' blocks are
// decoded into a scratch of 128-token tiles, then the attention kernel reads
// the tiles.
#include <algorithm>

#include "ecco_block.cuh"
#include "ecco_paged.cuh"

namespace ecco {
namespace {

constexpr int kTile = 128;                     // tokens of a scratch tile
constexpr int kTileBytes = kTile * kG * 2;     // one head's K (or V) of a tile
constexpr int64_t kRoundBytes = (int64_t)1 << 30;

// What the device-side arrays say of one sequence, bounded.
struct Seq {
    int q0, q;      // its rows: q0 .. q0 + q - 1
    int base;       // position of row q0 (new token i is at base + i); may be negative
    int keys;       // keys that exist (bounded by max_kv and the page table)
};

struct Bounds {
    int64_t tokens;
    int max_q, max_kv, window;
};

__device__ __forceinline__ Seq seq_of(const ecco_paged& p, const Bounds& w, int b)
{
    const int64_t a = p.cu_q[b], e = p.cu_q[b + 1], n = p.kv_lens[b];
    Seq s;
    const int64_t first = min(max(a, (int64_t)0), w.tokens);
    const int64_t all = max(e - a, (int64_t)0);
    s.q0 = (int)first;
    s.q = (a < 0) ? 0 : (int)min(min(all, (int64_t)w.max_q), w.tokens - first);
    s.base = (int)min(max(n - all, -((int64_t)1 << 30)), (int64_t)1 << 30);
    s.keys = paged_kv_len(p, b, w.max_kv);
    return s;
}

// Keys [lo, hi) that new tokens i0 .. i1 of the sequence see between them.
__device__ __forceinline__ void visible(const Seq& s, int window, int i0, int i1, int& lo, int& hi)
{
    hi = min(s.keys, s.base + i1 + 1);
    lo = window > 0 ? max(0, s.base + i0 - window + 1) : 0;
    if (hi <= lo) lo = hi = 0;
}

// The tiles of sequence b that are decoded: [first, first + count).
__device__ __forceinline__ void seq_tiles(const Seq& s, int window, int& first, int& count)
{
    int lo = 0, hi = 0;
    if (s.q > 0) visible(s, window, 0, s.q - 1, lo, hi);
    first = lo / kTile;
    count = (hi + kTile - 1) / kTile - first;
    if (hi <= lo) count = 0;
}

// Exclusive prefix sums of v[0..n) in place, v[n] = the total.  One warp.
__device__ __forceinline__ void warp_prefix(int* v, int n, int lane)
{
    int run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane, x = i < n ? v[i] : 0;
        int s = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += t;
        }
        if (i < n) v[i] = run + s - x;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) v[n] = run;
}

// Last b with v[b] <= x (v non-decreasing, v[0] <= x < v[n]).
__device__ __forceinline__ int find_seq(const int* v, int n, int x)
{
    int b = 0, top = n - 1;
    while (b < top) {
        const int mid = (b + top + 1) >> 1;
        if (v[mid] <= x)
            b = mid;
        else
            top = mid - 1;
    }
    return b;
}

// Byte offset of 16-byte piece c (0..15) of row r in a tile: two halves of 64
// values, 128 bytes a row, the 8 pieces of a row XOR-ed with the row's low
// bits -- the 128-byte swizzle that the tensor cores read, so a tile goes to
// shared memory as one contiguous copy.
__device__ __forceinline__ uint32_t tile_offset(int r, int c)
{
    return (uint32_t)((c >> 3) * (kTileBytes / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ------------------------------------------------------------ decode into tiles
constexpr int kDecThreads = 896;
constexpr size_t kDecLut = sizeof(((DevTables*)0)->lut), kDecCt = sizeof(((DevTables*)0)->Ct);
constexpr size_t kDecSmem = kSmemAlign + kDecLut + kDecCt + (size_t)16 * kDecThreads * 4 +
                            (size_t)(2 * ECCO_MAX_BATCH + 1) * sizeof(int);

struct StageArgs {
    ecco_paged p;
    Bounds w;
    const DevTables* tb[2];
    const uint8_t* pages[2];
    uint8_t* scratch;  // [2][heads of the round][tiles][kTileBytes]
    int h0, hn;
};

// Stores values 16 j .. 16 j + 15 of a row: its 32-byte piece, the two halves
// swapped in odd rows.
__device__ __forceinline__ void store_piece(uint8_t* row, uint32_t x, int j, const uint32_t a[4], const uint32_t b[4])
{
    uint8_t* d = row + (j >> 2) * (kTileBytes / 2) + (((j & 3) ^ (x >> 1)) << 5);
    if (x & 1u)
        stg256(d, b, a);
    else
        stg256(d, a, b);
}

__global__ void __launch_bounds__(kDecThreads, 1) paged_decode_kernel(const __grid_constant__ StageArgs A)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = aligned_smem(smem_raw);
    uint8_t* s_lut = smem;
    float* s_Ct = reinterpret_cast<float*>(smem + kDecLut);
    uint32_t* s_w = reinterpret_cast<uint32_t*>(smem + kDecLut + kDecCt);
    int* s_cu = reinterpret_cast<int*>(s_w + 16 * kDecThreads);  // [batch + 1] tiles before sequence b
    int* s_first = s_cu + ECCO_MAX_BATCH + 1;                    // [batch] its first tile
    const int tid = threadIdx.x;
    uint32_t* ws = s_w + tid;

    for (int b = tid; b < A.p.batch; b += kDecThreads) {
        int first, count;
        seq_tiles(seq_of(A.p, A.w, b), A.w.window, first, count);
        s_cu[b] = count;
        s_first[b] = first;
    }
    __syncthreads();
    if (tid < 32) warp_prefix(s_cu, A.p.batch, tid);
    __syncthreads();
    const int tiles = s_cu[A.p.batch];
    const int64_t each = (int64_t)tiles * A.hn * kTile, total = 2 * each;
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t begin = (int64_t)blockIdx.x * share, end = min(total, begin + share);

    for (int kv = 0; kv < 2; ++kv) {
        const int64_t lo = max(begin, kv * each) - kv * each, hi = min(end, (kv + 1) * each) - kv * each;
        if (lo >= hi) continue;
        const DevTables* tb = A.tb[kv];
        const uint8_t* pool = A.pages[kv];
        uint8_t* out = A.scratch + (int64_t)kv * A.hn * tiles * kTileBytes;
        __syncthreads();  // the keys' tables are no longer read
        stage_tables<kDecThreads>(tb, s_lut, s_Ct, tid);
        const float S_t = tb->S_t;
        __syncthreads();

        // the source block of row `i` of the round, or null: past the keys, or in no page
        auto locate = [&](int64_t i) -> const uint8_t* {
            const int lin = (int)(i >> 7), h = lin / tiles, tile = lin - h * tiles;
            const int b = find_seq(s_cu, A.p.batch, tile);
            const int t = (s_first[b] + tile - s_cu[b]) * kTile + (int)(i & (kTile - 1));
            if (t >= paged_kv_len(A.p, b, A.w.max_kv)) return nullptr;
            const int64_t blk = paged_block(A.p, b, A.h0 + h, t);
            return blk < 0 ? nullptr : pool + blk * ECCO_BLOCK_BYTES;
        };
        const int part = (int)(hi - lo);
        const int rounds = (part + kDecThreads - 1) / kDecThreads, per_round = (part + rounds - 1) / rounds;
        const int64_t stop = (tid < per_round) ? hi : 0;
        int64_t i = lo + tid;
        const uint8_t* src = i < stop ? locate(i) : nullptr;
        for (; i < stop; i += per_round) {
            uint8_t* row = out + (i >> 7) * kTileBytes + (i & (kTile - 1)) * 128;
            const uint32_t x = (uint32_t)(i & 7);
            uint4 q0 = make_uint4(0u, 0u, 0u, 0u), q1 = q0, q2 = q0, q3 = q0;
            if (src) {
                q0 = ldg_nc_v4(src);
                q1 = ldg_nc_v4(src + 16);
                q2 = ldg_nc_v4(src + 32);
                q3 = ldg_nc_v4(src + 48);
            }
            if (i + per_round < stop) {  // this thread's next block: on its way to L2 while this one decodes
                src = locate(i + per_round);
                if (src) asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
            }
            const uint32_t code = q0.x & 0xffu;
            if (scale_code_is_null(code)) {
                const uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < kG / 16; ++j) store_piece(row, x, j, z, z);
                continue;
            }
            stage_words(ws, kDecThreads, q0, q1, q2, q3);
            const int p = (int)((q0.x >> 8) & 63u);
            const uint32_t lkey = lut_key(s_lut, (q0.x >> 8) & 255u);
            const float s = __fmul_rn(S_t, e4m3_to_f32(code));
            const ValuePlanes vp = make_planes(s, s_Ct, p);
            Stream st{q0.x, q0.y, kHdrBits, 2, kPayloadBits};
#pragma unroll 1
            for (int j = 0; j < kG / 16; ++j) {
                uint32_t wa[4], wb[4];
                chunk_values(st, lkey, ws, kDecThreads, vp, wa);
                chunk_values(st, lkey, ws, kDecThreads, vp, wb);
                store_piece(row, x, j, wa, wb);
            }
            if (st.room >= 0) {  // unclipped: outlier records follow the codewords
                const int n = min(kMaxRec, st.room / kRecBits), at0 = kBlockBits - st.room;
                for (int k = 0; k < n; ++k) {
                    const uint32_t rec = read_record(ws, kDecThreads, at0 + k * kRecBits), e = rec & 127u;
                    const float o = q_over_127((int)(int8_t)(uint8_t)(rec >> 7));
                    *reinterpret_cast<uint16_t*>(row + (e >> 6) * (kTileBytes / 2) + ((((e >> 3) & 7u) ^ x) << 4) +
                                                 (e & 7u) * 2) = (uint16_t)f32_to_bf16_bits(__fmul_rn(s, o));
                }
            }
        }
    }
}

// ------------------------------------------------------------ attention
struct AttnArgs {
    ecco_paged p;
    Bounds w;
    const uint8_t* scratch;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    int64_t q_token, q_head, out_token, out_head;
    int group, h0, hn;
    float scale;
};

constexpr int kWarps = 8;

// One warp a (row, query head): lane l holds values 4 l .. 4 l + 3.
__global__ void __launch_bounds__(kWarps * 32) paged_attention_kernel(const __grid_constant__ AttnArgs A)
{
    __shared__ int s_cu[ECCO_MAX_BATCH + 1], s_first[ECCO_MAX_BATCH];
    const int tid = threadIdx.x, lane = tid & 31;
    for (int b = tid; b < A.p.batch; b += kWarps * 32) {
        int first, count;
        seq_tiles(seq_of(A.p, A.w, b), A.w.window, first, count);
        s_cu[b] = count;
        s_first[b] = first;
    }
    __syncthreads();
    if (tid < 32) warp_prefix(s_cu, A.p.batch, tid);
    __syncthreads();
    const int tiles = s_cu[A.p.batch], heads = A.hn * A.group;
    for (int b = 0; b < A.p.batch; ++b) {
        const Seq s = seq_of(A.p, A.w, b);
        const int64_t work = (int64_t)s.q * heads;
        for (int64_t u = (int64_t)blockIdx.x * kWarps + (tid >> 5); u < work; u += (int64_t)gridDim.x * kWarps) {
            const int i = (int)(u / heads), j = (int)(u - (int64_t)i * heads), h = j / A.group;
            const int64_t row = s.q0 + i;
            const int qh = A.h0 * A.group + j;
            const uint16_t* q = A.q + row * A.q_token + qh * A.q_head + 4 * lane;
            float qv[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) qv[k] = bf16_bits_to_f32(q[k]);
            int lo, hi;
            visible(s, A.w.window, i, i, lo, hi);
            for (int t = lo; t < hi; ++t) {
                const int64_t tile = (int64_t)h * tiles + s_cu[b] + t / kTile - s_first[b];
                const uint8_t* kt = A.scratch + tile * kTileBytes;
                const uint8_t* vt = kt + (int64_t)A.hn * tiles * kTileBytes;
                const uint32_t at = tile_offset(t % kTile, lane >> 1) + (lane & 1) * 8;
                const uint2 kw = *reinterpret_cast<const uint2*>(kt + at), vw = *reinterpret_cast<const uint2*>(vt + at);
                float d = qv[0] * __uint_as_float(kw.x << 16) + qv[1] * __uint_as_float(kw.x & 0xffff0000u) +
                          qv[2] * __uint_as_float(kw.y << 16) + qv[3] * __uint_as_float(kw.y & 0xffff0000u);
#pragma unroll
                for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
                d *= A.scale;
                const float mn = fmaxf(m, d), c = __expf(m - mn), p = __expf(d - mn);
                m = mn;
                l = l * c + p;
                o[0] = o[0] * c + p * __uint_as_float(vw.x << 16);
                o[1] = o[1] * c + p * __uint_as_float(vw.x & 0xffff0000u);
                o[2] = o[2] * c + p * __uint_as_float(vw.y << 16);
                o[3] = o[3] * c + p * __uint_as_float(vw.y & 0xffff0000u);
            }
            const float inv = hi > lo ? 1.0f / l : 0.0f;
            uint2 w;
            w.x = pack_bf16x2(o[0] * inv, o[1] * inv);
            w.y = pack_bf16x2(o[2] * inv, o[3] * inv);
            *reinterpret_cast<uint2*>(A.out + row * A.out_token + qh * A.out_head + 4 * lane) = w;
            if (A.lse && lane == 0)
                A.lse[row * (int64_t)A.p.kv_heads * A.group + qh] = hi > lo ? m + logf(l) : -INFINITY;
        }
    }
}

// Heads of a round: as many as keep the scratch within kRoundBytes, at least one.
int round_heads(int batch, int kv_heads, int max_kv)
{
    const int64_t per_head = 2 * (int64_t)batch * ((max_kv + kTile - 1) / kTile) * kTileBytes;
    return (int)std::max<int64_t>(1, std::min<int64_t>(kv_heads, per_head ? kRoundBytes / per_head : kv_heads));
}

}  // namespace

size_t paged_attention_bytes(int batch, int kv_heads, int group, int max_q, int max_kv)
{
    const int64_t tiles = (int64_t)batch * ((max_kv + kTile - 1) / kTile);
    return (size_t)(2 * round_heads(batch, kv_heads, max_kv) * tiles * kTileBytes) + 1024;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* workspace, cudaStream_t s)
{
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_max_smem_once(configured, (const void*)paged_decode_kernel, kDecSmem);
    if (e != cudaSuccess) return e;
    uint8_t* scratch = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 1023) / 1024 * 1024);
    const int hn = round_heads(a.p.batch, a.p.kv_heads, a.max_kv);
    const Bounds w{a.tokens, a.max_q, a.max_kv, a.window};
    for (int h0 = 0; h0 < a.p.kv_heads; h0 += hn) {
        const int n = std::min(hn, a.p.kv_heads - h0);
        const StageArgs st{a.p, w, {a.tb[0], a.tb[1]}, {a.pages[0], a.pages[1]}, scratch, h0, n};
        paged_decode_kernel<<<device_sm_count(), kDecThreads, kDecSmem, s>>>(st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const AttnArgs at{a.p, w, scratch, a.q, a.out, a.lse, a.q_token, a.q_head, a.out_token, a.out_head,
                          a.group, h0, n, a.scale};
        paged_attention_kernel<<<device_sm_count() * 8, kWarps * 32, 0, s>>>(at);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ecco
