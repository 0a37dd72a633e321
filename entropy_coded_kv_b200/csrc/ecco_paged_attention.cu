// Attention of new tokens over a paged compressed cache.
//
// Few rows over few keys take one kernel (paged_small_kernel), everything else
// three a round of KV heads: the visible keys' and values' blocks are
// decoded into a scratch of 128-token tiles (each once, whatever the number of
// new tokens), the attention kernel reads the tiles, and the items that it cut
// are joined.  On one B200, 32 query and 8 KV heads, whole calls replayed from
// a graph (medians; the long ones under the 1 kW power cap):
//   1 new over 650 keys          13.8 us  (one kernel; 22 in three)
//   8 x 1 new over up to 4096      72 us  (decode 47, attention 21, join 3)
//   500 new over 131072          1.43 ms  (decode 0.22; 750 TFLOP/s)
//   4096 new over 16384          0.96 ms  (1.0 PFLOP/s; 0.83 ms at full clock)
// The single tokens are bound by the decoder's serial walk (ecco_decode.cu) and
// by latencies, the prompts by the exponentials and
// the hand-overs between softmax and tensor cores.
#include <algorithm>

#include "ecco_block.cuh"
#include "ecco_paged.cuh"

namespace ecco {
namespace {

constexpr int kTile = 128;                     // tokens of a scratch tile
// One head's K (or V) of a tile: two halves of 64 values, 128 bytes a row, the
// eight 16-byte pieces of a row XOR-ed with the row's low three bits -- the
// 128-byte swizzle that the tensor cores read, so a tile goes to shared memory
// as one contiguous copy.
constexpr int kTileBytes = kTile * kG * 2;
// The scratch of a round of KV heads, or of one head where that is more (128
// sequences of 131072 keys: 8.6 GB).  Rounds within 140 or 280 MB took 71.5 and
// 70.4 us for 70.6 at 8 x 1 over up to 4096, 179 and 165 for 165.7 at 1 over
// 60000; larger calls were not compared.
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

// ------------------------------------------------------------ barriers, copies, launches
constexpr uint32_t kSpinLimit = 1u << 17;
__device__ unsigned int g_timeouts = 0;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// One untiled copy to shared memory, counted on `bar` (16-byte aligned, a
// multiple of 16 bytes).
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A wait that gives up counts itself, raises the host-visible flag and marks
// the CTA dead, so that its other waits end too.
__device__ __noinline__ void wait_gave_up(volatile uint32_t* dead, int* flag)
{
    *dead = 1u;
    atomicAdd(&g_timeouts, 1u);
    if (flag) {
        *reinterpret_cast<volatile int*>(flag) = 1;
        __threadfence_system();
    }
}

// Waits for the phase of the given parity: at most `limit` polls, each of which
// the hardware suspends for some microseconds (kSpinLimit: about a second).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* dead, int* flag,
                                          uint32_t limit = kSpinLimit)
{
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if (*dead) return false;
    }
    wait_gave_up(dead, flag);
    return false;
}

// The kernels of a call follow one another with programmatic launches: the
// next one's CTAs may start (and plan, and load their queries) once every CTA
// has come this far and left its SM; they wait with after_previous() before
// they touch what the previous kernel writes.  Every CTA of a kernel waits, so
// that its end means the previous one's.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------ decode into tiles
constexpr int kDecThreads = 896;
constexpr size_t kDecLut = sizeof(((DevTables*)0)->lut), kDecCt = sizeof(((DevTables*)0)->Ct);
constexpr size_t kDecSmem = kSmemAlign + kDecLut + kDecCt + (size_t)16 * kDecThreads * 4 +
                            (size_t)(3 * ECCO_MAX_BATCH + 1) * sizeof(int);

struct StageArgs {
    ecco_paged p;
    Bounds w;
    const DevTables* tb[2];
    const uint8_t* pages[2];
    uint8_t* scratch;  // [2][heads of the round][tiles][kTileBytes]
    int h0, hn;
    bool wide;  // pools 32-byte aligned: 32-byte loads
    int* flag;
};

// The first half of the CTAs decodes the keys, the second the values, each an
// equal run of rows of the round's tiles, one row a thread; a CTA's tables come
// by bulk copies while it works out where its rows are.  The walk is
// ecco_decode.cu's, bound by the L1's data path and the integer pipe (72 and
// 68% busy): 47 us for 0.37 M blocks, 9.4 G blocks/s on 2.1 M.
__global__ void __launch_bounds__(kDecThreads, 1) paged_decode_kernel(const __grid_constant__ StageArgs A)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar;
    uint8_t* smem = aligned_smem(smem_raw);
    uint8_t* s_lut = smem;
    float* s_Ct = reinterpret_cast<float*>(smem + kDecLut);
    uint32_t* s_w = reinterpret_cast<uint32_t*>(smem + kDecLut + kDecCt);
    int* s_cu = reinterpret_cast<int*>(s_w + 16 * kDecThreads);  // [batch + 1] tiles before sequence b
    int* s_first = s_cu + ECCO_MAX_BATCH + 1;                    // [batch] its first tile
    int* s_keys = s_first + ECCO_MAX_BATCH;                      // [batch] its keys
    const int tid = threadIdx.x;
    uint32_t* ws = s_w + tid;
    const int half = gridDim.x / 2, kv = blockIdx.x >= half;
    const DevTables* tb = A.tb[kv];
    launch_dependents();

    const uint32_t bar = smem_u32(&s_bar);
    if (tid == 0) {
        mbar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_expect(bar, (uint32_t)(kDecLut + kDecCt));
        bulk_copy(smem_u32(s_lut), &tb->lut[0][0], (uint32_t)kDecLut, bar);
        bulk_copy(smem_u32(s_Ct), &tb->Ct[0][0], (uint32_t)kDecCt, bar);
    }
    for (int b = tid; b < A.p.batch; b += kDecThreads) {
        int first, count;
        const Seq s = seq_of(A.p, A.w, b);
        seq_tiles(s, A.w.window, first, count);
        s_cu[b] = count;
        s_first[b] = first;
        s_keys[b] = s.keys;
    }
    __syncthreads();
    if (tid < 32) warp_prefix(s_cu, A.p.batch, tid);
    __syncthreads();
    const int tiles = s_cu[A.p.batch];
    const int64_t total = (int64_t)tiles * A.hn * kTile;
    const int64_t share = ((total + half - 1) / half + 1) & ~(int64_t)1;  // even, so that lane pairs stay together
    const int64_t lo = (int64_t)(blockIdx.x - kv * half) * share, hi = min(total, lo + share);
    const uint8_t* pool = A.pages[kv];
    uint8_t* out = A.scratch + (int64_t)kv * A.hn * tiles * kTileBytes;

    // the source block of row `i` of the round, or null: past the keys, or in no page
    auto locate = [&](int64_t i) -> const uint8_t* {
        const int lin = (int)(i >> 7), h = lin / tiles, tile = lin - h * tiles;
        const int b = find_seq(s_cu, A.p.batch, tile);
        const int t = (s_first[b] + tile - s_cu[b]) * kTile + (int)(i & (kTile - 1));
        if (t >= s_keys[b]) return nullptr;
        const int64_t blk = paged_block(A.p, b, A.h0 + h, t);
        return blk < 0 ? nullptr : pool + blk * ECCO_BLOCK_BYTES;
    };
    const int part = (int)max(hi - lo, (int64_t)0);
    const int rounds = max(1, (part + kDecThreads - 1) / kDecThreads), per_round = ((part + rounds - 1) / rounds + 1) & ~1;
    const int64_t stop = (tid < per_round) ? hi : 0;
    int64_t i = lo + tid;
    const uint8_t* src = i < stop ? locate(i) : nullptr;
    uint32_t dead = 0u;
    // The lanes trade values below: all of a warp go on, or none.
    if (!__all_sync(0xffffffffu, mbar_wait(bar, 0u, &dead, A.flag))) {  // no tables: nothing is decoded, and the flag says so
        dead = 0u;
        mbar_wait(bar, 0u, &dead, nullptr);  // the copies have landed before the CTA ends
        return;
    }
    const float S_t = tb->S_t;
    for (; i < stop; i += per_round) {
        const int here = min((int)(hi - (i - (tid & 31))), per_round - (tid & ~31));  // rows of this warp in the round: even
        const unsigned pm = here >= 32 ? 0xffffffffu : (1u << here) - 1u;
        uint8_t* even = out + (i >> 7) * kTileBytes + (i & (kTile - 2)) * 128;  // the pair's first row (an even one)
        const uint32_t x = (uint32_t)(i & 7);
        uint4 q0 = make_uint4(0u, 0u, 0u, 0u), q1 = q0, q2 = q0, q3 = q0;
        if (src) {
            if (A.wide) {
                ldg_nc_v8(src, q0, q1);
                ldg_nc_v8(src + 32, q2, q3);
            } else {
                q0 = ldg_nc_v4(src);
                q1 = ldg_nc_v4(src + 16);
                q2 = ldg_nc_v4(src + 32);
                q3 = ldg_nc_v4(src + 48);
            }
        }
        if (i + per_round < stop) {  // this thread's next block: on its way to L2 while this one decodes
            src = locate(i + per_round);
            if (src) asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
        }
        const uint32_t code = q0.x & 0xffu;
        const bool null = scale_code_is_null(code);
        stage_words(ws, kDecThreads, q0, q1, q2, q3);
        const int p = (int)((q0.x >> 8) & 63u);
        const uint32_t lkey = lut_key(s_lut, (q0.x >> 8) & 255u);
        const float s = __fmul_rn(S_t, e4m3_to_f32(code));
        ValuePlanes vp = make_planes(s, s_Ct, p);
        if (null) {  // 128 times +0, whatever the stream says
#pragma unroll
            for (int k = 0; k < 4; ++k) vp.lo[k] = vp.hi[k] = 0u;
        }
        Stream st{q0.x, q0.y, kHdrBits, 2, kPayloadBits};
        // Lanes 2k and 2k + 1 store 64 contiguous bytes of one row an instruction
        // (ecco_decode.cu measured the pairing): each sends its partner the 16
        // values that belong to the partner's store.  A 32-byte piece stays a
        // piece under the swizzle, its halves swapped in odd rows.
        const bool odd = tid & 1;
#pragma unroll 1
        for (int c = 0; c < kG / 16; c += 2) {
            uint32_t a0[4], b0[4], a1[4], b1[4], ra[4], rb[4];
            chunk_values(st, lkey, ws, kDecThreads, vp, a0);
            chunk_values(st, lkey, ws, kDecThreads, vp, b0);
            chunk_values(st, lkey, ws, kDecThreads, vp, a1);
            chunk_values(st, lkey, ws, kDecThreads, vp, b1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // the even lane sends piece c + 1, the odd lane piece c
                ra[k] = __shfl_xor_sync(pm, odd ? a0[k] : a1[k], 1);
                rb[k] = __shfl_xor_sync(pm, odd ? b0[k] : b1[k], 1);
            }
            const int j = c + odd;
            uint8_t* d = even + (j >> 2) * (kTileBytes / 2) + (((j & 3) ^ (x >> 1)) << 5);
            if (odd) {
                stg256(d, ra, rb);
                stg256(d + 128, b1, a1);
            } else {
                stg256(d, a0, b0);
                stg256(d + 128, rb, ra);
            }
        }
        __syncwarp(pm);  // the partner's part of this row is stored before the records change it
        if (!null && st.room >= 0) {  // unclipped: outlier records follow the codewords
            uint8_t* row = even + (odd ? 128 : 0);
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

// ------------------------------------------------------------ attention
// Persistent kernel, one CTA an SM.  An item is (sequence, KV head, 256 rows),
// a row being (new token, query head of the group), so that a tile of keys
// serves every query head that shares it.  An item costs, for each 128-key
// tile that its rows see, two units, or one if it has at most 128 rows; the
// units of all items, in one line, are cut into equal shares, so a CTA's share
// may begin and end inside items: such parts leave (O, max, sum) in the
// workspace, and a second kernel joins them.  The cut needs no rule for the
// number of splits, and prompts with triangular costs, ragged batches and
// single tokens over a long cache all fill the SMs alike.
//
// Inside an item, two engines alternate on the tensor cores:
//   S_i = Q_i K_j^T   (128 x 128 x 128, both from shared memory, into TMEM)
//   P_i = exp2(c S_i - c m), one thread a row, back to TMEM as bf16 over S_i
//   O_i += P_i V_j    (P from TMEM, V as it lies: rows of keys, N-major)
// With more than 128 rows ("wide") engine i has rows 128 i .. of every tile;
// with fewer ("thin") both have the same rows, engine i the key tiles i, i + 2,
// .. of the part, and engine 0 joins the two; or two thin parts of as many tiles
// have an engine each.  Warps 0-3 and 4-7 are the
// engines' softmax, a thread a row = a TMEM lane; warp 8 issues the products,
// warp 9 the copies (a tile is one 32 KB bulk copy), warp 10 works out the
// share's parts and hands them to the others.
// The maximum m is only moved, and O rescaled, when a row's new maximum is
// above it by more than 2^8: until then the weights stay below 2^8 and sum and
// products are as exact as with the true maximum.
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
    // partial results: slots 2c (a share's part of an item begun before it) and
    // 2c + 1 (an item that goes on in the next share) of CTA c
    float* part_o;   // [slot][32][slot_rows] float4
    float* part_ml;  // [slot][2][slot_rows]: maximum (in units of log2), sum
    int4* part_item; // [CTA]: the item begun in this share and unfinished -- first token row of its sequence, head (< 0: there
                     // is none), first row, last CTA that has a part of it + 2^16 times its rows
    int slot_rows;
    int* flag;
};

constexpr int kRows = 256;               // rows of an item
constexpr int kAttnThreads = 352;        // 8 softmax warps, products, copies, plan
constexpr int kStages = 4;               // K and V tiles in flight
constexpr int kParts = 4;                // parts (or pairs) planned ahead
constexpr int kPartBytes = 96;           // two of 48
constexpr int kPairTiles = 8;            // the longest first part of a pair
constexpr int kMaxCtas = 160;            // shares (and twice as many slots) at most
constexpr int kBars = 2 * kStages + 2 * kParts + 13;
constexpr size_t kOffRing = 2 * kTileBytes;
constexpr size_t kOffBars = kOffRing + (size_t)kStages * kTileBytes;
constexpr size_t kOffParts = kOffBars + (kBars * 8 + 8 + 15) / 16 * 16;  // the barriers, tensor-memory address, dead mark
constexpr size_t kOffMl = kOffParts + kParts * kPartBytes;               // engine 1's maxima and sums, for engine 0
constexpr size_t kOffSeq = kOffMl + 256 * sizeof(float);
constexpr size_t kOffUnits = kOffSeq + 16 * ECCO_MAX_BATCH;
constexpr size_t kOffTile = kOffUnits + 8 * (ECCO_MAX_BATCH + 1);
constexpr size_t kAttnSmem = 1024 + kOffTile + 4 * ECCO_MAX_BATCH;

// D fp32, A and B bf16, N = 128, M = 128; kIdescPV: B N-major (bit 16).
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);
constexpr uint32_t kNegateA = 1u << 13;  // for a negative scale

// Shared-memory matrix descriptor with the 128-byte swizzle (layout type 2):
// 8-row groups 1024 bytes apart; leading offset = the distance between the
// 64-value halves (used where the values run along N).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)((kTileBytes / 2) >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// The issuing warp runs as a whole (`leader` is true in one lane), so that the
// operands stay in uniform registers: issued from a branch of one lane, the
// eight products of a tile took 600 cycles to issue, more than they run.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kIdescPV), "r"(accumulate), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(leader)
        : "memory");
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

#define ECCO_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define ECCO_I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])

// 32 columns of this warp's 32 lanes; the registers hold them after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : ECCO_R8(v, 0), ECCO_R8(v, 8), ECCO_R8(v, 16), ECCO_R8(v, 24)
        : "r"(addr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : ECCO_R8(v, 0), ECCO_R8(v, 8)
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::ECCO_I8(v, 0),
        ECCO_I8(v, 8), "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The weights 2^(c s - mc) of 32 scores, packed as bf16 into w, their sum added
// to `sum`.  bf16, because the second product takes both operands in one type and
// V~ is bf16 by its definition: fp16 would lose its range, and tf32 halves the
// rate and doubles the tiles.  The sum is of the fp32 weights, which the lse needs.
// A weight is off by half a step (2^-8) at most; the outputs are 1.04 to 1.29
// times as far from 64 bits as the same sums with fp32 weights (relative norm
// 1.6e-3, the output's own rounding, and up to 2.1e-3).
__device__ __forceinline__ void weights(const uint32_t* v, uint64_t c2, uint64_t mc2, uint32_t* w, uint64_t (&sum)[2])
{
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float a, b;
        unpair(fma2(pair(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2, mc2), a, b);
        a = ex2(a);
        b = ex2(b);
        sum[k & 1] = add2(sum[k & 1], pair(a, b));
        w[k] = pack_bf16x2(a, b);
    }
}

// The tiles [t0, t0 + n) that rows 256 qt .. of the sequence see, and its rows.
struct Span {
    int t0, n, rows;
};

__device__ __forceinline__ Span span_of(const Seq& s, int group, int window, int qt)
{
    Span r;
    const int r0 = qt * kRows;
    r.rows = min(kRows, s.q * group - r0);
    int lo, hi;
    visible(s, window, r0 / group, (r0 + r.rows - 1) / group, lo, hi);
    r.t0 = lo / kTile;
    r.n = hi > lo ? (hi + kTile - 1) / kTile - r.t0 : 0;
    return r;
}

// Units that a key tile of the span costs.
__device__ __forceinline__ int tile_cost(const Span& r) { return r.rows > 128 ? 2 : 1; }

// What the planning warp keeps in shared memory.
struct Plan {
    uint8_t* at;
    __device__ __forceinline__ int4* seqs() const { return reinterpret_cast<int4*>(at + kOffSeq); }
    __device__ __forceinline__ long long* units() const { return reinterpret_cast<long long*>(at + kOffUnits); }  // before sequence b, over the round's heads
    __device__ __forceinline__ int* tile() const { return reinterpret_cast<int*>(at + kOffTile); }  // scratch tile of (head 0, key tile 0) of sequence b
    __device__ __forceinline__ Seq seq(int b) const
    {
        const int4 v = seqs()[b];
        return Seq{v.x, v.y, v.z, v.w};
    }
};

// One part of an item, as the planning warp hands it to the others: key tiles
// [t0, t0 + n) of rows g0 .. g0 + rows - 1 (row = new token * group + query head
// of the group).  Two thin parts that follow one another and have as many tiles
// (or the second one less) go as a pair, an engine each: the copies and products
// are those of one thin part of the sum of their tiles.  Many short sequences of
// 8 heads, us a call without pairs and with: 128 x 1 over up to 100 keys 73.8 and
// 62.7, over 650 189 and 177.5, 64 x 4 over 200 65.2 and 54.8.  A part waits for
// the next one to be planned only up to kPairTiles tiles (16: 75.8 us for 74.8 at
// 16 x 1 over 2000, 73.6 without pairs), and never at a share's end.
struct Part {
    int q0, base, keys, g0;  // the sequence's first token row, position of new token 0, keys; first row
    int rows, t0, n, ends;   // rows = 0: no part follows; ends: 1 the item begins in this part, 2 it ends in it, 4 one of a pair
    int tile_k, tile_v, h;   // scratch tiles of key tile t0, head of the round
    __device__ __forceinline__ bool thin() const { return rows <= 128; }
    __device__ __forceinline__ bool pair() const { return ends & 4; }
    __device__ __forceinline__ bool split() const { return thin() && !pair(); }                  // its tiles on both engines
    __device__ __forceinline__ int row0(int i) const { return thin() ? 0 : 128 * i; }  // of engine i's tile
    __device__ __forceinline__ int tiles(int i) const { return split() ? (n + 1 - i) >> 1 : n; }
};

// a / b, not negative: in 32 bits where both fit (a 64-bit division costs 500
// cycles, and the first part waits for four of them).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The planning warp: works out the shares and hands this CTA's parts on.
__device__ void plan_parts(const AttnArgs& A, uint8_t* smem, uint32_t bar_part, uint32_t bar_taken, volatile uint32_t* dead, int lane)
{
    const Plan P{smem};
    const int batch = A.p.batch, group = A.group, window = A.w.window;
    int tiles = 0;
    long long total = 0;
    for (int b0 = 0; b0 < batch; b0 += 32) {
        const int b = b0 + lane;
        Seq s{0, 0, 0, 0};
        if (b < batch) s = seq_of(A.p, A.w, b);
        int first, count;
        seq_tiles(s, window, first, count);
        const int nq = (s.q * group + kRows - 1) / kRows;  // items of a head
        long long u = 0;
        if (nq == 1) {
            const Span r = span_of(s, group, window, 0);
            u = max(1, r.n) * tile_cost(r);
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, nq > 1); m; m &= m - 1) {  // longer ones, the warp together
            const int from = __ffs(m) - 1, n = __shfl_sync(0xffffffffu, nq, from);
            const Seq z{0, __shfl_sync(0xffffffffu, s.q, from), __shfl_sync(0xffffffffu, s.base, from),
                        __shfl_sync(0xffffffffu, s.keys, from)};
            long long w = 0;
            for (int qt = lane; qt < n; qt += 32) {
                const Span r = span_of(z, group, window, qt);
                w += max(1, r.n) * tile_cost(r);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
            if (lane == from) u = w;
        }
        u *= A.hn;
        int ct = count;
        long long cu = u;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, ct, d);
            const long long v = __shfl_up_sync(0xffffffffu, cu, d);
            if (lane >= d) {
                ct += t;
                cu += v;
            }
        }
        if (b < batch) {
            P.seqs()[b] = make_int4(s.q0, s.q, s.base, s.keys);
            P.units()[b] = total + cu - u;
            P.tile()[b] = tiles + ct - count - first;
        }
        tiles += __shfl_sync(0xffffffffu, ct, 31);
        total += __shfl_sync(0xffffffffu, cu, 31);
    }
    if (lane == 0) P.units()[batch] = total;
    __syncwarp();

    // shares of two units at least: each holds a tile's last
    const long long shares = min((long long)gridDim.x, max(1ll, total / 2));
    int4 cut = make_int4(0, -1, 0, 0);
    uint32_t slot = 0;
    bool ok = true;
    // A part that was planned and not handed on yet: the next one may go with it.
    int4 last[3]{make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
    bool waits = false;
    // Hands on `x`, before it the part that waits (with x, if they are a pair), or
    // lets x wait.  Out of line: the instructions of a call are fetched anew.
    auto hand = [&](const int4 (&x)[3], bool pair, bool wait) {
#pragma unroll 1
        for (int k = waits ? 0 : 1; k < (pair || wait ? 1 : 2); ++k) {
            const uint32_t i = slot % kParts, use = slot / kParts;
            // (as long as the softmax works on the parts ahead, so with a limit of its
            // own; it ends as well once any other wait of the CTA has given up)
            if (use > 0 && ok) ok = mbar_wait(bar_taken + 8 * i, (use - 1) & 1, dead, A.flag, 1u << 30);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane < 3) {
                int4* d = reinterpret_cast<int4*>(smem + kOffParts + kPartBytes * i);
                int4 v = lane == 0 ? last[0] : lane == 1 ? last[1] : last[2], w = lane == 0 ? x[0] : lane == 1 ? x[1] : x[2];
                if (k) v = w;
                if (lane == 1 && pair) {
                    v.w |= 4;
                    w.w |= 4;
                }
                d[lane] = v;
                if (pair) d[3 + lane] = w;
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(bar_part + 8 * i);
            ++slot;
        }
        waits = wait;
#pragma unroll
        for (int k = 0; k < 3; ++k) last[k] = x[k];
    };
    if (total > 0 && blockIdx.x < shares) {
        const long long u0 = quotient(total * blockIdx.x, shares), stop = quotient(total * (blockIdx.x + 1), shares);
        int b = 0, top = batch - 1;  // the sequence of unit u0: the last that begins at or before it
        while (b < top) {
            const int mid = (b + top + 1) >> 1;
            if (P.units()[mid] <= u0)
                b = mid;
            else
                top = mid - 1;
        }
        Seq s = P.seq(b);
        long long rem = u0 - P.units()[b];
        const long long per_head = quotient(P.units()[b + 1] - P.units()[b], A.hn);
        int h = (int)quotient(rem, per_head), qt = 0;
        rem -= h * per_head;
        const int n = (s.q * group + kRows - 1) / kRows;
        for (int q = 0; q < n; q += 32) {  // the item: 32 at a time
            Span r{0, 0, 0};
            if (q + lane < n) r = span_of(s, group, window, q + lane);
            const long long x = q + lane < n ? max(1, r.n) * tile_cost(r) : 0;
            long long sum = x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += t;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, sum > rem);
            if (m) {
                qt = q + __ffs(m) - 1;
                rem -= __shfl_sync(0xffffffffu, sum - x, __ffs(m) - 1);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, sum, 31);
        }
        long long item = u0 - rem;  // its first unit
        int skip = -1;              // its tiles before the share: from `rem`, once its cost is known
        while (item < stop && ok) {
            while (qt * kRows >= s.q * group) {  // the rows are done: the next head, or the next sequence with rows
                qt = 0;
                if (s.q > 0 && ++h < A.hn) break;
                h = 0;
                s = P.seq(++b);
            }
            const Span r = span_of(s, group, window, qt);
            const int units = max(1, r.n), cost = tile_cost(r);
            if (skip < 0) skip = (int)rem / cost;
            const int until = (int)min((long long)units, (stop - item) >> (cost - 1));  // cost 1 or 2
            if (until <= skip) break;
            const int begins = skip == 0, ends = until == units;
            const int tile = h * tiles + P.tile()[b] + r.t0 + skip;
            int4 part[3]{make_int4(s.q0, s.base, s.keys, qt * kRows),
                         make_int4(r.rows, r.t0 + skip, min(until, r.n) - skip, begins | ends << 1),
                         make_int4(tile, tile + A.hn * tiles, h, 0)};
            const int n0 = last[1].z, n1 = part[1].z;
            const bool pair = waits && r.rows <= 128 && n1 > 0 && (n0 == n1 || n0 == n1 + 1);
            hand(part, pair, !pair && r.rows <= 128 && n1 > 0 && n1 <= kPairTiles && item + (long long)units * cost < stop);
            if (begins && !ends)
                cut = make_int4(s.q0, h, qt * kRows, (int)quotient((item + (long long)units * cost) * shares - 1, total) | r.rows << 16);
            item += (long long)units * cost;
            skip = 0;
            ++qt;
        }
    }
    const int4 end[3]{make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
    hand(end, false, false);
    launch_dependents();  // no earlier: the joining CTAs would sit on the SMs meanwhile
    if (lane == 0) A.part_item[blockIdx.x] = cut;
}

__global__ void __launch_bounds__(kAttnThreads, 1) paged_attention_kernel(const __grid_constant__ AttnArgs A)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023u)) % 1024;
    const uint32_t bars = smem_u32(smem + kOffBars);
    const uint32_t bar_full = bars, bar_empty = bar_full + 8 * kStages;            // ring tiles: landed, free
    const uint32_t bar_part = bar_empty + 8 * kStages, bar_taken = bar_part + 8 * kParts;
    const uint32_t bar_q = bar_taken + 8 * kParts, bar_s = bar_q + 16, bar_p = bar_s + 16;  // [engine]; weights: [piece][engine]
    const uint32_t bar_o = bar_p + 32, bar_x = bar_o + 16, bar_end = bar_x + 16;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffBars + kBars * 8);
    volatile uint32_t* dead = s_tmem + 1;
    float* s_ml = reinterpret_cast<float*>(smem + kOffMl);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int window = A.w.window;

    if (tid < kBars) {  // arrivals: softmax rows, the softmax warps with products and copies, or one
        const uint32_t bar = bars + 8 * tid;
        const bool rows = (bar >= bar_q && bar < bar_s) || (bar >= bar_p && bar < bar_o) || (bar >= bar_x && bar < bar_end);
        mbar_init(bar, rows ? 128 : bar >= bar_taken && bar < bar_q ? 10 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) *dead = 0u;
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    bool ok = true;
    uint32_t taken = 0;
    auto read = [&](uint32_t i, int which) -> Part {
        const int4* d = reinterpret_cast<const int4*>(smem + kOffParts + kPartBytes * i) + 3 * which;
        const int4 a = d[0], b = d[1], c = d[2];
        return Part{a.x, a.y, a.z, a.w, ok ? b.x : 0, b.y, b.z, b.w, c.x, c.y, c.z};
    };
    // The next part, of a pair that of engine `engine`; rows = 0 after the last, or if
    // the CTA gave up.
    auto take = [&](int engine) -> Part {
        const uint32_t i = taken % kParts;
        if (ok) ok = mbar_wait(bar_part + 8 * i, (taken / kParts) & 1, dead, A.flag);
        ++taken;
        Part x = read(i, 0);
        if (engine && x.pair()) x = read(i, 1);
        return x;
    };
    auto other = [&]() -> Part { return read((taken - 1) % kParts, 1); };  // the pair's second, before it is given back
    auto give_back = [&]() { mbar_arrive(bar_taken + 8 * ((taken - 1) % kParts)); };  // one lane, once the part is in registers

    // The ring's tiles, in the order in which the products take them: wide parts
    // K_0 V_0 K_1 V_1 .., thin ones K_0 K_1 V_0 K_2 V_1 K_3 ..
    if (warp == 10) {
        plan_parts(A, smem, bar_part, bar_taken, dead, lane);
    } else if (warp == 9) {
        if (lane == 0) {
            // ---- copies
            uint32_t n = 0;
            after_previous();  // the tiles are decoded
            for (;;) {
                const Part x = take(0);
                Part y{};
                if (x.rows && x.pair()) y = other();
                give_back();
                if (!x.rows) break;
                int k = 0, v = 0;
                const int tiles = x.n + y.n;
                while (k + v < 2 * tiles) {
                    const bool key = k < min(tiles, v + (x.thin() ? 2 : 1));
                    const int at = key ? k++ : v++;
                    const Part& z = x.pair() && (at & 1) ? y : x;
                    const int64_t tile = (key ? z.tile_k : z.tile_v) + (x.pair() ? at >> 1 : at);
                    const uint32_t st = n % kStages, use = n / kStages;
                    if (use > 0 && ok) ok = mbar_wait(bar_empty + 8 * st, (use - 1) & 1, dead, A.flag);
                    if (!ok) break;
                    mbar_expect(bar_full + 8 * st, kTileBytes);
                    bulk_copy(smem_u32(smem + kOffRing) + st * kTileBytes, A.scratch + tile * kTileBytes, kTileBytes, bar_full + 8 * st);
                    ++n;
                }
            }
            // every copy has landed before the CTA ends (they have, unless it gave up)
            for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k) {
                uint32_t zero = 0u;
                mbar_wait(bar_full + 8 * (k % kStages), (k / kStages) & 1, &zero, nullptr);
            }
        }
    } else if (warp == 8) {
        // ---- products (the whole warp)
        const uint32_t leader = elect_one();
        const uint32_t ring = smem_u32(smem + kOffRing), qs = smem_u32(smem);
        const uint32_t idesc = kIdescQK | (A.scale < 0.0f ? kNegateA : 0u);
        uint32_t at = 0, np = 0, nq = 0;  // ring tiles taken; weights and queries waited for, a bit an engine (the parity)
        // The lanes agree on `ok` once a part.  Until then a wait that gave up (the
        // CTA's other waits then end at once) only spoils results that nobody
        // writes; a vote at each wait cost every step 500 cycles.
        auto wait = [&](uint32_t bar, uint32_t parity) { ok = mbar_wait(bar, parity & 1, dead, A.flag) && ok; };
        auto full = [&](uint32_t k) { wait(bar_full + 8 * (k % kStages), k / kStages); };  // ring tile k has landed
        for (;;) {
            const Part x = take(0);
            int n = x.n;
            if (x.rows && x.pair()) n += other().n;
            ok = __all_sync(0xffffffffu, ok);
            if (lane == 0) give_back();
            if (!x.rows || !ok) break;
            if (n == 0) continue;
            const bool thin = x.thin();
            const int steps = thin ? n : 2 * n;
            uint32_t v = 0, k = 0;  // ring tiles in use
            // step e: O_i += P_i times its values, then S_i of its engine's next keys (from step -2 on: S alone)
#pragma unroll 1
            for (int e = -2; e < steps; ++e) {
                const int i = e & 1;
                const bool fresh = thin || i == 0, last = thin || i == 1;  // of the engines that share the tiles
                const bool more = (thin ? e + 2 : (e >> 1) + 1) < n;
                if (fresh) {
                    if (e >= 0) full(v = at++);
                    if (more) full(k = at++);
                }
                if (e >= 0) {
                    const uint64_t b = sw128_desc(ring + (v % kStages) * kTileBytes);
#pragma unroll
                    for (int piece = 0; piece < 2; ++piece) {  // the weights of 96 keys, then of the last 32
                        wait(bar_p + 16 * piece + 8 * i, np >> i);
                        tc_fence_after();
#pragma unroll
                        for (int t = 6 * piece; t < 6 + 2 * piece; ++t)
                            mma_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * t, b + (uint64_t)(t * 2048 >> 4), (e > 1 || t > 0) ? 1u : 0u, leader);
                    }
                    np ^= 1u << i;
                    mma_commit(bar_o + 8 * i, leader);
                    if (last) mma_commit(bar_empty + 8 * (v % kStages), leader);
                }
                if (more) {
                    if (e < 0) {
                        wait(bar_q + 8 * i, nq >> i);
                        nq ^= 1u << i;
                    }
                    const uint64_t a = sw128_desc(qs + i * kTileBytes), b = sw128_desc(ring + (k % kStages) * kTileBytes);
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const uint64_t o = (uint64_t)(((t >> 2) * (kTileBytes / 2) + (t & 3) * 32) >> 4);
                        mma_ss(tmem + 128 * i, a + o, b + o, idesc, t > 0, leader);
                    }
                    mma_commit(bar_s + 8 * i, leader);
                    if (last) mma_commit(bar_empty + 8 * (k % kStages), leader);
                }
            }
        }
        // every product issued is done before the tensor memory is freed
        uint32_t zero = 0u;
        mma_commit(bar_end, leader);
        mbar_wait(bar_end, 0u, &zero, nullptr);
    } else {
        // ---- softmax: a thread a row of engine i
        const int i = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * i, to = tmem + lanes + 256 + 128 * i;
        const float c = fmaxf(fabsf(A.scale) * 1.44269504f, 1e-30f);  // 0: weights of 1, and masked scores stay -inf
        const uint64_t c2 = pair(c, c);
        uint32_t ns = 0, no = 0, nx = 0;
        Part x{};
        float m = -INFINITY, l = 0.0f;  // the row's maximum and sum, over the part so far
        auto wait = [&](uint32_t bar, uint32_t count) {  // the whole warp: tensor-memory instructions follow
            if (ok) ok = mbar_wait(bar, count & 1, dead, A.flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        // one pass more than parts: Q of the next part is loaded, and its first
        // products can start, before this one's output is written
        for (bool have = false;; have = true) {
            Part y = take(i);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) y.rows = 0;
            if (lane == 0) give_back();
            if (y.rows && y.tiles(i) > 0) {  // this thread's row of Q, zeros behind the item's rows (the scores that read the last Q are done)
                const int r = y.row0(i) + row, g = y.g0 + r, tok = g / A.group;
                const uint32_t live = r < y.rows ? 16u : 0u;
                const uint16_t* src = A.q;
                if (live) src += (int64_t)(y.q0 + tok) * A.q_token + (int64_t)((A.h0 + y.h) * A.group + g - tok * A.group) * A.q_head;
                const uint32_t dst = smem_u32(smem) + i * kTileBytes + row * 128;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     dst + (k >> 3) * (kTileBytes / 2) + (((k & 7) ^ (row & 7)) << 4)),
                                 "l"(src + 8 * k), "r"(live)
                                 : "memory");
                asm volatile("cp.async.wait_all;" ::: "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(bar_q + 8 * i);
            }
            if (have) {
                // ---- part x is done: its rows of the output, or of the part's slot
                const int r = x.row0(i) + row, g = x.g0 + r, n = x.tiles(i), tok = g / A.group;
                const bool both = x.split() && x.n > 1;  // a thin part on both engines
                const bool real = r < x.rows, idle = x.row0(i) + (warp & 3) * 32 >= x.rows;
                if (n > 0) wait(bar_o + 8 * i, no - 1);
                if (both && i == 1) {  // O_1 stays in tensor memory until engine 0 has read it
                    s_ml[row] = m;
                    s_ml[128 + row] = l;
                    tc_fence_before();
                    mbar_arrive(bar_x);
                    ++nx;
                } else if (i == 0 || !x.split()) {
                    float f0 = 1.0f, f1 = 0.0f;
                    if (both) {
                        wait(bar_x, nx++);
                        const float m1 = s_ml[row], l1 = s_ml[128 + row], mn = fmaxf(m, m1);
                        f0 = m == -INFINITY ? 0.0f : ex2((m - mn) * c);
                        f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - mn) * c);
                        l = l * f0 + l1 * f1;
                        m = mn;
                    }
                    const bool whole = (x.ends & 3) == 3;
                    const int64_t slot = 2 * (int64_t)blockIdx.x + (x.ends & 1);
                    const int qh = (A.h0 + x.h) * A.group + g - tok * A.group;
                    const int64_t at = (int64_t)x.q0 + tok;
                    if (whole) {
                        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                        f0 *= inv;
                        f1 *= inv;
                    }
                    if (!idle) {
                        uint4* out = reinterpret_cast<uint4*>(A.out + at * A.out_token + (int64_t)qh * A.out_head);
                        uint4* part = reinterpret_cast<uint4*>(A.part_o) + slot * 32 * A.slot_rows + r;
#pragma unroll 1
                        for (int k = 0; k < 128; k += 16) {
                            uint32_t o[16], o1[16];
                            __syncwarp();
                            if (n > 0) tmem_ld16(to + k, o);
                            if (both) tmem_ld16(to + 128 + k, o1);
                            tmem_wait_ld();
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                const float e = n > 0 ? __uint_as_float(o[t]) * f0 : 0.0f;  // n = 0: the row sees no key
                                o[t] = __float_as_uint(both ? fmaf(__uint_as_float(o1[t]), f1, e) : e);
                            }
                            if (ok && real) {
                                if (whole) {
#pragma unroll
                                    for (int t = 0; t < 8; ++t)
                                        o[t] = pack_bf16x2(__uint_as_float(o[2 * t]), __uint_as_float(o[2 * t + 1]));
                                    out[k / 8] = make_uint4(o[0], o[1], o[2], o[3]);
                                    out[k / 8 + 1] = make_uint4(o[4], o[5], o[6], o[7]);
                                } else {
#pragma unroll
                                    for (int t = 0; t < 4; ++t)
                                        part[(int64_t)(k / 4 + t) * A.slot_rows] = make_uint4(o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]);
                                }
                            }
                        }
                        if (ok && real) {
                            if (whole) {
                                if (A.lse)
                                    A.lse[at * A.p.kv_heads * A.group + qh] = l == 0.0f ? -INFINITY : fmaf(m, c * 0.69314718f, logf(l));
                            } else {
                                A.part_ml[(slot * 2) * A.slot_rows + r] = m == -INFINITY ? -INFINITY : m * c;
                                A.part_ml[(slot * 2 + 1) * A.slot_rows + r] = l;
                            }
                        }
                        __syncwarp();
                    }
                    tc_fence_before();  // O is read before the next part's first product is allowed in
                    if (both) mbar_arrive(bar_x + 8);
                }
            }
            if (!y.rows) break;
            x = y;
            const int r = x.row0(i) + row, n = x.tiles(i), step = x.split() ? 2 : 1;
            const Seq s{x.q0, 0, x.base, x.keys};
            const bool real = r < x.rows, idle = x.row0(i) + (warp & 3) * 32 >= x.rows;  // idle: no row of this warp is one
            const int tok = real ? (x.g0 + r) / A.group : 0;
            int klo, khi;  // keys that this row sees
            visible(s, window, tok, tok, klo, khi);
            if (!real) klo = khi = 0;
            // and those that every row of this tile sees: no mask for key tiles inside them
            const int r0 = x.g0 + x.row0(i), r1 = min(r0 + 127, x.g0 + x.rows - 1);
            const int ahi = min(s.keys, s.base + r0 / A.group + 1);
            const int alo = window > 0 ? max(0, s.base + r1 / A.group - window + 1) : 0;
            m = -INFINITY;
            l = 0.0f;
            for (int j = 0; j < n; ++j) {
                const int k0 = (x.t0 + (x.split() ? i : 0) + j * step) * kTile;
                wait(bar_s + 8 * i, ns++);
                if (j == 0 && i == 1 && nx > 0) wait(bar_x + 8, nx - 1);  // engine 0 has read the last thin part's O_1
                if (idle) {  // its lanes of P are whatever they are: rows do not mix
                    tc_fence_before();
                    mbar_arrive(bar_p + 8 * i);
                    mbar_arrive(bar_p + 16 + 8 * i);
                    ++no;
                    continue;
                }
                if (k0 < alo || k0 + kTile > ahi) {
                    // keys that the row does not see: -infinity, written back, so that the
                    // few such tiles share the code below.  16 columns at a time: left
                    // alone where every row sees them, not read where none does.
                    const int lo = klo - k0, hi = khi - k0;
#pragma unroll 1
                    for (int k = 0; k < 128; k += 16) {
                        if (__all_sync(0xffffffffu, lo <= k && k + 16 <= hi)) continue;
                        uint32_t o[16];
                        if (__all_sync(0xffffffffu, k >= hi || k + 16 <= lo)) {
#pragma unroll
                            for (int t = 0; t < 16; ++t) o[t] = 0xff800000u;
                            tmem_st16(ts + k, o);
                            continue;
                        }
                        tmem_ld16(ts + k, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            if (k + t < lo || k + t >= hi) o[t] = 0xff800000u;
                        tmem_st16(ts + k, o);
                    }
                    tmem_wait_st();
                }
                // Two passes over the scores, 64 columns at a time in loops that stay
                // loops: every SM fetches the step's instructions anew in every call
                // (8 x 1 over up to 4096, this kernel, when it was chosen: 34 us, and
                // 41 in one pass over 128 registers with the masked tiles in a copy of
                // their own).  4096 over 16384: 32 columns at a time take 5% longer;
                // one pass with registers moved between the warpgroups took 4% less
                // (864 us for 897), but 1 over 650 14% more, which has since had a
                // kernel of its own: that variant is open.
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int k = 0; k < 128; k += 64) {
                    uint32_t v[64];
                    tmem_ld32(ts + k, v);
                    tmem_ld32(ts + k + 32, v + 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int t = 0; t < 64; t += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top[e] = fmaxf(top[e], fmaxf(__uint_as_float(v[t + e]), __uint_as_float(v[t + e + 4])));
                }
                const float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                if (j == 0) {
                    m = mt;
                } else if (__any_sync(0xffffffffu, (mt - m) * c > 8.0f)) {
                    const float mn = fmaxf(m, mt), f = mn == -INFINITY ? 1.0f : ex2((m - mn) * c);
                    m = mn;
                    l *= f;
                    wait(bar_o + 8 * i, no - 1);
#pragma unroll 1
                    for (int k = 0; k < 128; k += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + k, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
                        tmem_st16(to + k, o);
                    }
                }
                const float mc = m == -INFINITY ? 0.0f : -m * c;
                const uint64_t mc2 = pair(mc, mc);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 2
                for (int k = 0; k < 4; ++k) {  // weights over scores already read
                    uint32_t v[32], w[16];
                    tmem_ld32(ts + 32 * k, v);
                    tmem_wait_ld();
                    weights(v, c2, mc2, w, sum);
                    tmem_st16(ts + 16 * k, w);
                    if (k >= 2) {  // the first 96 keys' weights, then the last 32
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(bar_p + 16 * (k - 2) + 8 * i);
                    }
                }
                ++no;
                float a, b;
                unpair(add2(sum[0], sum[1]), a, b);
                l += a + b;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the parts of the items that were cut, in a fixed order: block (c, piece)
// the item that CTA c began and left unfinished.  A thread joins 4 values of
// kJoinRows rows over every kJoinGroups-th part, their loads in flight together;
// a warp has 8 rows by 4 such pieces at a time, which is 128 bytes of every
// part's columns and a whole 32-byte sector of every output row.
// Many parts are a chain of loads, so four groups share them where there are
// many (16 or 32 shares an item) or the blocks few.  Whole calls, us, in one
// group and in four: 1 new over 131072 keys of one head 102 and 65, 64 new over
// 60000 of one head 112 and 69, 16 new over 8000 of 8 heads 43.7 and 40.0; but
// 32 new over 8000 45.8 and 46.7, 512 new over 4096 64.8 and 79.5: many large
// blocks, and two or three parts an item.
struct Joined {  // of one row: maximum, sum, 4 values
    float m, l;
    float4 o;
    __device__ __forceinline__ void add(float mc, float lc, const float4& v)
    {
        const float mn = fmaxf(m, mc), f = m == -INFINITY ? 0.0f : exp2f(m - mn), g = mc == -INFINITY ? 0.0f : exp2f(mc - mn);
        m = mn;
        l = l * f + lc * g;
        o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
    }
};

template <int kJoinRows, int kJoinGroups>
__global__ void __launch_bounds__(256 * kJoinGroups) paged_join_kernel(const __grid_constant__ AttnArgs A)
{
    constexpr int kOthers = kJoinGroups > 1 ? kJoinGroups - 1 : 1;
    __shared__ float4 s_o[kOthers][kJoinRows][kJoinGroups > 1 ? 256 : 1];
    __shared__ float2 s_ml[kOthers][kJoinRows][kJoinGroups > 1 ? 256 : 1];
    after_previous();
    const int4 it = A.part_item[blockIdx.x];
    const int rows = it.w >> 16, c0 = blockIdx.x, c1 = it.w & 0xffff, t = threadIdx.x & 255, group = threadIdx.x >> 8;
    if (it.y < 0 || (int)blockIdx.y * 8 * kJoinRows >= rows) return;
    const int r0 = blockIdx.y * 8 * kJoinRows + (t & 7), c4 = t >> 3;  // rows r0, r0 + 8, ..
    const int64_t step = 2 * (int64_t)A.slot_rows;  // from slot to slot of part_ml; part_o has 16 times as many float4
    const int64_t slot = 2 * ((int64_t)c0 + group) + (group == 0 ? 1 : 0);  // 2 c0 + 1, then 2 c of the others
    const float* ml = A.part_ml + slot * step + r0;
    const float4* po = reinterpret_cast<const float4*>(A.part_o) + slot * 16 * step + (int64_t)c4 * A.slot_rows + r0;
    Joined x[kJoinRows];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) x[k] = Joined{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll 2
    for (int c = c0 + group; c <= c1; c += kJoinGroups) {
        float mc[kJoinRows], lc[kJoinRows];
        float4 v[kJoinRows];
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k)
            if (r0 + 8 * k < rows) {
                mc[k] = ml[8 * k];
                lc[k] = ml[A.slot_rows + 8 * k];
                v[k] = po[8 * k];
            }
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k)
            if (r0 + 8 * k < rows) x[k].add(mc[k], lc[k], v[k]);
        ml += (2 * kJoinGroups - (c == c0 ? 1 : 0)) * step;
        po += (2 * kJoinGroups - (c == c0 ? 1 : 0)) * 16 * step;
    }
    if constexpr (kJoinGroups > 1) {
        if (group > 0)
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                s_o[group - 1][k][t] = x[k].o;
                s_ml[group - 1][k][t] = make_float2(x[k].m, x[k].l);
            }
        __syncthreads();
        if (group > 0) return;
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k)
        if (r0 + 8 * k < rows) {
            if constexpr (kJoinGroups > 1)
                for (int g = 1; g < kJoinGroups && c0 + g <= c1; ++g) x[k].add(s_ml[g - 1][k][t].x, s_ml[g - 1][k][t].y, s_o[g - 1][k][t]);
            const float inv = x[k].l == 0.0f ? 0.0f : 1.0f / x[k].l;
            const int g = it.z + r0 + 8 * k, tok = g / A.group, qh = (A.h0 + it.y) * A.group + g - tok * A.group;
            const int64_t row = (int64_t)it.x + tok;
            uint2 w;
            w.x = pack_bf16x2(x[k].o.x * inv, x[k].o.y * inv);
            w.y = pack_bf16x2(x[k].o.z * inv, x[k].o.w * inv);
            *reinterpret_cast<uint2*>(A.out + row * A.out_token + (int64_t)qh * A.out_head + 4 * c4) = w;
            if (A.lse && c4 == 0)
                A.lse[row * A.p.kv_heads * A.group + qh] = x[k].l == 0.0f ? -INFINITY : (x[k].m + log2f(x[k].l)) * 0.69314718f;
        }
}

// ------------------------------------------------------------ few rows over few keys
// One kernel for calls whose (sequence, KV head, key tile) triples all fit the
// GPU at once, with at most 32 rows an item: a CTA decodes one tile of keys and
// values straight into its shared memory, both tables with it, and computes its
// part of the item.  An item's CTAs are a cluster and join their parts through
// its shared memory, where an item has at most 8 tiles and 8 rows and the
// clusters all run at once (16 clusters of 8 did not: 29.5 us for 15.5);
// otherwise the joining kernel does it.  By cluster and by the kernel, 4 query
// heads over 650 keys: 1 new 13.7 and 15.0, 2 14.5 and 15.0, 4 15.9 and 15.1:
// remote loads are slow, 60 cycles each.
// One kernel, or one and the joining, against three with it, us a call: 8 KV
// heads, 1 new over 100 keys 12.2 and 23.5, over 650 13.8 and 22.3, over 2300
// (18 tiles) 16.6 and 22; 1 new over 7000 keys of 2 heads 20.5 and 27.8, over
// 18000 of one 27.7 and 30.6, 8 new 29.0 and 32.2.
// Of 11 us in the kernel the tables' landing takes 1.7, the walk 5, records,
// scores and weights 2, the join 2.
//
// Rows are TMEM lanes 0-31; the four warps that reach them (0, 4, 8, 12) weigh
// 32 keys each and write 32 columns of the output each.  The rest of Q's 128-row
// tile is whatever lies behind it in shared memory: rows of a product do not mix.
constexpr int kSmallThreads = 512, kSmallRows = 32;
constexpr size_t kSmallK = (size_t)kSmallRows * kG * 2, kSmallV = kSmallK + kTileBytes, kSmallLut = kSmallV + kTileBytes;
constexpr size_t kSmallCt = kSmallLut + 2 * kDecLut, kSmallWords = kSmallCt + 2 * kDecCt;
constexpr size_t kSmallExch = kSmallWords + (size_t)16 * 256 * 4;  // [2][4][32] maxima and sums
constexpr size_t kSmallMl = kSmallExch + 2 * 4 * 32 * sizeof(float);  // [2][32] the tile's
constexpr size_t kSmallBars = kSmallMl + 2 * 32 * sizeof(float);
constexpr int kSmallCluster = 8, kSmallClusterRows = 8;
constexpr size_t kSmallSmem = 1024 + kSmallBars + 32;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// What lies at this CTA's shared address `at` in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t at, uint32_t rank)
{
    float v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %1, %2;\n\t"
        "ld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(v)
        : "r"(at), "r"(rank)
        : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t at, uint32_t rank)
{
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(at), "r"(rank)
        : "memory");
    return v;
}

__global__ void __launch_bounds__(kSmallThreads, 1) paged_small_kernel(const __grid_constant__ AttnArgs A,
                                                                       const __grid_constant__ StageArgs D)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023u)) % 1024;
    const uint32_t bar_tables = smem_u32(smem + kSmallBars), bar_mma = bar_tables + 8;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kSmallBars + 16);
    volatile uint32_t* dead = s_tmem + 1;
    float* s_max = reinterpret_cast<float*>(smem + kSmallExch);
    float* s_sum = s_max + 4 * 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float4* s_o = reinterpret_cast<float4*>(smem + kSmallWords);  // [32 pieces of 4 values][32 rows], once the blocks are decoded
    float* s_ml = reinterpret_cast<float*>(smem + kSmallMl);
    uint32_t cluster;  // CTAs of the item, if they join their parts themselves; 1: a whole item, or left to the joining kernel
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cluster));
    const int tile = blockIdx.x, h = blockIdx.y, b = blockIdx.z, cta = (b * gridDim.y + h) * gridDim.x + tile;
    launch_dependents();
    if (tid == 0) {
        mbar_init(bar_tables, 1);
        mbar_init(bar_mma, 1);
        *dead = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_expect(bar_tables, (uint32_t)(2 * (kDecLut + kDecCt)));
        for (int kv = 0; kv < 2; ++kv) {
            bulk_copy(smem_u32(smem + kSmallLut + kv * kDecLut), &D.tb[kv]->lut[0][0], (uint32_t)kDecLut, bar_tables);
            bulk_copy(smem_u32(smem + kSmallCt + kv * kDecCt), &D.tb[kv]->Ct[0][0], (uint32_t)kDecCt, bar_tables);
        }
    }
    if (warp == 15) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(256u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const Seq s = seq_of(A.p, A.w, b);
    const int window = A.w.window, rows = s.q * A.group;
    int first, count;
    seq_tiles(s, window, first, count);
    const bool live = tile < count, none = count == 0 && tile == 0 && rows > 0;  // none: rows that see no key
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    bool ok = true;  // of a thread, then of the CTA, then of a warp

    if (live) {
        if (warp < 8) {  // ---- decode: thread = a row of the key tile, then of the value tile
            const int kv = tid >> 7, row = tid & 127, t = (first + tile) * kTile + row;
            uint4 q0 = make_uint4(0u, 0u, 0u, 0u), q1 = q0, q2 = q0, q3 = q0;
            const int64_t blk = t < s.keys ? paged_block(A.p, b, h, t) : -1;
            if (blk >= 0) {
                const uint8_t* src = D.pages[kv] + blk * ECCO_BLOCK_BYTES;
                q0 = ldg_nc_v4(src);
                q1 = ldg_nc_v4(src + 16);
                q2 = ldg_nc_v4(src + 32);
                q3 = ldg_nc_v4(src + 48);
            }
            uint32_t* ws = reinterpret_cast<uint32_t*>(smem + kSmallWords) + tid;
            const uint32_t code = q0.x & 0xffu;
            const bool null = scale_code_is_null(code);
            stage_words(ws, 256, q0, q1, q2, q3);
            const float sc = __fmul_rn(D.tb[kv]->S_t, e4m3_to_f32(code));
            ok = mbar_wait(bar_tables, 0u, dead, A.flag);
            ok = __all_sync(0xffffffffu, ok);
            const uint32_t lkey = lut_key(smem + kSmallLut + kv * kDecLut, (q0.x >> 8) & 255u);
            ValuePlanes vp = make_planes(sc, reinterpret_cast<const float*>(smem + kSmallCt + kv * kDecCt), (int)((q0.x >> 8) & 63u));
            if (null) {  // 128 times +0, whatever the stream says
#pragma unroll
                for (int k = 0; k < 4; ++k) vp.lo[k] = vp.hi[k] = 0u;
            }
            Stream st{q0.x, q0.y, kHdrBits, 2, kPayloadBits};
            uint8_t* dst = smem + (kv ? kSmallV : kSmallK) + row * 128;
            const uint32_t x = (uint32_t)row & 7u;
            const auto put = [&](uint32_t c, const uint32_t (&a)[4]) {
                *reinterpret_cast<uint4*>(dst + (c >> 3) * (kTileBytes / 2) + (((c & 7u) ^ x) << 4)) = make_uint4(a[0], a[1], a[2], a[3]);
            };
            // Two warps a scheduler: the walk's latency is what counts.  The next word
            // is there before it is needed, and the values of a chunk are worked out between
            // the lookups of the next one.
            uint32_t c = 0, a[4], nib = 0;
            for (; ok && c < kG / 8; ++c) {
                if (__any_sync(0xffffffffu, st.room < 64)) break;
                const uint32_t last = nib;
                int used = 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t next = st.widx < 16 ? ws[st.widx * 256] : 0u;
                    uint32_t cur = __funnelshift_r(st.lo, st.hi, st.b);
                    int u = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t e;
                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(lkey ^ (cur & 0xffu)));
                        const uint32_t len = e >> 4;
                        nib = __funnelshift_r(nib, e, 4);
                        cur >>= len;
                        u += (int)len;
                    }
                    st.b += u;
                    used += u;
                    if (st.b >= 32) {
                        st.lo = st.hi;
                        st.hi = next;
                        st.b -= 32;
                        ++st.widx;
                    }
                    if (half == 0) {
                        planes_to_bf16<0>(vp, last, last << 4, a[0], a[1]);
                        planes_to_bf16<1>(vp, last, last << 4, a[2], a[3]);
                        if (c > 0) put(c - 1, a);
                    }
                }
                st.room -= used;
            }
            if (c > 0) {
                planes_to_bf16<0>(vp, nib, nib << 4, a[0], a[1]);
                planes_to_bf16<1>(vp, nib, nib << 4, a[2], a[3]);
                put(c - 1, a);
            }
#pragma unroll 1
            for (; ok && c < kG / 8; ++c) {  // near the end of the block
                chunk_values(st, lkey, ws, 256, vp, a);
                put(c, a);
            }
            if (ok && !null && st.room >= 0) {  // unclipped: outlier records follow the codewords
                const int n = min(kMaxRec, st.room / kRecBits), at0 = kBlockBits - st.room;
                for (int k = 0; k < n; ++k) {
                    const uint32_t rec = read_record(ws, 256, at0 + k * kRecBits), e = rec & 127u;
                    const float o = q_over_127((int)(int8_t)(uint8_t)(rec >> 7));
                    *reinterpret_cast<uint16_t*>(dst + (e >> 6) * (kTileBytes / 2) + ((((e >> 3) & 7u) ^ x) << 4) + (e & 7u) * 2) =
                        (uint16_t)f32_to_bf16_bits(__fmul_rn(sc, o));
                }
            }
        } else if (warp == 8 && lane < rows) {  // ---- queries: lane = row
            const int tok = lane / A.group;
            const uint16_t* src = A.q + (int64_t)(s.q0 + tok) * A.q_token + (int64_t)(h * A.group + lane - tok * A.group) * A.q_head;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                *reinterpret_cast<uint4*>(smem + (k >> 3) * (kSmallRows * 128) + lane * 128 + (((k & 7) ^ (lane & 7)) << 4)) =
                    *reinterpret_cast<const uint4*>(src + 8 * k);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    ok = *dead == 0u;

    if (live && warp == 9) {  // ---- products
        const uint32_t leader = elect_one(), idesc = kIdescQK | (A.scale < 0.0f ? kNegateA : 0u);
        const uint64_t kd = sw128_desc(smem_u32(smem + kSmallK)), vd = sw128_desc(smem_u32(smem + kSmallV));
#pragma unroll
        for (int t = 0; t < 8; ++t)
            mma_ss(tmem, sw128_desc(smem_u32(smem) + (t >> 2) * (kSmallRows * 128) + (t & 3) * 32),
                   kd + (uint64_t)(((t >> 2) * (kTileBytes / 2) + (t & 3) * 32) >> 4), idesc, t > 0, leader);
        mma_commit(bar_mma, leader);
        asm volatile("bar.sync 2, 160;" ::: "memory");  // the weights are there
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < 8; ++t) mma_ts(tmem + 128, tmem + 8 * t, vd + (uint64_t)(t * 2048 >> 4), t > 0, leader);
        mma_commit(bar_mma, leader);
        uint32_t zero = 0u;  // every product is done before the tensor memory is freed
        mbar_wait(bar_mma, 1u, &zero, nullptr);
    } else if (live && (warp & 3) == 0) {  // ---- softmax: lane = row, this warp's keys 32 part .. of the tile
        const int part = warp >> 2, tok = min(lane, rows - 1) / A.group;
        const float c = fmaxf(fabsf(A.scale) * 1.44269504f, 1e-30f);
        auto wait = [&](uint32_t parity) {
            if (ok) ok = mbar_wait(bar_mma, parity, dead, A.flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        int klo, khi;
        visible(s, window, tok, tok, klo, khi);
        klo -= (first + tile) * kTile + 32 * part;
        khi -= (first + tile) * kTile + 32 * part;
        const uint32_t seen = (khi >= 32 ? ~0u : khi > 0 ? (1u << khi) - 1u : 0u) & (klo <= 0 ? ~0u : klo < 32 ? ~0u << klo : 0u);
        uint32_t v[32], w[16];
        wait(0u);
        tmem_ld32(tmem + 32 * part, v);
        tmem_wait_ld();
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            if (!(seen >> k & 1u)) v[k] = 0xff800000u;
            m = fmaxf(m, __uint_as_float(v[k]));
        }
        s_max[part * 32 + lane] = m;
        tc_fence_before();
        asm volatile("bar.sync 1, 128;" ::: "memory");  // every warp has its scores in registers
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, s_max[k * 32 + lane]);
        const float mc = m == -INFINITY ? 0.0f : -m * c;
        uint64_t sum[2] = {0ull, 0ull};
        weights(v, pair(c, c), pair(mc, mc), w, sum);
        float a, e;
        unpair(add2(sum[0], sum[1]), a, e);
        s_sum[part * 32 + lane] = a + e;
        tmem_st16(tmem + 16 * part, w);
        tmem_wait_st();
        tc_fence_before();
        asm volatile("bar.arrive 2, 160;" ::: "memory");
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const float l = (s_sum[lane] + s_sum[32 + lane]) + (s_sum[64 + lane] + s_sum[96 + lane]);
        wait(1u);
        tmem_ld32(tmem + 128 + 32 * part, v);
        tmem_wait_ld();
        if (cluster > 1) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s_o[(8 * part + k) * 32 + lane] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                              __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
            if (part == 0) {
                s_ml[lane] = m == -INFINITY ? -INFINITY : m * c;
                s_ml[32 + lane] = l;
            }
        } else if (ok && lane < rows) {
            const int qh = h * A.group + lane - tok * A.group;
            const int64_t at = (int64_t)s.q0 + tok;
            if (count == 1) {  // the whole item
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint4* out = reinterpret_cast<uint4*>(A.out + at * A.out_token + (int64_t)qh * A.out_head) + 4 * part;
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = pack_bf16x2(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
#pragma unroll
                for (int k = 0; k < 4; ++k) out[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                if (A.lse && part == 0)
                    A.lse[at * A.p.kv_heads * A.group + qh] = l == 0.0f ? -INFINITY : fmaf(m, c * 0.69314718f, logf(l));
            } else {
                const int64_t slot = 2 * (int64_t)cta + (tile == 0 ? 1 : 0);
                uint4* o = reinterpret_cast<uint4*>(A.part_o) + (slot * 32 + 8 * part) * A.slot_rows + lane;
#pragma unroll
                for (int k = 0; k < 8; ++k) o[(int64_t)k * A.slot_rows] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                if (part == 0) {
                    A.part_ml[slot * 2 * A.slot_rows + lane] = m == -INFINITY ? -INFINITY : m * c;
                    A.part_ml[(slot * 2 + 1) * A.slot_rows + lane] = l;
                }
            }
        }
        tc_fence_before();
    } else if (none && tid < rows * 16) {  // the first rows * 16 threads of the CTA: 16 bytes each
        const int r = tid >> 4, tok = r / A.group, qh = h * A.group + r - tok * A.group;
        const int64_t at = (int64_t)s.q0 + tok;
        reinterpret_cast<uint4*>(A.out + at * A.out_token + (int64_t)qh * A.out_head)[tid & 15] = make_uint4(0u, 0u, 0u, 0u);
        if (A.lse && (tid & 15) == 0) A.lse[at * A.p.kv_heads * A.group + qh] = -INFINITY;
    }
    if (cluster > 1) {  // ---- join: the first CTA, a thread 4 values of one of its rows (at most kSmallThreads / 32)
        cluster_arrive();
        cluster_wait();
        const int r = tid >> 5, c4 = tid & 31;
        if (ok && tile == 0 && count > 0 && r < rows) {
            const uint32_t at_ml = smem_u32(s_ml + r), at_o = smem_u32(s_o + c4 * 32 + r);
            float mc[kSmallCluster], lc[kSmallCluster], m = -INFINITY, l = 0.0f;
            float4 v[kSmallCluster], o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kSmallCluster; ++k)
                if (k < count) {
                    mc[k] = ld_cluster(at_ml, k);
                    lc[k] = ld_cluster(at_ml + 128, k);
                    v[k] = ld_cluster4(at_o, k);
                    m = fmaxf(m, mc[k]);
                }
#pragma unroll
            for (int k = 0; k < kSmallCluster; ++k)
                if (k < count) {
                    const float f = m == -INFINITY ? 0.0f : ex2(mc[k] - m);
                    l = fmaf(lc[k], f, l);
                    o = make_float4(fmaf(v[k].x, f, o.x), fmaf(v[k].y, f, o.y), fmaf(v[k].z, f, o.z), fmaf(v[k].w, f, o.w));
                }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int tok = r / A.group, qh = h * A.group + r - tok * A.group;
            const int64_t at = (int64_t)s.q0 + tok;
            uint2 w;
            w.x = pack_bf16x2(o.x * inv, o.y * inv);
            w.y = pack_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(A.out + at * A.out_token + (int64_t)qh * A.out_head + 4 * c4) = w;
            if (A.lse && c4 == 0)
                A.lse[at * A.p.kv_heads * A.group + qh] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
        }
        cluster_arrive();
        cluster_wait();  // the others have read this CTA's part
    }
    if (tid == 0) {
        if (cluster == 1) A.part_item[cta] = live && tile == 0 && count > 1 ? make_int4(s.q0, h, 0, (cta + count - 1) | rows << 16) : make_int4(0, -1, 0, 0);
        uint32_t zero = 0u;  // the copies have landed before the CTA ends (they have, where blocks were decoded)
        if (!live || !ok) mbar_wait(bar_tables, 0u, &zero, live ? nullptr : A.flag);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 15) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256u) : "memory");
}

// Scratch of one KV head.
int64_t head_bytes(int batch, int max_kv) { return 2 * (int64_t)batch * ((max_kv + kTile - 1) / kTile) * kTileBytes; }

// Waits, as the kernels above do but for some milliseconds, for a barrier at
// which nothing arrives.
__global__ void paged_wait_selftest_kernel(int* flag)
{
    __shared__ __align__(8) uint64_t s_bar;
    if (threadIdx.x == 0) {
        uint32_t dead = 0u;
        mbar_init(smem_u32(&s_bar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_wait(smem_u32(&s_bar), 0u, &dead, flag, kSpinLimit >> 6);
    }
}

// Heads of a round: as many as keep the scratch within kRoundBytes, at least one.
int round_heads(int batch, int kv_heads, int max_kv)
{
    const int64_t per_head = head_bytes(batch, max_kv);
    return (int)std::max<int64_t>(1, std::min<int64_t>(kv_heads, per_head ? kRoundBytes / per_head : kv_heads));
}

// Workspace: items cut [kMaxCtas], (max, sum) and O of the slots, the scratch.
struct Layout {
    size_t ml, o, scratch, bytes;
    int slot_rows;
};

Layout layout(int batch, int kv_heads, int group, int max_q, int max_kv)
{
    const auto up = [](size_t n) { return (n + 1023) / 1024 * 1024; };
    Layout L;
    L.slot_rows = (int)std::min<int64_t>(kRows, std::max<int64_t>(1, (int64_t)max_q * group));
    L.ml = up(kMaxCtas * sizeof(int4));
    L.o = L.ml + up((size_t)2 * kMaxCtas * 2 * L.slot_rows * sizeof(float));
    L.scratch = L.o + up((size_t)2 * kMaxCtas * 32 * L.slot_rows * sizeof(float4));
    // A round may leave part of kRoundBytes free, more or less of it as the bounds
    // grow.  It is asked for all the same: the size never shrinks when a bound grows.
    const int64_t per_head = head_bytes(batch, max_kv);
    L.bytes = L.scratch + (size_t)std::max(per_head, std::min(kv_heads * per_head, kRoundBytes)) + 1024;
    return L;
}

}  // namespace

size_t paged_attention_bytes(int batch, int kv_heads, int group, int max_q, int max_kv)
{
    return layout(batch, kv_heads, group, max_q, max_kv).bytes;
}

cudaError_t paged_timeouts(unsigned int* n) { return cudaMemcpyFromSymbol(n, g_timeouts, sizeof(*n)); }

cudaError_t launch_paged_wait_selftest(cudaStream_t s)
{
    paged_wait_selftest_kernel<<<1, 32, 0, s>>>(timeout_flag());
    return cudaGetLastError();
}

// Launches a kernel whose CTAs may start before the previous kernel has ended
// (it waits with after_previous).
static cudaError_t launch_after(void (*kernel)(AttnArgs), dim3 grid, int threads, size_t smem, cudaStream_t s, const AttnArgs& a)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, a);
}

static cudaLaunchAttribute cluster_of(int size)
{
    cudaLaunchAttribute c{};
    c.id = cudaLaunchAttributeClusterDimension;
    c.val.clusterDim.x = (unsigned)size;
    c.val.clusterDim.y = c.val.clusterDim.z = 1;
    return c;
}

static cudaLaunchConfig_t small_launch(dim3 grid, cudaLaunchAttribute* cluster, cudaStream_t s)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(kSmallThreads);
    c.dynamicSmemBytes = kSmallSmem;
    c.stream = s;
    c.attrs = cluster;
    c.numAttrs = 1;
    return c;
}

// Clusters of `size` CTAs of the small kernel that the current device runs at
// once (a cluster stays inside one of its processor groups); 0 if it can't say.
static int clusters_at_once(int size)
{
    static std::atomic<int> cached[kMaxDeviceBits][kSmallCluster + 1];  // + 1; 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool slot = dev >= 0 && dev < kMaxDeviceBits;
    int n = slot ? cached[dev][size].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n - 1;
    cudaLaunchAttribute item = cluster_of(size);
    const cudaLaunchConfig_t c = small_launch(dim3(size), &item, nullptr);
    if (cudaOccupancyMaxActiveClusters(&n, paged_small_kernel, &c) != cudaSuccess) {
        cudaGetLastError();  // not this call's
        n = 0;
    }
    if (slot) cached[dev][size].store(n + 1, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* workspace, cudaStream_t s)
{
    static std::atomic<uint64_t> configured[3]{};
    cudaError_t e = set_max_smem_once(configured[0], (const void*)paged_decode_kernel, kDecSmem);
    if (e == cudaSuccess) e = set_max_smem_once(configured[1], (const void*)paged_attention_kernel, kAttnSmem);
    if (e == cudaSuccess) e = set_max_smem_once(configured[2], (const void*)paged_small_kernel, kSmallSmem);
    if (e != cudaSuccess) return e;
    const Layout L = layout(a.p.batch, a.p.kv_heads, a.group, a.max_q, a.max_kv);
    uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 1023) / 1024 * 1024);
    uint8_t* scratch = ws + L.scratch;
    const int hn = round_heads(a.p.batch, a.p.kv_heads, a.max_kv);
    const int ctas = std::min(device_sm_count(), kMaxCtas);
    const Bounds w{a.tokens, a.max_q, a.max_kv, a.window};
    const bool wide = ((reinterpret_cast<uintptr_t>(a.pages[0]) | reinterpret_cast<uintptr_t>(a.pages[1])) & 31u) == 0;
    const auto stage = [&](int h0, int n) {
        return StageArgs{a.p, w, {a.tb[0], a.tb[1]}, {a.pages[0], a.pages[1]}, scratch, h0, n, wide, timeout_flag()};
    };
    const auto attn = [&](int h0, int n) {
        return AttnArgs{a.p, w, scratch, a.q, a.out, a.lse, a.q_token, a.q_head, a.out_token, a.out_head, a.group, h0, n,
                        a.scale, reinterpret_cast<float*>(ws + L.o), reinterpret_cast<float*>(ws + L.ml),
                        reinterpret_cast<int4*>(ws), L.slot_rows, timeout_flag()};
    };
    const auto join = [&](int n_ctas, const AttnArgs& at) {
        const int64_t items = (int64_t)a.p.batch * at.hn * (((int64_t)a.max_q * a.group + kRows - 1) / kRows);
        const bool few = L.slot_rows <= 32 || (L.slot_rows <= 64 && items * 16 <= ctas) || items * 32 <= ctas;
        return few ? launch_after(paged_join_kernel<1, 4>, dim3(n_ctas, (L.slot_rows + 7) / 8), 1024, 0, s, at)
                   : launch_after(paged_join_kernel<2, 1>, dim3(n_ctas, (L.slot_rows + 15) / 16), 256, 0, s, at);
    };
    // key tiles that an item can see
    int64_t seen = std::max(1, (a.max_kv + kTile - 1) / kTile);
    if (a.window > 0) seen = std::min<int64_t>(seen, ((int64_t)a.window + a.max_q - 2) / kTile + 2);
    const int64_t triples = seen * a.p.kv_heads * a.p.batch;
    if (L.slot_rows <= kSmallRows && triples <= ctas) {
        const AttnArgs at = attn(0, a.p.kv_heads);
        const bool together = seen == 1 || (seen <= kSmallCluster && L.slot_rows <= kSmallClusterRows &&
                                            clusters_at_once((int)seen) >= triples / seen);
        cudaLaunchAttribute item = cluster_of(together ? (int)seen : 1);
        const cudaLaunchConfig_t c = small_launch(dim3((unsigned)seen, a.p.kv_heads, a.p.batch), &item, s);
        if ((e = cudaLaunchKernelEx(&c, paged_small_kernel, at, stage(0, a.p.kv_heads))) != cudaSuccess) return e;
        return together ? cudaSuccess : join((int)triples, at);
    }
    for (int h0 = 0; h0 < a.p.kv_heads; h0 += hn) {
        const int n = std::min(hn, a.p.kv_heads - h0);
        // (the first kernel of a round waits for all before it: the workspace is free)
        paged_decode_kernel<<<std::max(2, device_sm_count() & ~1), kDecThreads, kDecSmem, s>>>(stage(h0, n));
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const AttnArgs at = attn(h0, n);
        if ((e = launch_after(paged_attention_kernel, dim3(ctas), kAttnThreads, kAttnSmem, s, at)) != cudaSuccess) return e;
        if ((e = join(ctas, at)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ecco
