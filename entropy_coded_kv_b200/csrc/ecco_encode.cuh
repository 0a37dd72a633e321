// The encoder of one group (shared by the encode kernels): 16 lanes per
// 128-value group, lane l owning values 8l..8l+7; 8 lanes per 64-value group.
// The steps and their cost are described in ecco_encode.cu.
#pragma once

#include "ecco_bucket.cuh"
#include "ecco_internal.cuh"

namespace ecco {
namespace {

constexpr int kRow = 97;      // words per pattern row: T[16] | lens4[16] | code[4][16] | pad
constexpr int kRowLens = 16;
constexpr int kRowCode = 32;

struct Counters {  // uniform within a half-warp
    uint32_t groups, zero, clipped, padded, records, nonfinite;
    unsigned long long bits;
};

__device__ __forceinline__ uint32_t hw_max(uint32_t m, uint32_t v) { return __reduce_max_sync(m, v); }
__device__ __forceinline__ uint32_t hw_min(uint32_t m, uint32_t v) { return __reduce_min_sync(m, v); }
__device__ __forceinline__ uint32_t hw_add(uint32_t m, uint32_t v) { return __reduce_add_sync(m, v); }

__device__ __forceinline__ float hw_minf(uint32_t m, float v)
{
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(m));
    return r;
}

__device__ __forceinline__ float hw_maxf(uint32_t m, float v)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(m));
    return r;
}

// key = |x| << 8 | (127 - i) << 1 | sign: the largest key is the first index
// of the largest magnitude, and it carries that element's sign.
__device__ __forceinline__ uint32_t keyof(uint32_t v, int i)
{
    return ((v & 0x7fffu) << 8) | ((uint32_t)(127 - i) << 1) | (v >> 15);
}

// Sorts 8 keys descending (Batcher's odd-even merge sort, 19 comparators).
__device__ __forceinline__ void sort8_desc(uint32_t (&k)[8])
{
#define ECCO_CMPX(a, b)                    \
    {                                      \
        const uint32_t hi = max(k[a], k[b]); \
        k[b] = min(k[a], k[b]);            \
        k[a] = hi;                         \
    }
    ECCO_CMPX(0, 1) ECCO_CMPX(2, 3) ECCO_CMPX(4, 5) ECCO_CMPX(6, 7)
    ECCO_CMPX(0, 2) ECCO_CMPX(1, 3) ECCO_CMPX(4, 6) ECCO_CMPX(5, 7)
    ECCO_CMPX(1, 2) ECCO_CMPX(5, 6)
    ECCO_CMPX(0, 4) ECCO_CMPX(1, 5) ECCO_CMPX(2, 6) ECCO_CMPX(3, 7)
    ECCO_CMPX(2, 4) ECCO_CMPX(3, 5)
    ECCO_CMPX(1, 2) ECCO_CMPX(3, 4) ECCO_CMPX(5, 6)
#undef ECCO_CMPX
}

// 32-bit shared-window address of a word of the pattern rows.
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// sym = number of thresholds T[0..13] of the row at shared address `R`
// strictly below v (R9), by the bucket map: L = the pattern's 256 counts
// (256-byte aligned), qm = its (a, b).  Thresholds in buckets below v's are
// below v, those in buckets above are not, and the one threshold that may
// share v's bucket is T[lo] (the thresholds are non-decreasing), so sym =
// lo + (T[lo] < v); T[14] = +inf.
__device__ __forceinline__ int quantise_bucket(uint32_t R, uint32_t L, float4 qm, float v)
{
    const uint32_t lo = lds_u8(L | threshold_bucket(v, qm.x, qm.y));
    return (int)lo + ((__uint_as_float(lds_u32(R + 4u * lo)) < v) ? 1 : 0);
}

// The same count by bisection (patterns with two thresholds in one bucket):
// T[7] is in a register, the other three levels read T[idx + 3], T[idx + 1],
// T[idx].
__device__ __forceinline__ int quantise(uint32_t R, float t7, float v)
{
    int idx = (t7 < v) ? 8 : 0;
    idx += (__uint_as_float(lds_u32(R + 4u * (uint32_t)idx + 12u)) < v) ? 4 : 0;
    idx += (__uint_as_float(lds_u32(R + 4u * (uint32_t)idx + 4u)) < v) ? 2 : 0;
    idx += (__uint_as_float(lds_u32(R + 4u * (uint32_t)idx)) < v) ? 1 : 0;
    return idx;
}

// The min / max rule's pattern (R8): this lane evaluates patterns hl + kLanes k
// (those below npat).  e >= +0, so bit order is value order; a pattern past
// npat gets 0xffffffff, above every error including +inf, so a group whose
// errors are all +inf still gets the lowest index, as scanning does.
template <int kLanes>
__device__ __forceinline__ int minmax_pattern(const DevTables* __restrict__ tb, const float2 (&ends)[4], float umin,
                                              float umax, int hl, uint32_t gmask, int npat)
{
    constexpr int kPatPerLane = kNPat / kLanes;
    uint32_t eb = 0xffffffffu, bp = 64u;
#pragma unroll
    for (int k = 0; k < kPatPerLane; ++k) {
        const int pat = hl + kLanes * k;
        // 8 lanes (activation groups) hold 8 patterns each: read from L1 instead of registers
        const float2 cp = (kPatPerLane <= 4) ? ends[k % 4] : __ldg(&tb->ends[pat]);
        float d0 = __fsub_rn(umin, cp.x), d1 = __fsub_rn(umax, cp.y);
        float e = __fadd_rn(__fmul_rn(d0, d0), __fmul_rn(d1, d1));
        const uint32_t ek = (pat < npat) ? __float_as_uint(e) : 0xffffffffu;
        if (ek < eb) {
            eb = ek;
            bp = (uint32_t)pat;
        }
    }
    const uint32_t emin = hw_min(gmask, eb);
    return (int)hw_min(gmask, eb == emin ? bp : 64u);
}

// Encodes one group of G values with the G/8 lanes of `gmask`; hl = lane
// within the group, q = its values 8 hl .. 8 hl + 7.  cent: centroids [64][16]
// (SEL = 1 only).
template <int SEL, int G>
__device__ __forceinline__ void encode_group(const DevTables* __restrict__ tb, const uint32_t* rows,
                                             uint32_t QL, const float4* qmap, const float* cent, uint32_t* buf, uint32_t* top,
                                             const float2 (&ends)[4], const uint4 q, uint8_t* dst, int hl,
                                             uint32_t gmask, int npat, Counters& cnt)
{
    constexpr int kLanes = G / 8;             // lanes per group
    constexpr int kPatPerLane = kNPat / kLanes;
    constexpr int kWords = 16 / kLanes;       // block words each lane stores
    uint32_t b[8] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16,
                     q.z & 0xffffu, q.z >> 16, q.w & 0xffffu, q.w >> 16};
    const int i0 = 8 * hl;

    // every element's key, kept for the outlier records
    uint32_t kk[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) kk[j] = keyof(b[j], i0 + j);
    uint32_t key = max(max(max(kk[0], kk[1]), max(kk[2], kk[3])), max(max(kk[4], kk[5]), max(kk[6], kk[7])));
    key = hw_max(gmask, key);
    if ((key >> 8) >= 0x7f80u) {  // a NaN or Inf in the group: encoded as +0, counted
        uint32_t nf = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((b[j] & 0x7f80u) == 0x7f80u) {
                b[j] = 0;
                ++nf;
            }
        cnt.nonfinite += hw_add(gmask, nf);
#pragma unroll
        for (int j = 0; j < 8; ++j) kk[j] = keyof(b[j], i0 + j);
        key = max(max(max(kk[0], kk[1]), max(kk[2], kk[3])), max(max(kk[4], kk[5]), max(kk[6], kk[7])));
        key = hw_max(gmask, key);
    }
    const int m = 127 - (int)((key >> 1) & 127u);
    const bool owner = (hl == (m >> 3));
    const int mj = m & 7;

    // ---- group scale by table: E4M3(|x_m| / S_t) with x_m's sign; then 1/s
    const uint32_t code = (uint32_t)__ldg(&tb->code_of_mag[key >> 8]) | ((key & 1u) << 7);
    cnt.groups += 1;
    if ((code & 0x7fu) == 0u) {
        if constexpr (kWords == 1)
            reinterpret_cast<uint32_t*>(dst)[hl] = 0u;
        else
            reinterpret_cast<uint2*>(dst)[hl] = make_uint2(0u, 0u);
        cnt.zero += 1;
        return;
    }
    const float inv = __ldg(&tb->inv_of_code[code]);

    // ---- normalise; min / max over i != m.  s carries x_m's sign, so u_m =
    // |x_m| / |s| > 0 and no u_i exceeds it (|x_i| <= |x_m|, and rounding a
    // product by the same factor keeps the order): u_m is the group's largest
    // value, the minimum over i != m is the minimum over all i, and only the
    // maximum has to leave slot m out.
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = __fmul_rn(bf16_bits_to_f32(b[j]), inv);
    const int jm = owner ? mj : 8;  // this lane's slot of m, if it has it
    const float lmin = fminf(fminf(fminf(u[0], u[1]), fminf(u[2], u[3])), fminf(fminf(u[4], u[5]), fminf(u[6], u[7])));
    float lmax;
    {
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = (j == jm) ? -INFINITY : u[j];
        lmax = fmaxf(fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])), fmaxf(fmaxf(e[4], e[5]), fmaxf(e[6], e[7])));
    }
    const float umin = hw_minf(gmask, lmin);
    const float umax = hw_maxf(gmask, lmax);
    int p = minmax_pattern<kLanes>(tb, ends, umin, umax, hl, gmask, npat);
    if constexpr (SEL == 1) {
        // ---- pattern by the full squared error (slot m adds +0): the first
        // pattern, in index order, with the least error.  An error is a tree
        // of rounded additions of non-negative terms; rounding is monotone, so
        // setting every term but two to zero can only lower it, and what is
        // left is the rounded sum of those two: term(umin) + term(umax) (two
        // distinct elements other than m, computed with the same operations)
        // bounds each pattern's error from below.  A pattern whose bound
        // exceeds the min / max rule's pattern's error cannot be the first
        // minimum; the others are summed in order, and once one is the best
        // so far, the later ones whose bound is not below it are dropped too
        // (a tie goes to the earlier index).
        auto term = [&](int q, float v) {
            const uint32_t Rq = (uint32_t)__cvta_generic_to_shared(rows) + (uint32_t)(q * kRow) * 4u;
            const float4 qmq = qmap[q];
            const int sq = (qmq.z == 0.0f) ? quantise_bucket(Rq, QL + (uint32_t)q * 256u, qmq, v)
                                           : quantise(Rq, __uint_as_float(lds_u32(Rq + 28u)), v);
            const float d = __fsub_rn(v, cent[q * 16 + sq]);
            return __fmul_rn(d, d);
        };
        auto error = [&](int q) {
            const uint32_t Rq = (uint32_t)__cvta_generic_to_shared(rows) + (uint32_t)(q * kRow) * 4u;
            const float* Cq = cent + q * 16;
            const float tq = __uint_as_float(lds_u32(Rq + 28u));
            const float4 qmq = qmap[q];
            const uint32_t Lq = QL + (uint32_t)q * 256u;
            float d2[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int sj = (qmq.z == 0.0f) ? quantise_bucket(Rq, Lq, qmq, u[j]) : quantise(Rq, tq, u[j]);
                const float d = __fsub_rn(u[j], Cq[sj]);
                d2[j] = (owner && j == mj) ? 0.0f : __fmul_rn(d, d);
            }
            float v = __fadd_rn(__fadd_rn(__fadd_rn(d2[0], d2[1]), __fadd_rn(d2[2], d2[3])),
                                __fadd_rn(__fadd_rn(d2[4], d2[5]), __fadd_rn(d2[6], d2[7])));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) v = __fadd_rn(v, __shfl_xor_sync(gmask, v, o));
            return v;
        };
        const float known = error(p);
        const int base = __ffs(gmask) - 1;  // the group's first lane in the warp
        float lb[kPatPerLane];              // bounds of this lane's patterns hl + kLanes k
        uint64_t keep = 0;                  // bit q: pattern q may be the first minimum
#pragma unroll
        for (int k = 0; k < kPatPerLane; ++k) {
            const int pat = hl + kLanes * k;
            lb[k] = (pat < npat) ? __fadd_rn(term(pat, umin), term(pat, umax)) : __int_as_float(0x7f800000);
            const bool may = pat < npat && !(lb[k] > known);
            const uint32_t bits = (__ballot_sync(gmask, may) >> base) & ((1u << kLanes) - 1u);
            keep |= (uint64_t)bits << (kLanes * k);
        }
        float best = 0.0f;
        p = -1;
        while (keep) {  // uniform in the group
            const int q = __ffsll((long long)keep) - 1;
            keep &= keep - 1;
            const float v = error(q);
            if (p < 0 || v < best) {
                best = v;
                p = q;
                uint64_t below = 0;  // the patterns whose bound is below the new best
#pragma unroll
                for (int k = 0; k < kPatPerLane; ++k) {
                    const uint32_t bits = (__ballot_sync(gmask, lb[k] < best) >> base) & ((1u << kLanes) - 1u);
                    below |= (uint64_t)bits << (kLanes * k);
                }
                keep &= below;
            }
        }
    }

    // ---- quantise (count of thresholds strictly below u); lengths
    const uint32_t R = (uint32_t)__cvta_generic_to_shared(rows) + (uint32_t)(p * kRow) * 4u;
    const float4 qm = qmap[p];
    int sym[8];
    if (qm.z == 0.0f) {
        const uint32_t L = QL + (uint32_t)p * 256u;
#pragma unroll
        for (int j = 0; j < 8; ++j) sym[j] = (j == jm) ? 15 : quantise_bucket(R, L, qm, u[j]);
    } else {
        const float t7 = __uint_as_float(lds_u32(R + 28u));
#pragma unroll
        for (int j = 0; j < 8; ++j) sym[j] = (j == jm) ? 15 : quantise(R, t7, u[j]);
    }
    uint32_t acc = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc += lds_u32(R + 4u * (uint32_t)(kRowLens + sym[j]));
    const uint32_t lo = hw_add(gmask, acc & 0x00ff00ffu);         // h = 0, 2
    const uint32_t hi = hw_add(gmask, (acc >> 8) & 0x00ff00ffu);  // h = 1, 3
    int h = 0, L = (int)(lo & 0xffffu);
    if ((int)(hi & 0xffffu) < L) { L = (int)(hi & 0xffffu); h = 1; }
    if ((int)(lo >> 16) < L) { L = (int)(lo >> 16); h = 2; }
    if ((int)(hi >> 16) < L) { L = (int)(hi >> 16); h = 3; }

    // ---- two chunks of 4 codewords each, in stream order (<= 32 bits each)
    const uint32_t CW = R + 4u * (uint32_t)(kRowCode + 16 * h);
    uint32_t ch[2];
    int cl[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t w = 0;
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t e = lds_u32(CW + 4u * (uint32_t)sym[4 * c + j]);
            w |= (e & 0xffu) << n;
            n += (int)(e >> 8);
        }
        ch[c] = w;
        cl[c] = n;
    }
    const int tot = cl[0] + cl[1];
    int off = tot;  // inclusive scan over the group's lanes
#pragma unroll
    for (int dlt = 1; dlt < kLanes; dlt <<= 1) {
        int t = __shfl_up_sync(gmask, off, dlt, kLanes);
        if (hl >= dlt) off += t;
    }
    off -= tot;

    // ---- OR the chunks into the block; bits at or past 512 are dropped (clip)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int bpos = kHdrBits + off + (c ? cl[0] : 0);
        const int w = bpos >> 5, sh = bpos & 31;
        if (w < 16) atomicOr(&buf[w], ch[c] << sh);
        if (sh != 0 && sh + cl[c] > 32 && w + 1 < 16) atomicOr(&buf[w + 1], ch[c] >> (32 - sh));
    }
    if (hl == 0) atomicOr(&buf[0], code | ((uint32_t)p << 8) | ((uint32_t)h << 14));

    // ---- outlier records in the spare bits of an unclipped block
    if (L <= kPayloadBits) {
        const int n = min(kMaxRec, (kPayloadBits - L) / kRecBits);
        if (n > 0) {
            // candidates: key + 1 (0 = the scale element / taken), each lane's 8
            // sorted descending once (Batcher odd-even merge network); every round
            // takes the largest head of the group's lanes into the shared list
            // `top` and its lane pops it.  Then lane r < n writes record r: the key
            // holds the element's bf16 bits and index, so nothing else is needed.
            uint32_t k[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = (j == jm) ? 0u : kk[j] + 1u;
            sort8_desc(k);
            for (int r = 0; r < n; ++r) {
                const uint32_t bestk = hw_max(gmask, k[0]);
                if (k[0] == bestk) {  // exactly one lane: keys are unique
                    top[r] = bestk - 1u;
#pragma unroll
                    for (int j = 0; j < 7; ++j) k[j] = k[j + 1];
                    k[7] = 0u;
                }
            }
            __syncwarp(gmask);
#pragma unroll
            for (int pass = 0; pass < kMaxRec / kLanes; ++pass) {  // 16-lane groups: 1 pass, 8-lane: 2
                const int r = hl + pass * kLanes;
                if (r < n) {
                    const uint32_t key = top[r];
                    const int i = 127 - (int)((key >> 1) & 127u);
                    const uint32_t xb = ((key >> 8) & 0x7fffu) | ((key & 1u) << 15);
                    const float uv = __fmul_rn(bf16_bits_to_f32(xb), inv);
                    const float v = fminf(fmaxf(rintf(__fmul_rn(uv, 127.0f)), -127.0f), 127.0f);
                    const uint32_t rec = (uint32_t)i | (((uint32_t)(int)v & 0xffu) << 7);
                    const int at = kHdrBits + L + r * kRecBits;
                    const int ww = at >> 5, ss = at & 31;
                    atomicOr(&buf[ww], rec << ss);
                    if (ss > 32 - kRecBits) atomicOr(&buf[ww + 1], rec >> (32 - ss));
                }
            }
            cnt.records += n;
            cnt.padded += 1;
        }
        cnt.bits += L;
    } else {
        cnt.clipped += 1;
        cnt.bits += kPayloadBits;
    }

    __syncwarp(gmask);
    if constexpr (kWords == 1) {
        reinterpret_cast<uint32_t*>(dst)[hl] = buf[hl];
        buf[hl] = 0u;
    } else {
        reinterpret_cast<uint2*>(dst)[hl] = make_uint2(buf[2 * hl], buf[2 * hl + 1]);
        buf[2 * hl] = 0u;
        buf[2 * hl + 1] = 0u;
    }
    __syncwarp(gmask);
}

// Copies a tensor's pattern rows (thresholds, lengths, codewords), bucket
// counts and bucket maps into shared memory (NT threads).
template <int NT>
__device__ __forceinline__ void stage_pattern_rows(const DevTables* __restrict__ tb, uint32_t* rows, uint8_t* qlo,
                                                   float4* qmap, int tid)
{
    {
        // 24 16-byte pieces per pattern row (thresholds, lengths, codewords),
        // all loads issued before any store so the copy costs one latency.
        constexpr int kRowVec = 24, kPer = kNPat * kRowVec / NT;
        uint4 v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * NT, p = i / kRowVec, part = i - p * kRowVec;
            const uint4* src = part < 4   ? reinterpret_cast<const uint4*>(tb->T16[p]) + part
                               : part < 8 ? reinterpret_cast<const uint4*>(tb->lens4[p]) + (part - 4)
                                          : reinterpret_cast<const uint4*>(&tb->code[p][0][0]) + (part - 8);
            v[k] = __ldg(src);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = tid + k * NT, p = i / kRowVec, part = i - p * kRowVec;
            uint32_t* d = rows + p * kRow + 4 * part;  // T at 0..15, lengths 16..31, codewords 32..95
            d[0] = v[k].x;
            d[1] = v[k].y;
            d[2] = v[k].z;
            d[3] = v[k].w;
        }
    }
    {
        constexpr int kQVec = kNPat * 256 / 16, kPerQ = kQVec / NT;
        uint4 w[kPerQ];
#pragma unroll
        for (int k = 0; k < kPerQ; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(&tb->qlo[0][0]) + tid + k * NT);
#pragma unroll
        for (int k = 0; k < kPerQ; ++k) reinterpret_cast<uint4*>(qlo)[tid + k * NT] = w[k];
        if (tid < kNPat) qmap[tid] = __ldg(&tb->qmap[tid]);
    }
}

// Adds a group's lanes' counters (one lane's copy: they are uniform) to the caller's.
__device__ __forceinline__ void add_counters(ecco_stats* stats, const Counters& cnt)
{
    if (stats && cnt.groups) {
        atomicAdd(&stats->n_groups, (unsigned long long)cnt.groups);
        if (cnt.zero) atomicAdd(&stats->n_zero, (unsigned long long)cnt.zero);
        if (cnt.clipped) atomicAdd(&stats->n_clipped, (unsigned long long)cnt.clipped);
        if (cnt.padded) atomicAdd(&stats->n_padded, (unsigned long long)cnt.padded);
        if (cnt.records) atomicAdd(&stats->n_records, (unsigned long long)cnt.records);
        if (cnt.nonfinite) atomicAdd(&stats->n_nonfinite, (unsigned long long)cnt.nonfinite);
        if (cnt.bits) atomicAdd(&stats->payload_bits, cnt.bits);
    }
}

}  // namespace
}  // namespace ecco
