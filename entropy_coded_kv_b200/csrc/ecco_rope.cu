// Rotary positions: the table of angles and the turn itself.
//
// y_a = a cos - b sin, y_b = b cos + a sin, every operation one fp32 rounding
// (no fused multiply-add), so the turned keys that ecco_paged_append encodes
// and the ones this kernel writes are the same bits.
#include "ecco_paged.cuh"
#include "ecco_rope.cuh"

namespace ecco {
namespace {

constexpr int kMaxFreq = 512;
struct Freqs {
    double f[kMaxFreq];
};

__global__ void rope_table_kernel(const __grid_constant__ Freqs F, int n_freq, double magnitude, int64_t total,
                                  float2* table)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t p = i / n_freq;
        double sn, cs;
        sincos((double)p * F.f[i - p * n_freq], &sn, &cs);
        table[i] = make_float2((float)(magnitude * cs), (float)(magnitude * sn));
    }
}

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads whose loads a thread has in flight (y may be x: the compiler cannot move a load over a store)

template <typename T>
struct Vec8 {  // 8 values: 16 bytes of a 16-bit type, 32 of fp32
    uint4 w[sizeof(T) / 2];
};

// x is read once and streams past L2, which y should find room in: 22 us for
// [8191, 32, 128] bf16 against 28 with plain loads (6.1 and 4.9 TB/s).  Calls one
// behind the other on arrays that L2 does not hold: bf16 and fp16 26.7 us (5.1
// TB/s), fp32 51.2 us (5.3 TB/s), halves or adjacent pairs, all of a head or half.
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p)
{
    Vec8<T> v;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v.w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    return v;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& v)
{
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = v.w[i];
}

// A thread has one unit of a token's heads: pieces u and u + rotary / 16 of 8
// values, turned together -- halves: value k of the one with value k of the
// other; interleaved: each has its own pairs -- or two pieces behind the turned
// part, copied.  Neighbouring threads have neighbouring pieces, whatever they
// do with them.  A thread does so for every head h0, h0 + groups, .. of the
// token, so cos and sin are loaded once for them and the heads' loads overlap.
// `per` = units * groups threads a token, 32-bit indices inside it.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs A, int units, int groups,
                                                        int tokens_per_block)
{
    const int per = units * groups, pairs8 = A.rotary / 16;
    const int lt = threadIdx.x / per;
    const int64_t t = (int64_t)blockIdx.x * tokens_per_block + lt;
    if (lt >= tokens_per_block || t >= A.tokens) return;
    const T* xt = static_cast<const T*>(A.x) + t * A.x_token;
    T* yt = static_cast<T*>(A.y) + t * A.y_token;
    const int64_t pos = min(max((int64_t)A.positions[t], (int64_t)0), A.n_positions - 1);
    for (int w = threadIdx.x - lt * per; w < per; w += kThreads) {
        const int h0 = w / units, u = w - h0 * units;
        const bool turn = u < pairs8;
        const int rest = (A.dim - A.rotary) / 8, apart = turn ? pairs8 : (rest + 1) / 2;
        const int ia = 8 * (turn ? u : 2 * pairs8 + u - pairs8), ib = ia + 8 * apart;
        const bool two = turn || ib < A.dim;  // an odd piece is left over behind the turned part
        float4 cs[4];  // cos, sin of 8 pairs
        if (turn) {
            const float4* table = reinterpret_cast<const float4*>(A.table + pos * A.rotary);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cs[k] = __ldg(table + (A.interleaved ? 2 * u + (k & 1) + (k >> 1) * 2 * pairs8 : 4 * u + k));
                if (A.inverse) {
                    cs[k].y = -cs[k].y;
                    cs[k].w = -cs[k].w;
                }
            }
        }
        for (int h = h0; h < A.heads; h += kBatch * groups) {
            Vec8<T> a[kBatch], b[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (h + k * groups < A.heads) {
                    const T* x = xt + (h + k * groups) * A.x_head;
                    a[k] = load8(x + ia);
                    if (two) b[k] = load8(x + ib);
                }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (h + k * groups >= A.heads) break;
                T* ea = reinterpret_cast<T*>(&a[k]);
                T* eb = reinterpret_cast<T*>(&b[k]);
                if (turn) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        if (A.interleaved) {
                            T* e = (p < 2) ? ea + 4 * p : eb + 4 * (p - 2);
                            rope_turn(e[0], e[1], cs[p].x, cs[p].y);
                            rope_turn(e[2], e[3], cs[p].z, cs[p].w);
                        } else {
                            rope_turn(ea[2 * p], eb[2 * p], cs[p].x, cs[p].y);
                            rope_turn(ea[2 * p + 1], eb[2 * p + 1], cs[p].z, cs[p].w);
                        }
                    }
                }
                T* y = yt + (h + k * groups) * A.y_head;
                store8(y + ia, a[k]);
                if (two) store8(y + ib, b[k]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_table(const double* inv_freq, int n_freq, double magnitude, int64_t n_positions, float* table,
                              cudaStream_t s)
{
    Freqs F;
    for (int i = 0; i < n_freq; ++i) F.f[i] = inv_freq[i];
    const int64_t total = n_positions * n_freq, want = (total + 255) / 256, cap = (int64_t)device_sm_count() * 8;
    rope_table_kernel<<<(int)(want < cap ? want : cap), 256, 0, s>>>(F, n_freq, magnitude, total,
                                                                     reinterpret_cast<float2*>(table));
    return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t s)
{
    const int units = a.rotary / 16 + (a.copy_rest ? ((a.dim - a.rotary) / 8 + 1) / 2 : 0);
    // heads a thread does in turn: 8 where that leaves every SM 1024 threads, else fewer
    const int64_t spare = a.tokens * a.heads * units / ((int64_t)device_sm_count() * 1024);
    const int each = spare >= 8 ? 8 : spare >= 4 ? 4 : spare >= 2 ? 2 : 1;
    const int groups = (a.heads + each - 1) / each, per = units * groups;
    const int tokens_per_block = per < kThreads ? kThreads / per : 1;
    const unsigned grid = (unsigned)((a.tokens + tokens_per_block - 1) / tokens_per_block);
    if (dtype == ECCO_BF16)
        rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a, units, groups, tokens_per_block);
    else if (dtype == ECCO_F16)
        rope_kernel<__half><<<grid, kThreads, 0, s>>>(a, units, groups, tokens_per_block);
    else
        rope_kernel<float><<<grid, kThreads, 0, s>>>(a, units, groups, tokens_per_block);
    return cudaGetLastError();
}

}  // namespace ecco
