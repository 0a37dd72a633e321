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

template <typename T>
struct Vec8 {  // 8 values: 16 bytes of a 16-bit type, 32 of fp32
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p)
{
    Vec8<T> v;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v.w[i] = reinterpret_cast<const uint4*>(p)[i];
    return v;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& v)
{
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = v.w[i];
}

// A thread turns one unit of a head: 8 pairs (values 8u.. and their partners
// rotary / 2 further on, or 16 values in a row), or copies 8 values behind
// the turned part.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs A, int units, int64_t total)
{
    const int pairs8 = A.rotary / 16;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t th = i / units, t = th / A.heads;
        const int u = (int)(i - th * units), h = (int)(th - t * A.heads);
        const T* x = static_cast<const T*>(A.x) + t * A.x_token + h * A.x_head;
        T* y = static_cast<T*>(A.y) + t * A.y_token + h * A.y_head;
        if (u >= pairs8) {
            const int at = A.rotary + 8 * (u - pairs8);
            store8(y + at, load8(x + at));
            continue;
        }
        const int ia = A.interleaved ? 16 * u : 8 * u, ib = A.interleaved ? ia + 8 : ia + A.rotary / 2;
        Vec8<T> a = load8(x + ia), b = load8(x + ib);
        const int64_t pos = min(max((int64_t)A.positions[t], (int64_t)0), A.n_positions - 1);
        const float4* cs = reinterpret_cast<const float4*>(A.table + (pos * (A.rotary / 2) + 8 * u) * 2);
        T* ea = reinterpret_cast<T*>(&a);
        T* eb = reinterpret_cast<T*>(&b);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // pairs 2k, 2k + 1
            const float4 c = __ldg(cs + k);
            const float s0 = A.inverse ? -c.y : c.y, s1 = A.inverse ? -c.w : c.w;
            if (A.interleaved) {
                T* e = (k < 2) ? ea + 4 * k : eb + 4 * (k - 2);
                rope_turn(e[0], e[1], c.x, s0);
                rope_turn(e[2], e[3], c.z, s1);
            } else {
                rope_turn(ea[2 * k], eb[2 * k], c.x, s0);
                rope_turn(ea[2 * k + 1], eb[2 * k + 1], c.z, s1);
            }
        }
        store8(y + ia, a);
        store8(y + ib, b);
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
    const int units = a.rotary / 16 + (a.copy_rest ? (a.dim - a.rotary) / 8 : 0);
    const int64_t total = a.tokens * a.heads * units;
    const int64_t want = (total + kThreads - 1) / kThreads, cap = (int64_t)device_sm_count() * 64;
    const int grid = (int)(want < cap ? want : cap);
    if (dtype == ECCO_BF16)
        rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a, units, total);
    else if (dtype == ECCO_F16)
        rope_kernel<__half><<<grid, kThreads, 0, s>>>(a, units, total);
    else
        rope_kernel<float><<<grid, kThreads, 0, s>>>(a, units, total);
    return cudaGetLastError();
}

}  // namespace ecco
