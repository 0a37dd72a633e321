// One rotary pair, shared by ecco_rope and ecco_paged_append.
#pragma once

#include <cuda_fp16.h>

#include "ecco_internal.cuh"

namespace ecco {

__device__ __forceinline__ float rope_load(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float rope_load(__half v) { return __half2float(v); }
__device__ __forceinline__ float rope_load(float v) { return v; }
__device__ __forceinline__ void rope_store(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void rope_store(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void rope_store(float& d, float v) { d = v; }

// (a, b) -> (a cos - b sin, b cos + a sin), each product and sum rounded to fp32.
template <typename T>
__device__ __forceinline__ void rope_turn(T& a, T& b, float cs, float sn)
{
    const float x = rope_load(a), y = rope_load(b);
    rope_store(a, __fsub_rn(__fmul_rn(x, cs), __fmul_rn(y, sn)));
    rope_store(b, __fadd_rn(__fmul_rn(y, cs), __fmul_rn(x, sn)));
}

}  // namespace ecco
