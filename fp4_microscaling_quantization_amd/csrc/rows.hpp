// Device building blocks of the row operators (norm, token log probabilities,
// distillation): element access and reductions over a wave and a workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_device.hpp"

namespace mxq {

typedef __bf16 bf16_t;

__device__ __forceinline__ float wave_sum(float v)
{
    v += lane_xor_f<1>(v);
    v += lane_xor_f<2>(v);
    v += lane_xor_f<4>(v);
    v += lane_xor_f<8>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, lane_xor_f<1>(v));
    v = fmaxf(v, lane_xor_f<2>(v));
    v = fmaxf(v, lane_xor_f<4>(v));
    v = fmaxf(v, lane_xor_f<8>(v));
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
    return v;
}

// Sum over the workgroup's NT threads, in every thread; `lds` holds NT / 64
// floats and is free again after the next barrier of the caller's.
template <int NT> __device__ __forceinline__ float block_sum(float v, float *lds)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w)
        s += lds[w];
    return s;
}
template <int NT> __device__ __forceinline__ float block_max(float v, float *lds)
{
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = lds[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w)
        s = fmaxf(s, lds[w]);
    return s;
}

}  // namespace mxq
