// Device building blocks of the row operators (norm, token log probabilities,
// distillation): 16-byte accesses at any element address, a stretch of a row
// held in registers, and reductions over a wave and a workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "mxq_device.hpp"

namespace mxq {

typedef __bf16 bf16_t;

// ---- 16-byte accesses ----------------------------------------------------------
// Rows may start at any element (odd lengths, odd leading dimensions).  The
// hardware takes 16-byte accesses at any address here, a wave's 1 KB then
// touches one line more, so the same loads serve every alignment.
template <class T> constexpr int kElems = 16 / (int)sizeof(T);
template <class T> struct Unaligned;
template <> struct Unaligned<bf16_t> {
    typedef gv4u v4 __attribute__((aligned(2)));
    typedef gv2u v2 __attribute__((aligned(2)));
};
template <> struct Unaligned<float> {
    typedef gv4u v4 __attribute__((aligned(4)));
    typedef gv2u v2 __attribute__((aligned(4)));
};

template <class T> __device__ __forceinline__ gv4u load_vec(const T *p)
{
    return *(const MXQ_GLOBAL typename Unaligned<T>::v4 *)p;
}
template <class T> __device__ __forceinline__ float load_one(const T *p)
{
    return (float)*(const MXQ_GLOBAL T *)p;
}

// `raw` as kElems<T> floats (exact)
__device__ __forceinline__ void unpack(gv4u raw, float (&f)[8], bf16_t *)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = as_f(raw[j] << 16);
        f[2 * j + 1] = as_f(raw[j] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(gv4u raw, float (&f)[4], float *)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = as_f(raw[j]);
}

// two floats as bf16, each to the nearest, ties to even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}

// E consecutive elements
template <int E> __device__ __forceinline__ void store_vec(bf16_t *p, const float (&f)[E])
{
    if constexpr (E == 8)
        *(MXQ_GLOBAL Unaligned<bf16_t>::v4 *)p = (gv4u){pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                        pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    else
        *(MXQ_GLOBAL Unaligned<bf16_t>::v2 *)p = (gv2u){pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
}
template <int E> __device__ __forceinline__ void store_vec(float *p, const float (&f)[E])
{
#pragma unroll
    for (int j = 0; j < E; j += 4)
        *(MXQ_GLOBAL Unaligned<float>::v4 *)(p + j) =
            (gv4u){as_u(f[j]), as_u(f[j + 1]), as_u(f[j + 2]), as_u(f[j + 3])};
}
// the first `left` of them (left may be E or more)
template <class O, int E>
__device__ __forceinline__ void store_some(O *p, const float (&f)[E], int left)
{
    if (left >= E) {
        store_vec(p, f);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (j < left)
                *(MXQ_GLOBAL O *)(p + j) = (O)f[j];
    }
}

// kElems<T> elements of which the first `left` are there; the others are `fill`
// (a bit pattern of two bf16 or one fp32)
template <class T> __device__ __forceinline__ gv4u load_some(const T *p, int left, uint32_t fill)
{
    if (left >= kElems<T>)
        return load_vec(p);
    gv4u v = {fill, fill, fill, fill};
#pragma unroll
    for (int j = 0; j < kElems<T> - 1; ++j) {
        if (j < left) {
            if constexpr (sizeof(T) == 4) {
                v[j] = *(const MXQ_GLOBAL uint32_t *)(p + j);
            } else {
                const uint32_t h = *(const MXQ_GLOBAL uint16_t *)(p + j);
                v[j / 2] = j % 2 ? (v[j / 2] & 0xFFFFu) | (h << 16) : (v[j / 2] & 0xFFFF0000u) | h;
            }
        }
    }
    return v;
}

// A uniform value that the compiler takes for a new one: what a pass derives from it
// (the predicates of a row's last, partial vectors) is made again in the next pass
// and not kept in registers for it.
__device__ __forceinline__ int fresh(int v)
{
    asm volatile("" : "+s"(v));
    return v;
}

// The thread's vector of the NT vectors of E elements at p: a uniform address and
// an unsigned offset, so that no 64-bit address per vector is kept in registers.
template <int E, class T> __device__ __forceinline__ T *lane_at(T *p)
{
    return p + threadIdx.x * (unsigned)E;
}

// ---- a stretch of a row in the registers of a workgroup -------------------------
// n elements from p, NV vectors a thread: vector i of thread t starts at element
// (i NT + t) kElems.  What lies beyond n is `fill`.  The whole stretch is in
// flight at once, and a second pass over it costs no memory traffic.
template <class T, int NT, int NV> struct Held {
    static constexpr int E = kElems<T>;
    static constexpr int kMost = NT * NV * E;
    gv4u v[NV];

    static __device__ __forceinline__ int at(int i) { return (i * NT + (int)threadIdx.x) * E; }
    static __device__ __forceinline__ bool any(int i, int n) { return i * NT * E < n; }

    __device__ __forceinline__ void load(const T *p, int n, uint32_t fill)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i + 1) * NT * E <= n)
                v[i] = load_vec(lane_at<E>(p + i * NT * E));
            else if (any(i, n))
                v[i] = load_some(lane_at<E>(p + i * NT * E), n - at(i), fill);
            else
                v[i] = (gv4u){fill, fill, fill, fill};
        }
    }
    // Before a second pass: what the first one made of the vectors (their unpacked
    // values) is not kept in registers for it.
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            asm volatile("" : "+v"(v[i]));
    }
    __device__ __forceinline__ void get(int i, float (&f)[E]) const { unpack(v[i], f, (T *)nullptr); }
};

template <class O, int NT, int E>
__device__ __forceinline__ void store_held(O *p, int i, int n, const float (&f)[E])
{
    if ((i + 1) * NT * E <= n)
        store_vec(lane_at<E>(p + i * NT * E), f);
    else
        store_some(lane_at<E>(p + i * NT * E), f, n - (i * NT + (int)threadIdx.x) * E);
}

// ---- reductions -----------------------------------------------------------------
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

}  // namespace mxq
