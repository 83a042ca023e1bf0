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

// Workgroups of a launch over rows; more rows loop.  (The tests have a build in which a
// handful of rows do.)
#ifndef MXQ_ROW_GRID
#define MXQ_ROW_GRID (1 << 20)
#endif
constexpr int64_t kMaxGrid = MXQ_ROW_GRID;

// ---- 16-byte accesses ----------------------------------------------------------
// Rows may start at any element (odd lengths, odd leading dimensions); the hardware
// takes 16-byte accesses at any address here.
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
// ONCE: what is not read again leaves the caches to what is (16-byte loads and stores
// with the non-temporal hint; 4096 x 32000 bf16 logits to gradients: 112 to 101 us).
template <bool ONCE, class T> __device__ __forceinline__ gv4u load_vec(const T *p)
{
    const auto *g = (const MXQ_GLOBAL typename Unaligned<T>::v4 *)p;
    if constexpr (ONCE)
        return __builtin_nontemporal_load(g);
    else
        return *g;
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
__device__ __forceinline__ void unpack(gv2u raw, float (&f)[4], bf16_t *)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
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

// E consecutive elements, not read again here
template <int E> __device__ __forceinline__ void store_vec(bf16_t *p, const float (&f)[E])
{
    if constexpr (E == 8)
        __builtin_nontemporal_store((gv4u){pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                           pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])},
                                    (MXQ_GLOBAL Unaligned<bf16_t>::v4 *)p);
    else
        __builtin_nontemporal_store((gv2u){pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])},
                                    (MXQ_GLOBAL Unaligned<bf16_t>::v2 *)p);
}
template <int E> __device__ __forceinline__ void store_vec(float *p, const float (&f)[E])
{
#pragma unroll
    for (int j = 0; j < E; j += 4)
        __builtin_nontemporal_store(
            (gv4u){as_u(f[j]), as_u(f[j + 1]), as_u(f[j + 2]), as_u(f[j + 3])},
            (MXQ_GLOBAL Unaligned<float>::v4 *)(p + j));
}

// A row's last vector may be partial.  It is loaded whole, from the row's last E
// elements, so that a load is the same straight code everywhere (a branch around it
// would make the compiler wait for all loads in flight): the vector that should start
// at element `at` of n starts at vec_start, and its first skipped() elements belong to
// the vector before it (E and more: there is none at `at`).
template <int E> __device__ __forceinline__ int vec_start(int at, int n) { return min(at, n - E); }

// elements from `skip` on
template <class O, int E>
__device__ __forceinline__ void store_from(O *p, const float (&f)[E], int skip)
{
    if (skip == 0) {
        store_vec(p, f);
    } else {
#pragma unroll
        for (int j = 1; j < E; ++j)
            if (j >= skip)
                *(MXQ_GLOBAL O *)(p + j) = (O)f[j];
    }
}

// The only vector of a row with fewer than kElems<T> elements, as load_vec would give
// it: element j of it is element j - (kElems<T> - n) of the row.
template <class T> __device__ __forceinline__ gv4u load_short(const T *p, int n)
{
    gv4u v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 1; j < kElems<T>; ++j) {
        const int e = j - (kElems<T> - n);
        if (e >= 0) {
            if constexpr (sizeof(T) == 4) {
                v[j] = *(const MXQ_GLOBAL uint32_t *)(p + e);
            } else {
                const uint32_t h = *(const MXQ_GLOBAL uint16_t *)(p + e);
                v[j / 2] |= j % 2 ? h << 16 : h;
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
// (i NT + t) kElems.  The whole stretch is in flight at once, and a second pass over
// it costs no memory traffic.  A stretch of fewer than kElems elements has to follow
// others of its row, or the row is short.
template <class T, int NT, int NV> struct Held {
    static constexpr int E = kElems<T>;
    static constexpr int kMost = NT * NV * E;
    gv4u v[NV];

    static __device__ __forceinline__ int at(int i) { return (i * NT + (int)threadIdx.x) * E; }
    // whether vector i is there for some thread, for all threads
    static __device__ __forceinline__ bool any(int i, int n) { return i * NT * E < n; }
    static __device__ __forceinline__ bool whole(int i, int n) { return (i + 1) * NT * E <= n; }
    // where the thread's vector i starts, and what of it is not its own
    static __device__ __forceinline__ int start(int i, int n) { return vec_start<E>(at(i), n); }
    static __device__ __forceinline__ int skip(int i, int n) { return at(i) - start(i, n); }

    // SHORT: the row has fewer than E elements; ONCE: it is not read again
    template <bool SHORT, bool ONCE> __device__ __forceinline__ void load(const T *p, int n)
    {
        if constexpr (SHORT) {
            v[0] = load_short(p, n);
#pragma unroll
            for (int i = 1; i < NV; ++i)
                v[i] = v[0];
        } else {
            n = fresh(n);  // or the offsets of a loop's rows, all the same, are kept
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                // a uniform address and an unsigned offset: no 64-bit address per vector
                const int lo = min(0, n - E);
                v[i] = load_vec<ONCE>((p + lo) + (unsigned)(start(i, n) - lo));
            }
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
    // What is not the thread's own is `none`; nor are the stretch's first `lead` < E
    // elements (bf16 only).
    __device__ __forceinline__ void get(int i, int n, float none, float (&f)[E], int lead = 0) const
    {
        get(i, f);
        if (!whole(i, n) || has_lead(i, lead)) {
            const int d = first_own(i, n, lead);
#pragma unroll
            for (int j = 0; j < E; ++j)
                f[j] = j >= d ? f[j] : none;
        }
    }
    // f as vector i of a stretch at o
    template <class O>
    static __device__ __forceinline__ void put(O *o, int i, int n, const float (&f)[E],
                                               int lead = 0)
    {
        if (whole(i, n) && !has_lead(i, lead)) {
            store_vec(lane_at<E>(o + i * NT * E), f);
        } else {
            const int d = first_own(i, n, lead);
            if (d < E)
                store_from(o + start(i, n), f, d);
        }
    }

    static __device__ __forceinline__ bool has_lead(int i, int lead)
    {
        return sizeof(T) == 2 && i == 0 && lead > 0;
    }
    static __device__ __forceinline__ int first_own(int i, int n, int lead)
    {
        const int d = skip(i, n);
        return has_lead(i, lead) && threadIdx.x == 0 ? lead : d;
    }
};

// How many elements a row starts after a 16-byte boundary.  A bf16 row that starts in
// the middle of a word reads a third slower (2048 x 50257 against x 50256: 47.9 and 37.6
// us); its stretches then start at the boundary, and what lies before the row (within
// the same 16 bytes, so in the same allocation) is not its own.  fp32 rows lose 3%
// off the boundary and are left as they are, and so are rows shorter than a vector.
template <class T, bool SHORT> __device__ __forceinline__ int lead_of(const T *row)
{
    return sizeof(T) == 2 && !SHORT ? (int)((reinterpret_cast<uintptr_t>(row) >> 1) & 7) : 0;
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
