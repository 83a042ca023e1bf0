// A tile of a bf16 matrix product on the matrix cores, for the operators that put
// their own arithmetic behind it.
//
//   out[q][p] = sum over k of P[p][k] Q[q][k], fp32, p the contiguous side of out
//
// v_mfma_f32_16x16x32_bf16: lane (g, li) = (lane / 16, lane % 16) supplies row li of
// each operand and its values k = 8 g .. 8 g + 7; it holds rows 4 g .. 4 g + 3 of column
// li of the product, that is four neighbours of out's contiguous side.
//
// An operand lies in memory in one of two ways:
//   along k (ALONG):   a row of the operand is contiguous in k.  A step's tile is
//                      [rows][32 k], 64 bytes a row; a fragment is one 16-byte read.
//   across k (!ALONG): a value of k is a contiguous run over the operand's rows.  A
//                      step's tile is [32 k][rows]; the LDS turns it while it is read
//                      (ds_read_b64_tr_b16: the 16 lanes of a group read four k of 16
//                      rows, and lane li gets the four k of row li), two reads a
//                      fragment.
// Both are copied as they lie, 16 bytes a lane, into LDS.  A lane's place in LDS is
// fixed (16 bytes times its number), so the order within a tile is made by what each
// lane fetches: 16-byte chunks are exchanged within a row (chunk c of row r lies at
// c ^ x(r)) so that the 16 lanes that read at a time touch every bank once.
#pragma once

#include <type_traits>

#include "lds_copy.hpp"
#include "mxq_device.hpp"

namespace mxq {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kStepK = 32;  // k of a step

// One operand's tile of ROWS rows.
template <int ROWS, bool ALONG> struct Side {
    static constexpr int kBytes = ROWS * kStepK * 2;
    static constexpr int kChunks = kBytes / 1024;  // 1 KiB copies of a wave

    // What lane `lane` fetches for copy cc of a step, in bytes from the tile's first
    // element; ld in elements; rows past the last of `have` >= 1 fetch it again (their
    // products are not used).
    // of !ALONG: k past the last of `have_k` fetch it again.
    static __device__ __forceinline__ uint32_t offset(int cc, int lane, int64_t ld, int have,
                                                      int have_k = kStepK)
    {
        if constexpr (ALONG) {
            const int row = 16 * cc + (lane >> 2);
            const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
            return (uint32_t)(min(row, have - 1) * ld * 2 + chunk * 16);
        } else {
            constexpr int PER = ROWS / 8;  // chunks of one k
            const int k = cc * (64 / PER) + lane / PER;
            const int chunk = (lane % PER) ^ turn(k);
            return (uint32_t)(min(k, have_k - 1) * ld * 2 + min(chunk * 8, have - 8) * 2);
        }
    }
    // how far a step moves along k, in bytes
    static __device__ __forceinline__ int64_t stride(int64_t ld)
    {
        return ALONG ? kStepK * 2 : kStepK * ld * 2;
    }
    // Pairs of chunks (the 16 rows of one fragment) are exchanged: eight k of 256 bytes
    // or more each start in other banks; of 128 bytes, two follow each other.
    static __device__ __forceinline__ int turn(int k)
    {
        return ROWS >= 128 ? 2 * (k & 7) : 2 * ((k >> 1) & 3);
    }

    // Where a wave's fragments lie: wave w of W takes fragments (of 16 rows) w, w + W, ...
    // A lane keeps kBases addresses; fragment i and the tile's place are constants from there.
    template <int W> struct Reader {
        static constexpr int kBases = ALONG ? 1 : W >= 4 ? 1 : 4 / W;
        static_assert(ALONG || ROWS >= 128, "fragments across k are read from 256 bytes and more");
        uint32_t base[kBases];

        __device__ __forceinline__ void start(uint32_t l, int w, int lane)
        {
            const int g = lane >> 4, li = lane & 15;
            if constexpr (ALONG) {
                base[0] = l + w * 1024 + li * 64 + ((g ^ (li >> 2)) * 16);
            } else {
                // fragment t = w + W i lies at pair t ^ (k & 7) of its k, k & 7 = 4 u + li / 4
                // for the read u of the two: the pair's two low bits are the lane's and the
                // base's, the third is a constant's
                const int k = 8 * g + (li >> 2);
#pragma unroll
                for (int b = 0; b < kBases; ++b)
                    base[b] = l + k * (ROWS * 2) + (((w + W * b) & 3) ^ (li >> 2)) * 32 +
                              ((W >= 4 ? w >> 2 : 0) * 128) + ((li >> 1) & 1) * 16 + (li & 1) * 8;
            }
        }
        // fragment i of the tile `at` bytes behind the first
        template <int AT> __device__ __forceinline__ v8bf read(int i) const
        {
            if constexpr (ALONG) {
                typedef __attribute__((address_space(3))) const v8bf lds_v8bf;
                return *(lds_v8bf *)(uintptr_t)(base[0] + AT + i * (W * 1024));
            } else {
                typedef __attribute__((address_space(3))) v4s lds_v4s;
                const int t = W * i;  // and w, whose two low bits are in the base
                v4s h[2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_v4s *)(uintptr_t)(base[i % kBases] + AT + u * (4 * ROWS * 2) + (t >> 3) * 256 +
                                    (((t >> 2) & 1) ^ u) * 128));
                typedef short v8s __attribute__((ext_vector_type(8)));
                return __builtin_bit_cast(
                    v8bf, (v8s)__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
            }
        }
    };
};

// the pointer in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return reinterpret_cast<const uint8_t *>((uint64_t)hi << 32 | lo);
}

// A workgroup of WP x WQ waves, each with NP x NQ tiles of 16 x 16.
template <int WP_, int WQ_, int NP_, int NQ_, bool P_ALONG, bool Q_ALONG> struct Product {
    static constexpr int WP = WP_, WQ = WQ_, NP = NP_, NQ = NQ_;
    static constexpr int kP = 16 * WP * NP, kQ = 16 * WQ * NQ, kWaves = WP * WQ;
    static constexpr int kThreads = 64 * kWaves;
    using SideP = Side<kP, P_ALONG>;
    using SideQ = Side<kQ, Q_ALONG>;
    static constexpr int kStage = SideP::kBytes + SideQ::kBytes;
    static constexpr int kStages = 4;
    static constexpr int kLds = kStages * kStage;
    static constexpr int kPerP = SideP::kChunks / kWaves, kPerQ = SideQ::kChunks / kWaves;
    static constexpr int kPer = kPerP + kPerQ;
    static_assert(kPerP * kWaves == SideP::kChunks && kPerQ * kWaves == SideQ::kChunks,
                  "copies split evenly");

    v4f acc[NP][NQ];
    int lane, wave, wp, wq;
    typename SideP::template Reader<WP> read_p;
    typename SideQ::template Reader<WQ> read_q;
    uint32_t off_p[kPerP], off_q[kPerQ];
    uint32_t at_p, at_q;  // the wave's first copies in LDS
    // (P across k) a last step with fewer k, and what is fetched there
    int cut_step;
    uint32_t cut_p[P_ALONG ? 1 : kPerP];

    // lds: the workgroup's; p, q: leading dimensions and how many rows there are from the
    // tile's first
    __device__ __forceinline__ void start(uint8_t *lds, int64_t ldp, int have_p, int64_t ldq,
                                          int have_q)
    {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wp = wave % WP;
        wq = wave / WP;
        // all slots of P, then all of Q: either side's are within the constant offset of a read
        const uint32_t l = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t *)lds);
        read_p.start(l, wp, lane);
        read_q.start(l + kStages * SideP::kBytes, wq, lane);
        at_p = __builtin_amdgcn_readfirstlane(l + wave * 1024);
        at_q = __builtin_amdgcn_readfirstlane(l + kStages * SideP::kBytes + wave * 1024);
#pragma unroll
        for (int i = 0; i < kPerP; ++i)
            off_p[i] = SideP::offset(wave + i * kWaves, lane, ldp, have_p);
#pragma unroll
        for (int i = 0; i < kPerQ; ++i)
            off_q[i] = SideQ::offset(wave + i * kWaves, lane, ldq, have_q);
        cut_step = -1;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    // P across k: there are k_left values of k; Q is zero in a last step that is not whole
    __device__ __forceinline__ void cut(int k_left, int64_t ldp, int have_p)
    {
        cut_step = k_left % kStepK ? k_left / kStepK : -1;
#pragma unroll
        for (int i = 0; i < kPerP; ++i)
            cut_p[i] = SideP::offset(wave + i * kWaves, lane, ldp, have_p, max(1, k_left % kStepK));
    }
    // copy n of a step: P's first
    template <int SLOT>
    __device__ __forceinline__ void copy(int n, int s, const uint8_t *p, const uint8_t *q)
    {
        if (n < kPerP) {
            uint32_t o = off_p[n];
            if constexpr (!P_ALONG)
                o = s == cut_step ? cut_p[n] : o;
            copy16(p, o, at_p + SLOT * SideP::kBytes + n * (kWaves * 1024));
        } else {
            copy16(q, off_q[n - kPerP], at_q + SLOT * SideQ::kBytes + (n - kPerP) * (kWaves * 1024));
        }
    }
    // fragment n of a step: P's first, all of Q's, the rest of P's
    template <int SLOT>
    __device__ __forceinline__ void fragment(int n, v8bf (&fp)[NP], v8bf (&fq)[NQ]) const
    {
        if (n == 0 || n > NQ)
            fp[n ? n - NQ : 0] = read_p.template read<SLOT * SideP::kBytes>(n ? n - NQ : 0);
        else
            fq[n - 1] = read_q.template read<SLOT * SideQ::kBytes>(n - 1);
    }
    // `steps` steps from the (uniform) addresses p and q of the first one's tiles, each
    // dp and dq bytes further.  All of the LDS is free again when it returns.
    //
    // A ring of four slots.  A step's fragments are read during the step before it, into
    // the other of two register sets, and its copies are issued three steps before it, so
    // that the products run while both are in flight.  Past the last step the reads are
    // not used and the copies fetch the last step again, into slots that nobody reads, so
    // that every step waits for the same number of copies and the loop has no branches.
    __device__ __forceinline__ void run(int steps, const uint8_t *p, uint32_t dp, const uint8_t *q,
                                        uint32_t dq)
    {
        if (steps <= 0)
            return;
        steps = __builtin_amdgcn_readfirstlane(steps);
        p = uniform(p);
        q = uniform(q);
        const auto fetch = [&](int s, auto slot) {
            s = min(s, steps - 1);
#pragma unroll
            for (int n = 0; n < kPer; ++n)
                copy<decltype(slot)::value>(n, s, p + (uint64_t)(uint32_t)s * dp,
                                            q + (uint64_t)(uint32_t)s * dq);
        };
        using std::integral_constant;
        fetch(0, integral_constant<int, 0>{});
        fetch(1, integral_constant<int, 1>{});
        fetch(2, integral_constant<int, 2>{});
        __builtin_amdgcn_s_waitcnt(0x0070 | (2 * kPer));
        barrier_no_fence();
        v8bf fp[2][NP], fq[2][NQ];
#pragma unroll
        for (int n = 0; n < NP + NQ; ++n)
            fragment<0>(n, fp[0], fq[0]);
        const auto step = [&](int s, auto slot) {
            constexpr int SLOT = decltype(slot)::value, SET = SLOT & 1;
            __builtin_amdgcn_sched_barrier(0);
            // this wave's copies of step s + 1 have landed, and its reads of step s ...
            __builtin_amdgcn_s_waitcnt(0x0070 | kPer);
            // ... and everyone's: the slot of step s - 1 is free
            barrier_no_fence();
            __builtin_amdgcn_sched_barrier(0);
            // the reads, then the copies, between the products: in front of them they would
            // hold the wave until the LDS and the address unit have taken them
            s = min(s + 3, steps - 1);
            const uint8_t *ps = p + (uint64_t)(uint32_t)s * dp, *qs = q + (uint64_t)(uint32_t)s * dq;
            constexpr int kItems = NP + NQ + kPer, kProducts = NP * NQ;
#pragma unroll
            for (int n = 0; n < kItems; ++n) {
                if (n < NP + NQ)
                    fragment<(SLOT + 1) & 3>(n, fp[SET ^ 1], fq[SET ^ 1]);
                else
                    copy<(SLOT + 3) & 3>(n - NP - NQ, s, ps, qs);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int m = n * kProducts / kItems; m < (n + 1) * kProducts / kItems; ++m)
                    acc[m / NQ][m % NQ] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        fp[SET][m / NQ], fq[SET][m % NQ], acc[m / NQ][m % NQ], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        int s = 0;
        for (; s + 4 <= steps; s += 4) {
            step(s, integral_constant<int, 0>{});
            step(s + 1, integral_constant<int, 1>{});
            step(s + 2, integral_constant<int, 2>{});
            step(s + 3, integral_constant<int, 3>{});
        }
        if (s < steps)
            step(s, integral_constant<int, 0>{});
        if (s + 1 < steps)
            step(s + 1, integral_constant<int, 1>{});
        if (s + 2 < steps)
            step(s + 2, integral_constant<int, 2>{});
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070);
        barrier_no_fence();
    }
    // p of acc[i][.][0] and q of acc[.][j] within the tile
    __device__ __forceinline__ int p_of(int i) const { return 16 * (wp + WP * i) + 4 * (lane >> 4); }
    __device__ __forceinline__ int q_of(int j) const { return 16 * (wq + WQ * j) + (lane & 15); }
};

// Tile (tp, tq) of workgroup w of np x nq.  Workgroups go round-robin over the 8 XCDs;
// each XCD gets a contiguous run of tiles, four tiles of q deep, so that the tiles that
// share an XCD's L2 share panels of both operands.
__device__ __forceinline__ void product_tile(int w, int np, int nq, int &tp, int &tq)
{
    const int total = np * nq;
    const int whole = total / 8 * 8;
    if (w < whole)
        w = (w % 8) * (total / 8) + w / 8;
    constexpr int DEEP = 4;
    const int first = w / (DEEP * np) * DEEP;
    const int deep = min(nq - first, DEEP);
    const int loc = w - first * np;
    tq = first + loc % deep;
    tp = loc / deep;
}

}  // namespace mxq
