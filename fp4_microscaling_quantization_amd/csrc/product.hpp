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

    // fragment t (rows 16 t ..) of the tile at `lds`
    static __device__ __forceinline__ v8bf fragment(const uint8_t *lds, int t, int lane)
    {
        const int g = lane >> 4, li = lane & 15;
        if constexpr (ALONG) {
            return *reinterpret_cast<const v8bf *>(lds + t * 1024 + li * 64 +
                                                   ((g ^ (li >> 2)) * 16));
        } else {
            typedef __attribute__((address_space(3))) v4s lds_v4s;
            v4s h[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k = 8 * g + 4 * u + (li >> 2);
                const int chunk = (2 * t + ((li >> 1) & 1)) ^ turn(k);
                const uint8_t *at = lds + k * (ROWS * 2) + chunk * 16 + (li & 1) * 8;
                h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_v4s *)(__attribute__((address_space(3))) uint8_t *)at);
            }
            typedef short v8s __attribute__((ext_vector_type(8)));
            return __builtin_bit_cast(v8bf, (v8s)__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// A workgroup of WP x WQ waves, each with NP x NQ tiles of 16 x 16.
template <int WP_, int WQ_, int NP_, int NQ_, bool P_ALONG, bool Q_ALONG> struct Product {
    static constexpr int WP = WP_, WQ = WQ_, NP = NP_, NQ = NQ_;
    static constexpr int kP = 16 * WP * NP, kQ = 16 * WQ * NQ, kWaves = WP * WQ;
    static constexpr int kThreads = 64 * kWaves;
    using SideP = Side<kP, P_ALONG>;
    using SideQ = Side<kQ, Q_ALONG>;
    static constexpr int kStage = SideP::kBytes + SideQ::kBytes;
    static constexpr int kStages = 2;
    static constexpr int kLds = kStages * kStage;
    static constexpr int kPer = (SideP::kChunks + SideQ::kChunks) / kWaves;
    static_assert(kPer * kWaves == SideP::kChunks + SideQ::kChunks, "copies split evenly");

    v4f acc[NP][NQ];
    int lane, wave, wp, wq;
    uint32_t off[kPer];
    int cut_step = -1, cut_have, cut_rows;  // (P across k) a last step with fewer k
    int64_t cut_ld;

    // p, q: where the tile's first elements lie, with their leading dimensions and how
    // many rows there are from there
    __device__ __forceinline__ void start(int64_t ldp, int have_p, int64_t ldq, int have_q)
    {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        wp = wave % WP;
        wq = wave / WP;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = wave * kPer + i;
            off[i] = c < SideP::kChunks ? SideP::offset(c, lane, ldp, have_p)
                                        : SideQ::offset(c - SideP::kChunks, lane, ldq, have_q);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    // P across k: there are k_left values of k; Q is zero in a last step that is not whole
    __device__ __forceinline__ void cut_p(int k_left, int64_t ldp, int have_p)
    {
        if (k_left % kStepK) {
            cut_step = k_left / kStepK;
            cut_have = k_left % kStepK;
            cut_rows = have_p;
            cut_ld = ldp;
        }
    }
    __device__ __forceinline__ void copy(int s, const uint8_t *p, const uint8_t *q, uint8_t *to)
    {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = wave * kPer + i;
            uint32_t o = off[i];
            if constexpr (!P_ALONG)
                if (s == cut_step && c < SideP::kChunks)
                    o = SideP::offset(c, lane, cut_ld, cut_rows, cut_have);
            dma16_so(c < SideP::kChunks ? p : q, o, to + c * 1024);
        }
    }
    // `steps` steps; at_p(s), at_q(s): the (uniform) address of step s's tiles
    template <class AtP, class AtQ>
    __device__ __forceinline__ void run(uint8_t *lds, int steps, AtP at_p, AtQ at_q)
    {
        if (steps > 0)
            copy(0, at_p(0), at_q(0), lds);
        for (int s = 0; s < steps; ++s) {
            // this wave's copies of the step landed and its reads of the one before are done
            __builtin_amdgcn_s_waitcnt(0x0070);
            barrier_no_fence();
            if (s + 1 < steps)
                copy(s + 1, at_p(s + 1), at_q(s + 1), lds + ((s + 1) & 1) * kStage);
            const uint8_t *from = lds + (s & 1) * kStage;
            v8bf fp[NP], fq[NQ];
#pragma unroll
            for (int j = 0; j < NQ; ++j)
                fq[j] = SideQ::fragment(from + SideP::kBytes, wq * NQ + j, lane);
#pragma unroll
            for (int i = 0; i < NP; ++i)
                fp[i] = SideP::fragment(from, wp * NP + i, lane);
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j < NQ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[i], fq[j], acc[i][j], 0, 0, 0);
        }
    }
    // p of acc[i][.][0] and q of acc[.][j] within the tile
    __device__ __forceinline__ int p_of(int i) const { return 16 * (wp * NP + i) + 4 * (lane >> 4); }
    __device__ __forceinline__ int q_of(int j) const { return 16 * (wq * NQ + j) + (lane & 15); }
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
