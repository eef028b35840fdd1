// gemm_block128.hip -- grouped products of E4M3 operands with one FP32 scale per 128 (rows) and per
// 128 x 128 (weights) on gfx950:
//
//   D[r][n] = sum over groups g of 128 of K   xs[g][r] ws_e[n/128][g]  sum_k P_e[n][k] Q[r][k]
//
// for the rows r of each expert e (m_indptr), P_e its matrix of codes [Np, K] and Q the rows' codes:
//
//   mode       P                          Q                      K    output
//   B128_W13   W13_e, gate/up row pairs   xq[gather[r]]          d    a = f(g) u quantized along I: codes [R, I],
//                                                                     scales [I/128, R]
//   B128_W2    W2_e rows                  aq[r]                  I    o in FP16, in units of a power of two that puts the
//                                                                     largest of a row's block of 128 into 2^14 .. 2^15:
//                                                                     [R, d], [R, d/128].  Within 2^-11 of each value
//                                                                     down to a 2^-29th of the block's largest, in as many bytes
//                                                                     as BF16 (2^-8).  (Integers in units of the largest are
//                                                                     closer where all are of one size, but lose the
//                                                                     others beside one 2^12 times as large: 3.5e-2)
//   B128_PLAIN rows of a matrix           routed rows            Kp   BF16 [R, Np]: a product's forward and input gradient,
//                                                                     W2 of rows in expert order
//
// The inner sum is one v_mfma_f32_16x16x128_f8f6f4 with a zero third operand; its four results a
// lane are multiplied with their scale and added in FP32.  The rows are the instruction's columns: a
// lane's results belong to one row, and to one 128 x 128 square of P, so that they share one factor.
// The vector unit's four FMAs take half the time of the instruction.  Accumulators are operands of
// the vector unit and lie in its registers, which limits a wave to 128 x 64 outputs (the MXFP8
// products, whose scales the matrix unit applies, have 128 x 128).
//
// Workgroup tile 256 (P) x TQ (rows: 256, 192 or 128), eight waves of 128 x TQ / 4, a stage of 128 K in LDS while the next one
// is copied into the other buffer by direct global-to-LDS copies, one continuous stream of stages per
// workgroup over its tiles (the next tile's first stage is copied during the last of this one).
// LDS rows are 128 bytes, 16-byte chunk c of row r at slot c ^ (r / 2 % 8): the same chunk of 16
// consecutive rows, which a quarter of a wave reads, meets all 64 banks once.  (At slot c ^ (r & 7) half of the
// reads' cycles were conflicts.)
//
// Bound by the matrix unit at the clock that its power leaves and by the copies and LDS reads beside it.  16384 tokens of 4096 x
// 2048, 64 experts, k = 8: W13 2.12 ms, W2 1.19 ms, 2.08 and 1.85 PFLOP/s (matrix unit busy 54 and 48 % at 1.9 GHz);
// 65536 rows of 4096 x 4096 1.05 to 1.09 ms, 2.0-2.1 PFLOP/s (59 % at 1.6 GHz); 8192 tokens of 2048 x 768, 16 experts: 227 and 132 us
// (44 and 36 % at 2.0 and 2.1 GHz), where a tile's few stages (16 and 6) leave its epilogue a larger share.
#include "block128.h"

namespace moe {
namespace {

constexpr int TP = 256, TK = 128;
constexpr int kPBytes = TP * TK;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
// two floats in FP16, nearest even, the first in the low half
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const f32x2_t v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

// Order of an expert's tiles: as in the MXFP8 products, groups of kQGroup row tiles, inside a group
// the P tiles with the group's row tiles fastest, so that the tiles that an XCD runs at a time share
// operands in its L2.
constexpr int kQGroup = 6;
__device__ __forceinline__ void tile_order(int local, int nQt, int nPt, int& pt, int& qt) {
    const int gi = local / (kQGroup * nPt);
    const int rem = local - gi * kQGroup * nPt;
    const int left = nQt - gi * kQGroup;
    const int gsz = left < kQGroup ? left : kQGroup;
    pt = rem / gsz;
    qt = gi * kQGroup + (rem - pt * gsz);
}

struct Tile {
    int e, mb, rows, pt, qt;
};
__device__ __forceinline__ int swz(int r) { return r >> 1 & 7; }

template <int MODE, int kAct, int TQ>
__global__ __launch_bounds__(512, 1) void grouped_gemm_b128(Block128GemmArgs g) {
    constexpr int kWaves = 8, kThr = kWaves * MOE_WAVE;
    constexpr int kNB = TQ / 64;                         // fragments of 16 rows a wave
    constexpr int kBuf = kPBytes + TQ * TK;              // a stage: P then Q
    constexpr int kSlot = TQ * 4 + 256;                  // its scales: TQ words of Q, 64 of P
    constexpr int kPCopies = kPBytes / 1024 / kWaves, kQCopies = kNB;          // of 1 KiB a wave
    __shared__ __attribute__((aligned(1024))) char lds[2 * kBuf];
    __shared__ __attribute__((aligned(1024))) char lsc[2 * kSlot];
    __shared__ uint32_t tops[2][TQ];                     // B128_W13: magnitudes of a row's two halves
    __shared__ int cum[257], mptr[257];
    __shared__ int gsrc[2][TQ];                          // B128_W13: tokens of the next two tiles' rows
    __shared__ int wtot[4];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = wave & 1, wq = wave >> 1;
    // The lane id read afresh where code runs once per tile: offsets that depend on it, hoisted out of the loop
    // over tiles, would be spilled, and a reload waits for every copy in flight.
    auto fresh_lane = []() {
        int l;
        asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
        return l;
    };
    const int E = g.E, K = g.K, groups = K / TK;
    const int nPt = MODE == B128_W13 ? g.Np / 128 : (g.Np + TP - 1) / TP;
    const int prows = MODE == B128_W13 ? 2 * g.Np : g.Np;        // P rows of an expert

    // ---- tiles of expert e are cum[e] .. cum[e+1]-1
    for (int i = tid; i <= E; i += kThr) mptr[i] = g.m_indptr ? g.m_indptr[i] : i == 0 ? 0 : (int)g.R;
    __syncthreads();
    if (g.check) {
        const bool bad = tid <= E && (tid == 0 ? mptr[0] != 0 : mptr[tid] < mptr[tid - 1] || mptr[tid] > (int)g.R);
        if (__syncthreads_or(bad)) {
            if (blockIdx.x == 0 && tid == 0 && g.status) atomicOr(g.status, kDevBadIndptr);
            return;
        }
    }
    if (tid < 256) {
        int incl = tid < E ? (mptr[tid + 1] - mptr[tid] + TQ - 1) / TQ * nPt : 0;
        for (int off = 1; off < MOE_WAVE; off <<= 1) {
            const int u = __shfl_up(incl, off, MOE_WAVE);
            if (lane >= off) incl += u;
        }
        if (lane == MOE_WAVE - 1) wtot[wave] = incl;
        cum[tid + 1] = incl;
    }
    if (tid == 0) cum[0] = 0;
    __syncthreads();
    if (tid < 256)
        for (int w = 0; w < wave; ++w) cum[tid + 1] += wtot[w];
    __syncthreads();
    const int total = cum[E], G = gridDim.x;
    const int vid = (G % 8 == 0) ? (int)(blockIdx.x % 8) * (G / 8) + (int)(blockIdx.x / 8) : (int)blockIdx.x;
    if (vid >= total) return;

    auto coords = [&](int tile) {
        // largest e with cum[e] <= tile = number of e in [1, E) with cum[e] <= tile
        const int lane = fresh_lane();
        int lo = 0;
#pragma unroll
        for (int base = 1; base < 257; base += 64) {
            const int e = base + lane;
            lo += __builtin_popcountll(__ballot(e < E && cum[e] <= tile));
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        Tile c;
        c.e = lo;
        c.mb = __builtin_amdgcn_readfirstlane(mptr[lo]);
        c.rows = __builtin_amdgcn_readfirstlane(mptr[lo + 1]) - c.mb;
        tile_order(tile - __builtin_amdgcn_readfirstlane(cum[lo]), (c.rows + TQ - 1) / TQ, nPt, c.pt, c.qt);
        return c;
    };
    // row of P behind tile row r.  A wave's 32 rows follow one another, or are 16 and 16.
    auto p_row = [&](const Tile& c, int r) {
        if constexpr (MODE == B128_W13) {
            // 16-row pieces: gate rows 128 pt + 16 j .., then the up rows of the same outputs
            const int i = c.pt * 128 + (r >> 5) * 16 + (r & 15);
            return (r & 16) ? g.Np + i : i;
        } else {
            // a second half past the last row is the first again
            return c.pt * TP + (c.pt * TP + 128 < g.Np ? r : r & 127);
        }
    };
    // routed row behind tile row r (clamped to the expert's last)
    auto routed_row = [&](const Tile& c, int r) {
        const int rr = c.qt * TQ + r;
        return c.mb + (rr < c.rows ? rr : c.rows - 1);
    };

    // ------------------------------------------------------------ copies
    const uint32_t lds0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)lds;
    const uint32_t lsc0 = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)lsc;
    auto dma16 = [&](uint32_t dst, uint32_t voff, const char* base) {
        asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :: "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(voff), "s"(base) : "memory");
    };
    auto dma4 = [&](uint32_t dst, uint32_t voff, const char* base) {
        asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2"
                     :: "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(voff), "s"(base) : "memory");
    };
    // A wave copies the tokens of the rows whose data it copies itself, a tile ahead.
    auto gather_dma = [&](const Tile& c, int slot) {
        if constexpr (MODE == B128_W13) {
            const int lane = fresh_lane();
            const int r = 8 * kQCopies * wave + lane % (8 * kQCopies);
            const uint32_t dst = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) int*)&gsrc[slot][8 * kQCopies * wave];
            if (lane < 8 * kQCopies) dma4(dst, (uint32_t)routed_row(c, r) * 4u, reinterpret_cast<const char*>(g.gather));
        }
    };
    // Data: a wave copies consecutive 1 KiB pieces of either operand; lane l fetches 16 bytes that land
    // at piece + 16 l = row l / 8 of the piece, slot l % 8.  Scales: waves 0 .. TQ/64 - 1 one word
    // each of 64 rows, the others the words of the two squares of P that the tile meets.
    static_assert(kPCopies == 4, "32 rows a wave");
    uint32_t pvoff[2], qvoff[kQCopies], svoff;           // P: of even and odd pieces, the others by scalar offsets
    const char *pbase = nullptr, *qbase = nullptr, *sbase = nullptr;
    const bool q_scales = wave < TQ / 64;
    size_t sstep = 0;                                    // bytes between the scales of consecutive groups
    auto copy_offsets = [&](const Tile& c, int slot) {
        const int lane = fresh_lane();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * (kPCopies * wave + j) + (lane >> 3);
            pvoff[j] = (uint32_t)p_row(c, r) * (uint32_t)K + 16 * ((lane & 7) ^ swz(r));
        }
#pragma unroll
        for (int j = 0; j < kQCopies; ++j) {
            const int r = 8 * (kQCopies * wave + j) + (lane >> 3);
            const int src = MODE == B128_W13 ? gsrc[slot][r] : routed_row(c, r) - (c.mb + c.qt * TQ);
            qvoff[j] = (uint32_t)src * (uint32_t)K + 16 * ((lane & 7) ^ swz(r));
        }
        qbase = reinterpret_cast<const char*>(g.qq);
        if constexpr (MODE != B128_W13) qbase += (size_t)(c.mb + c.qt * TQ) * K;
        pbase = reinterpret_cast<const char*>(g.pq + (size_t)c.e * prows * K);
        if (q_scales) {
            svoff = (uint32_t)routed_row(c, 64 * wave + lane) * 4u;
            sbase = reinterpret_cast<const char*>(g.qs);
            sstep = (size_t)g.R * 4;
        } else {
            int b = MODE == B128_W13 ? (lane & 1) * (g.Np / 128) + c.pt : 2 * c.pt + (lane & 1);
            if (b >= prows / 128) b = prows / 128 - 1;
            svoff = (uint32_t)(b * groups) * 4u;
            sbase = reinterpret_cast<const char*>(g.ps + (size_t)c.e * (prows / 128) * groups);
            sstep = 4;
        }
    };
    auto dma_p = [&](int kt, int buf, int j) {
        const size_t rows16 = (size_t)(MODE == B128_W13 ? g.Np : 16) * K;
        dma16(lds0 + buf * kBuf + (kPCopies * wave + j) * 1024, pvoff[j & 1], pbase + kt * TK + (j >> 1) * rows16);
    };
    auto dma_q = [&](int kt, int buf, int j) {
        dma16(lds0 + buf * kBuf + kPBytes + (kQCopies * wave + j) * 1024, qvoff[j], qbase + kt * TK);
    };
    auto dma_scales = [&](int kt, int buf) {
        dma4(lsc0 + buf * kSlot + (q_scales ? 256 * wave : TQ * 4), svoff, sbase + kt * sstep);
    };

    // ------------------------------------------------------------ a stage
    const int row16 = lane & 15, quad = lane >> 4;
    // a fragment: 16 rows, lane (row16, quad) the chunks quad and quad + 4 of its row
    const int c0 = (quad ^ swz(row16)) * 16, c1 = c0 ^ 64;
    const int poff = (wp * 128 + row16) * TK, qoff = kPBytes + (wq * 16 * kNB + row16) * TK;
    auto read_frag = [&](const char* row) {
        const i32x4_t x = *reinterpret_cast<const i32x4_t*>(row + c0);
        const i32x4_t y = *reinterpret_cast<const i32x4_t*>(row + c1);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    f32x4_t acc[8][kNB];
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    i32x8_t qf[kNB], pf;                                   // the rows' fragments, the next one of P
    float sq[kNB], sp[2];                                  // scales: of this lane's rows, of the wave's squares of P
    auto read_q = [&](int buf, int b) {
        qf[b] = read_frag(lds + buf * kBuf + qoff + b * 16 * TK);
        sq[b] = reinterpret_cast<const float*>(lsc + buf * kSlot)[wq * 16 * kNB + b * 16 + row16];
    };
    auto read_p = [&](int buf, int a) { return read_frag(lds + buf * kBuf + poff + a * 16 * TK); };
    auto read_sp = [&](int buf) {
        const float* sc = reinterpret_cast<const float*>(lsc + buf * kSlot) + TQ;
        sp[0] = sc[MODE == B128_W13 ? 0 : wp];
        sp[1] = MODE == B128_W13 ? sc[1] : sp[0];
    };
    auto read_first = [&](int buf) {
        pf = read_p(buf, 0);
        read_sp(buf);
#pragma unroll
        for (int b = 0; b < kNB; ++b) read_q(buf, b);
    };
    // One stage from buffer buf, whose first fragments have been read: eight steps of one fragment of P.  A step
    // issues its four products, each followed by the FMAs of the step before, reads the next fragment and
    // issues copies of the stage at next_kt into the other buffer.  Before the last step everything of
    // this buffer has been read and the next stage has landed (a barrier); unless the tile ends, that
    // step reads the next stage's first fragments.
    auto stage = [&](auto last_tag, int buf, int next_kt) {
        constexpr bool kLast = decltype(last_tag)::value;
        float f0[kNB], f1[kNB];                              // factors; B128_W13: of gate and up rows
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            f0[b] = sq[b] * sp[0];
            f1[b] = MODE == B128_W13 ? sq[b] * sp[1] : f0[b];
        }
        f32x4_t part[kNB];
#pragma unroll
        for (int a = 0; a < 8; ++a) {
            i32x8_t pn = pf;
            if (a == 7) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
                if constexpr (!kLast) {
                    pn = read_p(buf ^ 1, 0);
                    read_sp(buf ^ 1);
                }
            } else {
                pn = read_p(buf, a + 1);
            }
#pragma unroll
            for (int b = 0; b < kNB; ++b) {
                const f32x4_t now = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf, qf[b], zero, 0, 0, 0, 0, 0, 0);
                // the last fragment's results, while this one's are computed
                if (a > 0)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        acc[a - 1][b][z] = __builtin_fmaf(part[b][z], (a - 1) & 1 ? f1[b] : f0[b], acc[a - 1][b][z]);
                // neither the products nor the FMAs have an ordering edge to anything here and would be
                // emitted all together: an empty asm that takes their results keeps them in this step
                asm volatile("" :: "v"(now));
                if (a > 0) asm volatile("" : "+v"(acc[a - 1][b]));
                part[b] = now;
                if constexpr (!kLast) {
                    if (a == 7) read_q(buf ^ 1, b);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                if (b == (kNB > 2 ? 1 : 0) && a < kPCopies) dma_p(next_kt, buf ^ 1, a);
                if (b == kNB - 1 && a < kQCopies) dma_q(next_kt, buf ^ 1, a);
                if (b == kNB - 1 && a == 4) dma_scales(next_kt, buf ^ 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            pf = pn;
        }
#pragma unroll
        for (int b = 0; b < kNB; ++b)
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[7][b][z] = __builtin_fmaf(part[b][z], f1[b], acc[7][b][z]);
    };

    // ------------------------------------------------------------ epilogues
    // buf: the buffer that the tile's last stage has been read from
    auto epilogue_w13 = [&](const Tile& c, int buf) {
        // a = f(g) u: fragments 2 m hold gate values, 2 m + 1 the up values of the same outputs,
        // i = 128 pt + 64 wp + 16 m + 4 quad + z of row 64 wq + 16 b + row16
        const int lane = fresh_lane(), row16 = lane & 15, quad = lane >> 4;
        char* stg = lds + buf * kBuf;                    // codes [TQ][128], chunks as the stages'
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            uint32_t top = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const float v = act_f<kAct>(acc[2 * m][b][z]) * acc[2 * m + 1][b][z];
                    acc[2 * m][b][z] = v;
                    const uint32_t t = __float_as_uint(v) & 0x7FFFFFFFu;
                    top = top > t ? top : t;
                }
#pragma unroll
            for (int o = 16; o < 64; o <<= 1) {
                const uint32_t t = __shfl_xor(top, o, MOE_WAVE);
                top = top > t ? top : t;
            }
            if (lane < 16) tops[wp][wq * 16 * kNB + b * 16 + row16] = top;
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            const int r = wq * 16 * kNB + b * 16 + row16;
            const uint32_t t0 = tops[0][r], t1 = tops[1][r];
            const float s = block_scale(t0 > t1 ? t0 : t1), inv = block_inverse(s);
#pragma unroll
            for (int m = 0; m < 4; ++m)
                *reinterpret_cast<uint32_t*>(stg + r * 128 + (((4 * wp + m) ^ swz(r)) * 16) + 4 * quad) =
                    block_codes4(acc[2 * m][b][0], acc[2 * m][b][1], acc[2 * m][b][2], acc[2 * m][b][3], s, inv);
            const int rr = c.qt * TQ + r;
            if (wp == 0 && quad == 0 && rr < c.rows) g.as[(size_t)c.pt * g.R + c.mb + rr] = s;
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < TQ / (8 * kWaves); ++it) {
            const int r = (it * kWaves + wave) * 8 + (lane >> 3), ch = lane & 7, rr = c.qt * TQ + r;
            const uint4 v = *reinterpret_cast<const uint4*>(stg + r * 128 + ((ch ^ swz(r)) * 16));
            if (rr < c.rows) *reinterpret_cast<uint4*>(g.aq + (size_t)(c.mb + rr) * g.Np + c.pt * 128 + ch * 16) = v;
        }
    };
    auto epilogue_rows = [&](const Tile& c, int buf) {
        // rows in BF16 (B128_W2: scaled FP16) by way of this wave's 4 KiB of the buffer, 16 at a time, stored as
        // whole 256-byte pieces past the caches (ordinary stores evict operands that the XCD's workgroups share)
        const int lane = fresh_lane(), row16 = lane & 15, quad = lane >> 4;
        char* stg = lds + buf * kBuf + wave * 4096;
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
            float inv = 0.f;
            if constexpr (MODE == B128_W2) {
                uint32_t top = 0;
#pragma unroll
                for (int a = 0; a < 8; ++a)
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const uint32_t t = __float_as_uint(acc[a][b][z]) & 0x7FFFFFFFu;
                        top = top > t ? top : t;
                    }
#pragma unroll
                for (int o = 16; o < 64; o <<= 1) {
                    const uint32_t t = __shfl_xor(top, o, MOE_WAVE);
                    top = top > t ? top : t;
                }
                // the unit's exponent, biased: at least 1, so that neither it nor its inverse is a denormal.  128 that
                // hold an infinity or NaN are NaN.
                const uint32_t e = top >> 23, ue = (e > 15u ? e : 15u) - 14u;
                inv = __uint_as_float((254u - ue) << 23);
                const float unit = __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : ue << 23);
                const int rr = c.qt * TQ + wq * 16 * kNB + b * 16 + row16, p = c.pt * TP + wp * 128;
                if (quad == 0 && rr < c.rows && p < g.Np) g.os[(size_t)(c.mb + rr) * (g.Np / 128) + p / 128] = unit;
            }
            auto pack = [&](float x, float y) {
                if constexpr (MODE == B128_W2) return pack_f16(x * inv, y * inv);
                else return pack_bf16(x, y);
            };
#pragma unroll
            for (int a = 0; a < 8; ++a) {
                const f32x4_t v = acc[a][b];
                const int c16 = 2 * a + (quad >> 1);
                *reinterpret_cast<uint2*>(stg + row16 * 256 + ((c16 ^ row16) * 16) + 8 * (quad & 1)) =
                    make_uint2(pack(v[0], v[1]), pack(v[2], v[3]));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int r = 4 * it + quad, c16 = row16;
                const uint4 v = *reinterpret_cast<const uint4*>(stg + r * 256 + ((c16 ^ r) * 16));
                const int rr = c.qt * TQ + wq * 16 * kNB + b * 16 + r, p = c.pt * TP + wp * 128 + 8 * c16;
                if (rr < c.rows && p < g.Np) store_nt(g.out + (size_t)(c.mb + rr) * g.Np + p, v);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    };

    // ------------------------------------------------------------ stream of stages
    int l_tile = vid, l_kt = 0, gslot = 0;               // the load cursor
    Tile lc = coords(l_tile), nc = lc;
    gather_dma(lc, 0);
    if (l_tile + G < total) { nc = coords(l_tile + G); gather_dma(nc, 1); }
    if constexpr (MODE == B128_W13) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    copy_offsets(lc, 0);
    auto advance_load = [&]() {
        if (++l_kt < groups) return;
        if (l_tile + G >= total) { l_kt = groups - 1; return; }      // past the end: the last stage again
        // the new tile's tokens were copied at the last switch, at least a stage's wait ago
        l_kt = 0;
        l_tile += G;
        gslot ^= 1;
        lc = nc;
        copy_offsets(lc, gslot);
        if (l_tile + G < total) { nc = coords(l_tile + G); gather_dma(nc, gslot ^ 1); }
    };
    dma_scales(0, 0);
#pragma unroll
    for (int j = 0; j < kPCopies; ++j) dma_p(0, 0, j);
#pragma unroll
    for (int j = 0; j < kQCopies; ++j) dma_q(0, 0, j);
    advance_load();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();

    Tile cc = coords(vid);
    int buf = 0;
    read_first(0);
    for (int c_tile = vid;;) {
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int b = 0; b < kNB; ++b) acc[a][b] = zero;
        for (int kt = 1; kt < groups; ++kt) {
            stage(std::false_type(), buf, l_kt);
            advance_load();
            buf ^= 1;
        }
        stage(std::true_type(), buf, l_kt);
        advance_load();
        if constexpr (MODE == B128_W13) epilogue_w13(cc, buf);
        else epilogue_rows(cc, buf);
        buf ^= 1;
        c_tile += G;
        if (c_tile >= total) break;
        __syncthreads();                                 // the staging rows are copied into again
        cc = coords(c_tile);
        read_first(buf);
    }
}

template <int MODE, int kAct, int TQ> hipError_t launch_t(const Block128GemmArgs& g, int num_cu, hipStream_t s) {
    const int64_t nPt = MODE == B128_W13 ? g.Np / 128 : (g.Np + TP - 1) / TP;
    int64_t grid = (g.R / TQ + (g.E < g.R ? g.E : g.R)) * nPt;       // tiles, at most
    grid = grid < num_cu ? grid : num_cu;
    if (grid >= 8) grid -= grid % 8;
    hipLaunchKernelGGL((grouped_gemm_b128<MODE, kAct, TQ>), dim3((unsigned)(grid < 1 ? 1 : grid)), dim3(512), 0, s, g);
    return hipGetLastError();
}

template <int TQ> hipError_t launch_act(Block128Mode mode, const Block128GemmArgs& g, int num_cu, hipStream_t s) {
    if (mode == B128_PLAIN) return launch_t<B128_PLAIN, kActSwiGLU, TQ>(g, num_cu, s);
    if (mode == B128_W2) return launch_t<B128_W2, kActSwiGLU, TQ>(g, num_cu, s);
    if (g.act == kActGeGLU) return launch_t<B128_W13, kActGeGLU, TQ>(g, num_cu, s);
    if (g.act == kActReGLU) return launch_t<B128_W13, kActReGLU, TQ>(g, num_cu, s);
    return launch_t<B128_W13, kActSwiGLU, TQ>(g, num_cu, s);
}

// y[t] = sum_j s[t][j] o[slots[t][j]] in FP32, j ascending from +0.0, of o in scaled FP16; eight columns a thread.  Reading
// o is its time: 65536 rows of 2048 52 us, 268 MB at 5.1 TB/s (58 with loads that stay in the caches).
__global__ __launch_bounds__(256) void combine16_kernel(MxGemmArgs g) {
    const int t = blockIdx.x, c = blockIdx.y * 256 + threadIdx.x, d = g.d;
    if (8 * c >= d) return;
    float y[8] = {};
#pragma unroll 8
    for (int j = 0; j < g.k; ++j) {
        const size_t r = (size_t)g.slots[(size_t)t * g.k + j];
        const u32x4_t u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(g.o + r * d + 8 * c));
        const float f = g.os[r * (d / 128) + c / 16], w = g.scores[(size_t)t * g.k + j];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const uint32_t word = u[z];                  // (a bit cast of u[z] itself takes u[0])
            const f16x2_t h = __builtin_bit_cast(f16x2_t, word);
            y[2 * z] = __builtin_fmaf(w, f * (float)h[0], y[2 * z]);
            y[2 * z + 1] = __builtin_fmaf(w, f * (float)h[1], y[2 * z + 1]);
        }
    }
    *reinterpret_cast<uint4*>(g.y + (size_t)t * d + 8 * c) =
        make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
}

// Rows of a tile: those with which the tiles' rounds over the chip take the least time, when one of 256 rows takes 1.
// The rows of several experts are taken to fill their last tiles by half, and their rounds, whose number is
// not known here, are not rounded up.  (4096 outputs of 2048 inputs: 2000 rows
// 36.2, 33.2 and 30.2 us with 256, 192 and 128, 6000 rows 72.5, 64.2 and 70.9, 20000 rows 182, 194 and 218; 128
// experts, 2048 routed rows in all: 152, 142 and 129.)
int rows_of_tile(Block128Mode mode, const Block128GemmArgs& g, int num_cu) {
    const int64_t nPt = mode == B128_W13 ? g.Np / 128 : (g.Np + TP - 1) / TP;
    int best = 256;
    float least = 0.f;
    for (int tq = 256; tq >= 128; tq -= 64) {
        const int64_t tiles = g.E == 1 ? (g.R + tq - 1) / tq : g.R / tq + (g.E < g.R ? g.E : g.R) / 2 + 1;
        float t = (float)(tiles * nPt) / (float)num_cu;
        t = g.E == 1 ? (float)((tiles * nPt + num_cu - 1) / num_cu) : t > 1.0f ? t : 1.0f;
        t *= tq == 256 ? 1.0f : tq == 192 ? 0.88f : 0.7f;
        if (tq == 256 || t < least) { least = t; best = tq; }
    }
    return best;
}

}  // namespace

hipError_t launch_gemm_block128(Block128Mode mode, const Block128GemmArgs& g, int num_cu, hipStream_t s) {
    if (g.E <= 0 || g.E > 256 || (!g.m_indptr && g.E != 1) || g.R < 0 || g.R > 0x7FFFFFFF || g.K <= 0 || g.K % 128 != 0 || g.Np <= 0 || g.Np % 128 != 0) return hipErrorInvalidValue;
    if (g.R == 0) return hipSuccess;
    switch (rows_of_tile(mode, g, num_cu)) {
        case 128: return launch_act<128>(mode, g, num_cu, s);
        case 192: return launch_act<192>(mode, g, num_cu, s);
        default: return launch_act<256>(mode, g, num_cu, s);
    }
}

// The layer's forward: x in 8 bits with its scales by routed row, W13, W2, the combine
hipError_t launch_layer_block128(MxMode mode, const MxGemmArgs& g, int num_cu, hipStream_t s) {
    const int64_t R = (int64_t)g.T * g.k;
    if (mode == MX_QUANT_X) {
        uint8_t* xq = const_cast<uint8_t*>(g.xq);
        float* xs = reinterpret_cast<float*>(const_cast<uint8_t*>(g.xs));
        if (!g.xs_rows) return launch_block128_rows(g.x, R, g.d, xq, xs, true, g.m_indptr + g.E, s);
        const hipError_t e = launch_block128_rows(g.x, g.T, g.d, xq, reinterpret_cast<float*>(g.xs_rows), false, nullptr, s);
        // (the scales of 128 values are a word, as four MX scales are)
        return e != hipSuccess ? e : launch_route_scales(g.xs_rows, g.T, g.gather, R, g.d, const_cast<uint8_t*>(g.xs), s);
    }
    Block128GemmArgs b{};
    b.E = g.E; b.R = R; b.m_indptr = g.m_indptr; b.act = g.act;
    if (mode == MX_W13) {
        b.K = g.d; b.Np = g.I; b.gather = g.gather;
        b.pq = g.w13q; b.ps = reinterpret_cast<const float*>(g.w13s);
        b.qq = g.xq; b.qs = reinterpret_cast<const float*>(g.xs);
        b.aq = g.aq; b.as = reinterpret_cast<float*>(g.as);
        return launch_gemm_block128(B128_W13, b, num_cu, s);
    }
    if (mode == MX_COMBINE) {
        if (g.T > 0) hipLaunchKernelGGL(combine16_kernel, dim3(g.T, (g.d / 8 + 255) / 256), dim3(g.d < 2048 ? (g.d / 8 + 63) & ~63 : 256), 0, s, g);
        return hipGetLastError();
    }
    if (mode != MX_W2) return hipErrorInvalidValue;
    b.K = g.I; b.Np = g.d;
    b.pq = g.w2q; b.ps = reinterpret_cast<const float*>(g.w2s);
    b.qq = g.aq; b.qs = reinterpret_cast<const float*>(g.as);
    b.out = g.o; b.os = g.os;
    return launch_gemm_block128(g.os ? B128_W2 : B128_PLAIN, b, num_cu, s);
}

}  // namespace moe
