// decode_mxfp4.hip -- weight-streaming path for expert weights in MXFP4 (mxfp4.hip's layout),
// T*k <= 256 routed rows.
//
// The same launches as with BF16 weights (decode.hip): W13 with the activation, then for one
// token W2 with the combine, else W2 and the combine kernel; a and o are rounded to BF16 at the
// same points.  The time is that of streaming 4.25 bits for each weight of the active experts.
//
// A wave reads a tile (16 weight rows x 128 of K, 1 KiB in a row) with one 16-byte load per
// lane: lane 16 q + n holds the block of 32 columns 128 s + 32 q of row n, with one scale.
// v_cvt_scalef32_pk_bf16_fp4 turns each quarter (8 codes, four conversions) with the scale into
// the exact BF16 B operand of a v_mfma_f32_16x16x32_bf16, so products and sums are those of
// the expanded BF16 weights.  The MFMA's own order of K is free as long as both operands
// agree: lane (m, q) of the A operand of quarter i holds columns 128 s + 32 q + 8 i .. + 7 of
// routed row m.
#include "decode_common.h"

namespace moe {
namespace {

constexpr int kB = 4;                // tiles along K with loads in flight per wave

// Scales of tiles s .. s + 3 of this lane's block, one byte each, from the words of a row tile
__device__ __forceinline__ uint32_t scale_bytes(const uint32_t* words, int s, int groups) {
    const int g0 = s >> 2, g1 = g0 + 1 < groups ? g0 + 1 : g0;
    const uint32_t lo = words[g0 * 64], hi = words[g1 * 64];
    return __builtin_amdgcn_alignbit(hi, lo, 8 * (s & 3));
}

// acc += A * B over the tiles s0 .. s1 - 1: codes and words point at this lane's piece of the
// row tile's first tile, ars / ao as for mma_line_pairs (the row's byte offset; kNoRow: zeros)
template <int B>
__device__ __forceinline__ f32x4_t mma_tiles(const uint8_t* codes, const uint32_t* words, int groups,
                                             __amdgpu_buffer_rsrc_t ars, uint32_t ao, int s0, int s1) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    ao += 64u * ((threadIdx.x & 63) >> 4);
    for (int s = s0; s < s1; s += B) {
        u32x4_t c[B];
        bf16x8_t a[B][4];
        uint32_t sb[(B + 3) / 4];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s + j < s1) c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + (size_t)(s + j) * 1024));
#pragma unroll
        for (int j = 0; j < B; j += 4)
            if (s + j < s1) sb[j / 4] = scale_bytes(words, s + j, groups);
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s + j < s1)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[j][i] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                               ars, ao + 256u * (uint32_t)(s + j) + 16u * i, 0, 0));
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s + j < s1) {
                const float x = __uint_as_float(((sb[j / 4] >> (8 * (j & 3))) & 0xFFu) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bf16x2_t w0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j][i], x, 0);
                    const bf16x2_t w1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j][i], x, 1);
                    const bf16x2_t w2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j][i], x, 2);
                    const bf16x2_t w3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[j][i], x, 3);
                    const bf16x8_t w = {w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j][i], w, acc, 0, 0, 0);
                }
            }
    }
    return acc;
}

// K split: wave w takes the tiles [S w / 4, S (w + 1) / 4)
template <bool kSplit> __device__ __forceinline__ void wave_tiles(int S, int& s0, int& s1) {
    const int w = threadIdx.x >> 6;
    s0 = kSplit ? __builtin_amdgcn_readfirstlane(S * w / kWaves) : 0;
    s1 = kSplit ? __builtin_amdgcn_readfirstlane(S * (w + 1) / kWaves) : S;
}

template <bool kSplit, int kAct>
__global__ __launch_bounds__(kThreads, 3) void decode4_w13(DecodeArgs g) {
    __shared__ DecodeSmem sm;
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    int par = 0;
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
    const bool lead = !kSplit || threadIdx.x < MOE_WAVE;
    const int d = g.d, I = g.I, k = g.k, nIB = I / 8, S = d / 128, groups = (S + 3) / 4;
    const bool one = g.T == 1;
    int items;
    if (one) {
        if (blockIdx.x == 0) decode_flags_one_token(g);
        one_token_slots(sm, g);
        items = k * nIB;
    } else {
        decode_setup(sm, g.ids, g.T, k, g.E, g.status, blockIdx.x == 0);
        items = sm.n_active * nIB;
    }
    int s0, s1;
    wave_tiles<kSplit>(S, s0, s1);
    for_items<kSplit>(items, nIB, [&](int slot, int ib) {
        int e, M, e0;
        if (!slot_info(g, sm, one, slot, e, M, e0)) return;
        auto entry = [&](int m) { return one ? e0 : sm.ent[e0 + m]; };
        const size_t tile = (size_t)e * nIB + ib;
        const uint8_t* codes = reinterpret_cast<const uint8_t*>(g.w13) + tile * S * 1024 + lane * 16;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(g.w13_scale) + tile * groups * 64 + lane;
        for (int m0 = 0; m0 < M; m0 += 16) {
            const int m = m0 + n;
            const uint32_t ao = m < M ? (uint32_t)((entry(m) / k) * d) * 2u : kNoRow;
            const f32x4_t acc = reduce_waves<kSplit>(
                mma_tiles<kB>(codes, words, groups, rows_rsrc(g.x, (uint32_t)g.T * d * 2u), ao, s0, s1), red, par);
            float up[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) up[z] = __shfl_down(acc[z], 8, 16);
            if (lead && n < 8) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int mm = m0 + 4 * kq + z;
                    if (mm < M)
                        g.a[(size_t)entry(mm) * I + ib * 8 + n] = (uint16_t)f32_to_bf16(act_f<kAct>(acc[z]) * up[z]);
                }
            }
        }
    });
}

template <bool kSplit>
__global__ __launch_bounds__(kThreads, 3) void decode4_w2(DecodeArgs g) {
    __shared__ DecodeSmem sm;
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    int par = 0;
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
    const bool lead = !kSplit || threadIdx.x < MOE_WAVE;
    const int d = g.d, I = g.I, nNB = d / 16, S = I / 128, groups = (S + 3) / 4;
    decode_setup(sm, g.ids, g.T, g.k, g.E, g.status, false);
    int s0, s1;
    wave_tiles<kSplit>(S, s0, s1);
    for_items<kSplit>(sm.n_active * nNB, nNB, [&](int slot, int nb) {
        int e, M, e0;
        slot_info(g, sm, false, slot, e, M, e0);
        const size_t tile = (size_t)e * nNB + nb;
        const uint8_t* codes = reinterpret_cast<const uint8_t*>(g.w2) + tile * S * 1024 + lane * 16;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(g.w2_scale) + tile * groups * 64 + lane;
        for (int m0 = 0; m0 < M; m0 += 16) {
            const int m = m0 + n;
            const uint32_t ao = m < M ? (uint32_t)(sm.ent[e0 + m] * I) * 2u : kNoRow;
            const f32x4_t acc = reduce_waves<kSplit>(
                mma_tiles<kB>(codes, words, groups, rows_rsrc(g.a, (uint32_t)(g.T * g.k) * I * 2u), ao, s0, s1), red,
                par);
            if (lead) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int mm = m0 + 4 * kq + z;
                    if (mm < M) g.o[(size_t)sm.ent[e0 + mm] * d + nb * 16 + n] = (uint16_t)f32_to_bf16(acc[z]);
                }
            }
        }
    });
}

// One token: W2 of all k experts and the combine, 8 output features per workgroup.  As in the
// BF16 kernel, experts 2p and 2p + 1 share one MFMA: columns 0..7 are rows n0 .. n0 + 7 of
// expert 2p, columns 8..15 the same rows of expert 2p + 1, A row 0 is a_2p and row 1 a_2p+1.
__global__ __launch_bounds__(kThreads, 1) void decode4_w2_one(DecodeArgs g) {
    __shared__ float ov[kMaxTopK][8];
    __shared__ float sc[kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int d = g.d, I = g.I, k = g.k, S = I / 128, groups = (S + 3) / 4, nNB = d / 16;
    const int npair = (k + 1) / 2;
    const float score = tid < k ? g.scores[tid] : 0.f;
    auto expert = [&](int j) {
        const int e = j < k ? __builtin_amdgcn_readfirstlane(g.ids[j]) : -1;
        return (unsigned)e < (unsigned)g.E ? e : -1;
    };
    for (int nb = blockIdx.x; nb < d / 8; nb += gridDim.x) {
        const int n0 = nb * 8, piece = 16 * kq + (n0 & 8) + (n & 7);
        for (int p = wave; p < npair; p += kWaves) {
            const int e_x = expert(2 * p), e_y = expert(2 * p + 1);
            const bool vx = e_x >= 0, vy = e_y >= 0;
            const int e = n < 8 ? (vx ? e_x : 0) : (vy ? e_y : 0);
            const size_t tile = (size_t)e * nNB + (n0 >> 4);
            const uint8_t* codes = reinterpret_cast<const uint8_t*>(g.w2) + tile * S * 1024 + piece * 16;
            const uint32_t* words = reinterpret_cast<const uint32_t*>(g.w2_scale) + tile * groups * 64 + piece;
            const bool rv = (n == 0 && vx) || (n == 1 && vy);
            const uint32_t ao = rv ? (uint32_t)((2 * p + n) * I) * 2u : kNoRow;
            const f32x4_t acc = mma_tiles<8>(codes, words, groups, rows_rsrc(g.a, (uint32_t)k * I * 2u), ao, 0, S);
            if (kq == 0) {
                if (n < 8 && 2 * p < k) ov[2 * p][n] = vx ? acc[0] : 0.f;
                if (n >= 8 && 2 * p + 1 < k) ov[2 * p + 1][n - 8] = vy ? acc[1] : 0.f;
            }
        }
        if (tid < k) sc[tid] = score;
        __syncthreads();
        if (tid < 8) {
            float y = 0.f;
            for (int j = 0; j < k; ++j) y = __builtin_fmaf(sc[j], bf16_to_f32(f32_to_bf16(ov[j][tid])), y);
            g.y[n0 + tid] = (uint16_t)f32_to_bf16(y);
        }
        __syncthreads();
    }
}

// A workgroup per item with K split over its waves while that leaves wave slots empty, else a
// wave per item.
template <class K1, class K2>
hipError_t launch4(K1 wave_kernel, K2 split_kernel, const DecodeArgs& g, int nblk, int num_cu, hipStream_t s) {
    const int R = g.T * g.k;
    const int slots = R < g.E ? R : g.E;
    const int items = slots * nblk;
    const int cap = 3 * num_cu;
    if (items < cap * kWaves) {
        hipLaunchKernelGGL(split_kernel, dim3(items < cap ? items : cap), dim3(kThreads), 0, s, g);
    } else {
        const int grid = (items + kWaves - 1) / kWaves;
        hipLaunchKernelGGL(wave_kernel, dim3(grid < cap ? grid : cap), dim3(kThreads), 0, s, g);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode4_w13(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T * g.k > kMaxDecodeRows || g.d % 128 != 0 || g.I % 128 != 0) return hipErrorInvalidValue;
    if (g.act == kActGeGLU) return launch4(decode4_w13<false, kActGeGLU>, decode4_w13<true, kActGeGLU>, g, g.I / 8, num_cu, s);
    if (g.act == kActReGLU) return launch4(decode4_w13<false, kActReGLU>, decode4_w13<true, kActReGLU>, g, g.I / 8, num_cu, s);
    return launch4(decode4_w13<false, kActSwiGLU>, decode4_w13<true, kActSwiGLU>, g, g.I / 8, num_cu, s);
}

hipError_t launch_decode4_w2(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T == 1) {
        if (g.k > kMaxTopK) return hipErrorInvalidValue;
        const int cap = 3 * num_cu, grid = g.d / 8;
        hipLaunchKernelGGL(decode4_w2_one, dim3(grid < cap ? grid : cap), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    return launch4(decode4_w2<false>, decode4_w2<true>, g, g.d / 16, num_cu, s);
}

}  // namespace moe
