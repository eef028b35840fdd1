// decode_mxfp4.hip -- weight-streaming path for expert weights in MXFP4 (mxfp4.hip's layout),
// T*k <= 256 routed rows.
//
// The same launches as with BF16 weights (decode.hip): W13 with the activation, then for one
// token W2 with the combine, else W2 and a combine.  a is rounded to BF16, the operand type of
// the W2 products; the experts' outputs o stay in FP32 until the one rounding of y.  The time is
// that of streaming 4.25 bits for each weight of the active experts.
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

// Scales of tiles s .. s + 3 of this lane's block, one byte each, from the words of a row tile
__device__ __forceinline__ uint32_t scale_bytes(const uint32_t* words, int s, int groups) {
    const int g0 = s >> 2, g1 = g0 + 1 < groups ? g0 + 1 : g0;
    const uint32_t lo = words[g0 * 64], hi = words[g1 * 64];
    return __builtin_amdgcn_alignbit(hi, lo, 8 * (s & 3));
}

// acc += A * B for one quarter of the lanes' blocks: eight codes and their scale to BF16, exact
__device__ __forceinline__ f32x4_t mma_quarter(bf16x8_t a, uint32_t codes, float x, f32x4_t acc) {
    const bf16x2_t w0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, x, 0);
    const bf16x2_t w1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, x, 1);
    const bf16x2_t w2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, x, 2);
    const bf16x2_t w3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, x, 3);
    const bf16x8_t w = {w0[0], w0[1], w1[0], w1[1], w2[0], w2[1], w3[0], w3[1]};
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w, acc, 0, 0, 0);
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
                for (int i = 0; i < 4; ++i) acc = mma_quarter(a[j][i], c[j][i], x, acc);
            }
    }
    return acc;
}

// Many items: a wave owns (active expert, kTiles row tiles) from the first load to the last
// store.  Its work is a sequence of units, one 16-row group of the expert's routed rows by B
// tiles along K; the codes of the next unit (of the next item too) are loaded before the
// current unit's products, behind its operand rows, so that the wait for those leaves them in
// flight.  An operand row piece is four loads for each load of codes; two row tiles share
// them.  32 tokens of the 128-expert layer (187 MB of W13, 93 MB of W2): one tile and B = 4
// 37.2 + 22.3 us, two tiles and B = 4 (three waves a SIMD) 31.3 + 19.1, two tiles and B = 2
// (four) 29.4 + 18.3, four tiles and B = 2 (three) 30.5 + 18.1.
constexpr int kTiles = 2, kB = 2, kWaveWGs = 4;       // workgroups a CU
struct Codes4 {
    u32x4_t c[kTiles][kB];
    uint32_t sb[kTiles];             // one byte for each of four tiles along K
};
struct Unit4 {
    int item, slot, blk, e, M, e0, m0, s;
    bool valid;
};
template <typename Store>
__device__ __forceinline__ void wave_items(const DecodeSmem& sm, const void* codes_base, const void* words_base,
                                           __amdgpu_buffer_rsrc_t ars, int nblk, int S, int row_bytes, int row_div,
                                           Store&& store) {
    const int lane = threadIdx.x & 63, n = lane & 15;
    const int groups = (S + 3) / 4, per = nblk / kTiles;
    const int items = __builtin_amdgcn_readfirstlane(sm.n_active) * per;
    const int nw = (int)gridDim.x * kWaves;
    auto begin = [&](int item) {
        Unit4 u = {};
        u.item = item;
        u.valid = item < items;
        if (!u.valid) return u;
        u.slot = item / per;
        u.blk = (item - u.slot * per) * kTiles;
        u.e = __builtin_amdgcn_readfirstlane(sm.slot_expert[u.slot]);
        u.e0 = __builtin_amdgcn_readfirstlane(sm.pfx[u.e]);
        u.M = __builtin_amdgcn_readfirstlane(sm.pfx[u.e + 1]) - u.e0;
        u.m0 = u.s = 0;
        return u;
    };
    auto after = [&](Unit4 u) {
        u.s += kB;
        if (u.s < S) return u;
        u.s = 0;
        u.m0 += 16;
        if (u.m0 < u.M) return u;
        return begin(u.item + nw);
    };
    auto load = [&](const Unit4& u, Codes4& w) {
        const size_t tile = (size_t)u.e * nblk + u.blk;
        const uint8_t* codes = static_cast<const uint8_t*>(codes_base) + (tile * S + u.s) * 1024 + lane * 16;
        const uint32_t* words = static_cast<const uint32_t*>(words_base) + (tile * groups + (u.s >> 2)) * 64 + lane;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int j = 0; j < kB; ++j)
                if (u.s + j < S)
                    w.c[t][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + (size_t)(t * S + j) * 1024));
            w.sb[t] = words[t * groups * 64];
        }
    };
    Unit4 u = begin((int)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)));
    if (!u.valid) return;
    Codes4 cur, next;
    load(u, cur);
    f32x4_t acc[kTiles] = {};
    bf16x8_t a[kB][4] = {};
    while (true) {
        const int m = u.m0 + n;
        if (m < u.M) {                                  // the rows of other lanes are never stored
            const uint32_t ao = (uint32_t)(sm.ent[u.e0 + m] / row_div) * (uint32_t)row_bytes + 64u * (lane >> 4) + 256u * u.s;
#pragma unroll
            for (int j = 0; j < kB; ++j)
                if (u.s + j < S)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        a[j][i] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(ars, ao + 256u * j + 16u * i, 0, 0));
        }
        const Unit4 v = after(u);
        if (v.valid) load(v, next);
#pragma unroll
        for (int j = 0; j < kB; ++j)
            if (u.s + j < S)
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const float x = __uint_as_float(((cur.sb[t] >> (8 * ((u.s & 3) + j))) & 0xFFu) << 23);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t] = mma_quarter(a[j][i], cur.c[t][j][i], x, acc[t]);
                }
        if (u.s + kB >= S) {
            store(u, acc);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        if (!v.valid) return;
        u = v;
        cur = next;
    }
}

template <int kAct>
__global__ __launch_bounds__(kThreads, kWaveWGs) void decode4_w13_wave(DecodeArgs g) {
    __shared__ DecodeSmem sm;
    decode_setup(sm, g.ids, g.T, g.k, g.E, g.status, blockIdx.x == 0);
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4, I = g.I;
    wave_items(sm, g.w13, g.w13_scale, rows_rsrc(g.x, (uint32_t)g.T * g.d * 2u), I / 8, g.d / 128, 2 * g.d, g.k,
                     [&](const Unit4& u, f32x4_t (&acc)[kTiles]) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            float up[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) up[z] = __shfl_down(acc[t][z], 8, 16);
            if (n < 8) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int mm = u.m0 + 4 * kq + z;
                    if (mm < u.M)
                        g.a[(size_t)sm.ent[u.e0 + mm] * I + (u.blk + t) * 8 + n] = (uint16_t)f32_to_bf16(act_f<kAct>(acc[t][z]) * up[z]);
                }
            }
        }
    });
}

__global__ __launch_bounds__(kThreads, kWaveWGs) void decode4_w2_wave(DecodeArgs g) {
    __shared__ DecodeSmem sm;
    decode_setup(sm, g.ids, g.T, g.k, g.E, g.status, false);
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4, d = g.d;
    float* o = reinterpret_cast<float*>(g.o);
    wave_items(sm, g.w2, g.w2_scale, rows_rsrc(g.a, (uint32_t)(g.T * g.k) * g.I * 2u), d / 16, g.I / 128, 2 * g.I, 1,
                     [&](const Unit4& u, f32x4_t (&acc)[kTiles]) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int mm = u.m0 + 4 * kq + z;
                if (mm < u.M) o[(size_t)sm.ent[u.e0 + mm] * d + (u.blk + t) * 16 + n] = acc[t][z];
            }
    });
}

// Few items: a workgroup per (active expert, row tile), its four waves a quarter of K each: all
// of the item's loads are in flight at once, and the partial sums meet in LDS.
constexpr int kSplitWGs = 3;
__device__ __forceinline__ void wave_tiles(int S, int& s0, int& s1) {
    const int w = threadIdx.x >> 6;
    s0 = __builtin_amdgcn_readfirstlane(S * w / kWaves);
    s1 = __builtin_amdgcn_readfirstlane(S * (w + 1) / kWaves);
}

template <int kAct>
__global__ __launch_bounds__(kThreads, kSplitWGs) void decode4_w13_split(DecodeArgs g) {
    __shared__ DecodeSmem sm;
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    int par = 0;
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
    const bool lead = threadIdx.x < MOE_WAVE;
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
    wave_tiles(S, s0, s1);
    for_items<true>(items, nIB, [&](int slot, int ib) {
        int e, M, e0;
        if (!slot_info(g, sm, one, slot, e, M, e0)) return;
        auto entry = [&](int m) { return one ? e0 : sm.ent[e0 + m]; };
        const size_t tile = (size_t)e * nIB + ib;
        const uint8_t* codes = reinterpret_cast<const uint8_t*>(g.w13) + tile * S * 1024 + lane * 16;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(g.w13_scale) + tile * groups * 64 + lane;
        for (int m0 = 0; m0 < M; m0 += 16) {
            const int m = m0 + n;
            const uint32_t ao = m < M ? (uint32_t)((entry(m) / k) * d) * 2u : kNoRow;
            const f32x4_t acc = reduce_waves<true>(
                mma_tiles<4>(codes, words, groups, rows_rsrc(g.x, (uint32_t)g.T * d * 2u), ao, s0, s1), red, par);
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

__global__ __launch_bounds__(kThreads, kSplitWGs) void decode4_w2_split(DecodeArgs g) {
    __shared__ DecodeSmem sm;
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    int par = 0;
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
    const bool lead = threadIdx.x < MOE_WAVE;
    const int d = g.d, I = g.I, nNB = d / 16, S = I / 128, groups = (S + 3) / 4;
    decode_setup(sm, g.ids, g.T, g.k, g.E, g.status, false);
    int s0, s1;
    wave_tiles(S, s0, s1);
    for_items<true>(sm.n_active * nNB, nNB, [&](int slot, int nb) {
        int e, M, e0;
        slot_info(g, sm, false, slot, e, M, e0);
        const size_t tile = (size_t)e * nNB + nb;
        const uint8_t* codes = reinterpret_cast<const uint8_t*>(g.w2) + tile * S * 1024 + lane * 16;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(g.w2_scale) + tile * groups * 64 + lane;
        for (int m0 = 0; m0 < M; m0 += 16) {
            const int m = m0 + n;
            const uint32_t ao = m < M ? (uint32_t)(sm.ent[e0 + m] * I) * 2u : kNoRow;
            const f32x4_t acc = reduce_waves<true>(
                mma_tiles<4>(codes, words, groups, rows_rsrc(g.a, (uint32_t)(g.T * g.k) * I * 2u), ao, s0, s1), red,
                par);
            if (lead) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int mm = m0 + 4 * kq + z;
                    if (mm < M) reinterpret_cast<float*>(g.o)[(size_t)sm.ent[e0 + mm] * d + nb * 16 + n] = acc[z];
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
            for (int j = 0; j < k; ++j) y = __builtin_fmaf(sc[j], ov[j][tid], y);
            g.y[n0 + tid] = (uint16_t)f32_to_bf16(y);
        }
        __syncthreads();
    }
}

// y[t] = sum_j s[t][j] o[t*k + j] in FP32, j ascending from +0.0; four features a thread
__global__ __launch_bounds__(kThreads) void decode4_combine(DecodeArgs g) {
    const int t = blockIdx.y, n = (blockIdx.x * kThreads + threadIdx.x) * 4;
    if (n >= g.d) return;
    const float* o = reinterpret_cast<const float*>(g.o) + (size_t)t * g.k * g.d + n;
    f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int j = 0; j < g.k; ++j) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(o + (size_t)j * g.d);
        const float s = g.scores[t * g.k + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(s, v[i], y[i]);
    }
    *reinterpret_cast<uint2*>(g.y + (size_t)t * g.d + n) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

#ifndef D4_SPLIT
#define D4_SPLIT 16
#endif
// nblk row tiles for each of at most `slots` active experts
template <class K1, class K2>
hipError_t launch4(K1 wave_kernel, K2 split_kernel, const DecodeArgs& g, int nblk, int num_cu, hipStream_t s) {
    const int R = g.T * g.k;
    const int slots = R < g.E ? R : g.E;
    const int items = slots * nblk;
    if (items < D4_SPLIT * num_cu) {
        const int cap = kSplitWGs * num_cu;
        hipLaunchKernelGGL(split_kernel, dim3(items < cap ? items : cap), dim3(kThreads), 0, s, g);
    } else {
        const int grid = (items / kTiles + kWaves - 1) / kWaves, cap = kWaveWGs * num_cu;
        hipLaunchKernelGGL(wave_kernel, dim3(grid < cap ? grid : cap), dim3(kThreads), 0, s, g);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode4_w13(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T * g.k > kMaxDecodeRows || g.d % 128 != 0 || g.I % 128 != 0) return hipErrorInvalidValue;
    if (g.act == kActGeGLU) return launch4(decode4_w13_wave<kActGeGLU>, decode4_w13_split<kActGeGLU>, g, g.I / 8, num_cu, s);
    if (g.act == kActReGLU) return launch4(decode4_w13_wave<kActReGLU>, decode4_w13_split<kActReGLU>, g, g.I / 8, num_cu, s);
    return launch4(decode4_w13_wave<kActSwiGLU>, decode4_w13_split<kActSwiGLU>, g, g.I / 8, num_cu, s);
}

hipError_t launch_decode4_w2(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T == 1) {
        if (g.k > kMaxTopK) return hipErrorInvalidValue;
        const int cap = 3 * num_cu, grid = g.d / 8;
        hipLaunchKernelGGL(decode4_w2_one, dim3(grid < cap ? grid : cap), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    const hipError_t e = launch4(decode4_w2_wave, decode4_w2_split, g, g.d / 16, num_cu, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(decode4_combine, dim3((g.d / 4 + kThreads - 1) / kThreads, g.T), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

}  // namespace moe
