// mxfp4.hip -- expert weights in OCP MXFP4 (E2M1 elements, E8M0 scale per 32 along K) on
// gfx950: BF16 -> codes and scales in the decode kernels' layout, and back to BF16.
//
// The scale of a block is the smallest power of two X with max|v| / X <= 6 (E2M1's largest),
// the element v / X rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even
// code).  The value of a code, element times X, is exact in BF16.
//
// Layout: a matrix of N rows (K columns) is cut into tiles of 16 rows x 128 columns of 1 KiB,
// the tiles of 16 rows one after another along K.  Inside a tile, 16-byte piece 16 q + n holds
// the block of columns 32 q .. 32 q + 31 of the tile's row n (element 2 i in the low half of
// byte i): the wave that loads a tile reads 1 KiB in a row and finds in each lane one whole
// block, whose four 8-element quarters are the operands of four MFMAs.  Scales: one word per
// tile row group, piece and four tiles along K, [N/16][ceil(K/512)][64] words; byte j is the
// scale of tile 4 g + j.  Tile b of W13 has gate rows 8 b .. 8 b + 7 as its rows 0 .. 7 and the
// same up rows as its rows 8 .. 15; tile b of W2 has rows 16 b .. 16 b + 15.
//
// Both directions are bound by memory.  Quantizing 16 experts of d = 2048, I = 768 (151 MB to
// 40 MB) takes 41 us (4.7 TB/s), 128 of them 282 us (5.4 TB/s); expanding the 16 29 us.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// the source row of tile row n
__device__ __forceinline__ int tile_row(int tile, int n, int I, bool w13) {
    return w13 ? (n < 8 ? 8 * tile + n : I + 8 * tile + n - 8) : 16 * tile + n;
}

// One launch takes both matrices: waves go over the units of the first, then the second's.
template <typename F> __device__ __forceinline__ void for_units(const Mxfp4Args& g, F&& f) {
    const int64_t step = (int64_t)gridDim.x * (kThreads / MOE_WAVE);
    const int64_t total = g.m[0].units + g.m[1].units;
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / MOE_WAVE) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         u < total; u += step) {
        if (u < g.m[0].units) f(g.m[0], u);
        else f(g.m[1], u - g.m[0].units);
    }
}

// A wave takes four tiles along K of one row tile: each lane quantizes the block that is its
// piece of each, so that codes leave as whole KiB and scales as whole words.
__global__ __launch_bounds__(kThreads) void mxfp4_pack_kernel(Mxfp4Args args) {
    const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
    for_units(args, [&](const Mxfp4Matrix& mat, int64_t u) {
        const int K = mat.K, N = mat.N, S = K / 128, groups = (S + 3) / 4, tiles = N / 16;
        const int64_t rt = u / groups;                  // expert and row tile
        const int g = (int)(u - rt * groups);
        const int e = (int)(rt / tiles), tile = (int)(rt - (int64_t)e * tiles);
        const uint16_t* src = mat.w + ((int64_t)e * N + tile_row(tile, n, N / 2, mat.w13)) * K + 512 * g + 32 * q;
        uint32_t word = 0;
        uint4 v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * g + j < S)
#pragma unroll
                for (int c = 0; c < 4; ++c) v[j][c] = *reinterpret_cast<const uint4*>(src + 128 * j + 8 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (4 * g + j >= S) break;
            uint32_t b[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                b[4 * c] = v[j][c].x; b[4 * c + 1] = v[j][c].y; b[4 * c + 2] = v[j][c].z; b[4 * c + 3] = v[j][c].w;
            }
            uint32_t hi = 0, lo = 0;                    // magnitudes of BF16 order like their bits
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t h = b[i] & 0x7FFF0000u, l = b[i] & 0x7FFFu;
                hi = hi > h ? hi : h;
                lo = lo > l ? lo : l;
            }
            const uint32_t top = (hi >> 16) > lo ? hi >> 16 : lo;
            const int byte = e8m0_scale_e2m1(top);
            const float x = __uint_as_float((uint32_t)byte << 23);
            uint32_t out[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t r = 0;
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, b[4 * c]), x, 0);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, b[4 * c + 1]), x, 1);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, b[4 * c + 2]), x, 2);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, b[4 * c + 3]), x, 3);
                out[c] = r;
            }
            *reinterpret_cast<uint4*>(mat.codes + ((rt * S + 4 * g + j) * 64 + lane) * 16) =
                make_uint4(out[0], out[1], out[2], out[3]);
            word |= (uint32_t)byte << (8 * j);
        }
        mat.scales[(rt * groups + g) * 64 + lane] = word;
    });
}

// A wave expands one tile: for each of four rounds, lanes 16 r .. 16 r + 15 write the 256
// consecutive bytes of tile row 4 round + r.
__global__ __launch_bounds__(kThreads) void mxfp4_expand_kernel(Mxfp4Args args) {
    const int lane = threadIdx.x & 63, c8 = lane & 15, q = c8 >> 2;
    for_units(args, [&](const Mxfp4Matrix& mat, int64_t u) {
        const int K = mat.K, N = mat.N, S = K / 128, groups = (S + 3) / 4, tiles = N / 16;
        const int64_t rt = u / S;
        const int s = (int)(u - rt * S);
        const int e = (int)(rt / tiles), tile = (int)(rt - (int64_t)e * tiles);
        uint32_t code[4], word[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 4 * r + (lane >> 4);
            code[r] = *reinterpret_cast<const uint32_t*>(mat.codes + (u * 64 + 16 * q + n) * 16 + 4 * (c8 & 3));
            word[r] = mat.scales[(rt * groups + (s >> 2)) * 64 + 16 * q + n];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = 4 * r + (lane >> 4);
            const float x = __uint_as_float(((word[r] >> (8 * (s & 3))) & 0xFFu) << 23);
            uint4 o;
            o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[r], x, 0));
            o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[r], x, 1));
            o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[r], x, 2));
            o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[r], x, 3));
            *reinterpret_cast<uint4*>(mat.w + ((int64_t)e * N + tile_row(tile, n, N / 2, mat.w13)) * K + 128 * s + 8 * c8) = o;
        }
    });
}

int grid_of(const Mxfp4Args& g) {
    const int64_t b = (g.m[0].units + g.m[1].units + kThreads / MOE_WAVE - 1) / (kThreads / MOE_WAVE);
    return (int)(b < 8192 ? b : 8192);
}
bool shapes_ok(const Mxfp4Args& g) {
    for (const Mxfp4Matrix& m : g.m)
        if (m.w && (m.N % 16 != 0 || m.K % 128 != 0)) return false;
    return true;
}

}  // namespace

hipError_t launch_mxfp4_pack(Mxfp4Args g, hipStream_t s) {
    if (!shapes_ok(g)) return hipErrorInvalidValue;
    for (Mxfp4Matrix& m : g.m) m.units = m.w ? (int64_t)m.E * (m.N / 16) * ((m.K / 128 + 3) / 4) : 0;
    hipLaunchKernelGGL(mxfp4_pack_kernel, dim3(grid_of(g)), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_mxfp4_expand(Mxfp4Args g, hipStream_t s) {
    if (!shapes_ok(g)) return hipErrorInvalidValue;
    for (Mxfp4Matrix& m : g.m) m.units = m.w ? (int64_t)m.E * (m.N / 16) * (m.K / 128) : 0;
    hipLaunchKernelGGL(mxfp4_expand_kernel, dim3(grid_of(g)), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

}  // namespace moe
