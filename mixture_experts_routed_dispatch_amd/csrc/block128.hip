// block128.hip -- operands in 8 bits with one FP32 scale per 128 (rows) or 128 x 128 (weights) on
// gfx950: rows and weights from BF16, weights back to BF16, and weights transposed.
//
// A block with largest magnitude m has the scale s = max(m / 448, 2^-100), rounded once; an element
// v the code E4M3(v / s), the nearest to the exact quotient, ties to even (block128.h).  The value of
// a code is its E4M3 number times s.
//   rows     [R, K]:    codes [R, K], scales [R, K/128], or [K/128, R] (block-major)
//   weights  [E, N, K]: codes [E, N, K], scales [E, N/128, K/128]
// All four are passes over memory.
#include "block128.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kB = 128;

// 16 lanes hold a block of a row, 8 elements each; a wave takes four consecutive blocks.
__global__ __launch_bounds__(kThreads) void rows_kernel(const uint16_t* __restrict__ v, int64_t blocks,
                                                        uint8_t* __restrict__ codes, float* __restrict__ scales) {
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < blocks * 16; i += step) {
        const uint4 x = *reinterpret_cast<const uint4*>(v + i * 8);
        const float s = block_scale(max16(bf16_amax_bits(x)));
        *reinterpret_cast<uint2*>(codes + i * 8) = block_codes8(x, s, block_inverse(s));
        if ((threadIdx.x & 15) == 0) scales[i >> 4] = s;
    }
}

// The same with block-major scales: a workgroup takes four blocks of 16 rows, a wave the four of every fourth row, and
// writes 16 consecutive scales at a time.  (Each wave the scales of its own four blocks: 65536 x 1536 83 us against
// 66.)  rows_dev (optional): only the first *rows_dev rows (at most rows).
__global__ __launch_bounds__(kThreads) void rows_block_major_kernel(const uint16_t* __restrict__ v, int64_t rows, int groups,
                                                                    const int32_t* __restrict__ rows_dev,
                                                                    uint8_t* __restrict__ codes, float* __restrict__ scales) {
    __shared__ float sc[4][16];
    int64_t n = rows;
    if (rows_dev) {
        n = *rows_dev;
        n = n < 0 ? 0 : n < rows ? n : rows;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, block = lane >> 4;
    const uint32_t spans = (uint32_t)(groups + 3) / 4, rg = blockIdx.x / spans, span = blockIdx.x - rg * spans;
    const int64_t row0 = (int64_t)rg * 16;
    if (row0 >= n) return;
    const int g = 4 * span + block;
    const bool in = g < groups;
    const int64_t at = (row0 + wave) * groups * kB + 512 * span + 8 * lane;
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (in && row0 + wave + 4 * u < n) x[u] = *reinterpret_cast<const uint4*>(v + at + (int64_t)4 * u * groups * kB);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (in && row0 + wave + 4 * u < n) {
            const float s = block_scale(max16(bf16_amax_bits(x[u])));
            *reinterpret_cast<uint2*>(codes + at + (int64_t)4 * u * groups * kB) = block_codes8(x[u], s, block_inverse(s));
            if ((lane & 15) == 0) sc[block][wave + 4 * u] = s;
        }
    __syncthreads();
    const int b = threadIdx.x >> 4, r = threadIdx.x & 15;
    if (threadIdx.x < 64 && 4 * (int)span + b < groups && row0 + r < n) scales[(int64_t)(4 * span + b) * rows + row0 + r] = sc[b][r];
}

// the same of FP32 rows, row-major scales
__global__ __launch_bounds__(kThreads) void rows_f32_kernel(const float* __restrict__ v, int64_t blocks,
                                                            uint8_t* __restrict__ codes, float* __restrict__ scales) {
    const int64_t pieces = blocks * 16, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < pieces; i += step) {
        f32x4_t x[2];
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x[h] = *reinterpret_cast<const f32x4_t*>(v + i * 8 + 4 * h);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint32_t m = __float_as_uint(x[h][z]) & 0x7FFFFFFFu;
                top = top > m ? top : m;
            }
        }
        const float s = block_scale(max16(top)), inv = block_inverse(s);
        *reinterpret_cast<uint2*>(codes + i * 8) = make_uint2(block_codes4(x[0][0], x[0][1], x[0][2], x[0][3], s, inv),
                                                              block_codes4(x[1][0], x[1][1], x[1][2], x[1][3], s, inv));
        if ((threadIdx.x & 15) == 0) scales[i >> 4] = s;
    }
}

// Workgroup = one 128 x 128 square of a matrix: a wave its rows 32 w .. 32 w + 31, four at a time
// (16 lanes x 16 bytes each), all in flight together.  One launch takes up to two matrices.
__global__ __launch_bounds__(kThreads) void squares_kernel(Block128Pair args) {
    __shared__ uint32_t tops[kThreads / MOE_WAVE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t u = blockIdx.x; u < args.m[0].units + args.m[1].units; u += gridDim.x) {
        const bool second = u >= args.m[0].units;
        const Block128Matrix& m = args.m[second];
        const int64_t sq = second ? u - args.m[0].units : u, br = sq / (m.K / kB);   // square, block row
        const int64_t at = (br * kB + 32 * wave + (lane >> 4)) * m.K + (sq - br * (m.K / kB)) * kB + 8 * (lane & 15);
        uint4 x[8];
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) x[r] = *reinterpret_cast<const uint4*>(m.w + at + (int64_t)4 * r * m.K);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const uint32_t t = bf16_amax_bits(x[r]);
            top = top > t ? top : t;
        }
        for (int o = 32; o; o >>= 1) {
            const uint32_t t = __shfl_xor(top, o, MOE_WAVE);
            top = top > t ? top : t;
        }
        __syncthreads();                                // the last square's maxima have been read
        if (lane == 0) tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / MOE_WAVE; ++w) top = top > tops[w] ? top : tops[w];
        const float s = block_scale(top), inv = block_inverse(s);
#pragma unroll
        for (int r = 0; r < 8; ++r)
            *reinterpret_cast<uint2*>(m.codes + at + (int64_t)4 * r * m.K) = block_codes8(x[r], s, inv);
        if (threadIdx.x == 0) m.scales[sq] = s;
    }
}

// 16 codes of a row at a time: E4M3 number times scale, rounded to BF16
__global__ __launch_bounds__(kThreads) void expand_kernel(Block128Pair args) {
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < args.m[0].units + args.m[1].units; u += step) {
        const bool second = u >= args.m[0].units;
        const Block128Matrix& m = args.m[second];
        const int64_t i = second ? u - args.m[0].units : u, per = m.K / 16, row = i / per;
        const int c = (int)(i - row * per);
        const uint4 q = *reinterpret_cast<const uint4*>(m.codes + i * 16);
        const float s = m.scales[row / kB * (m.K / kB) + c / 8];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
            const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
            o[2 * j] = pack_bf16(lo[0] * s, lo[1] * s);
            o[2 * j + 1] = pack_bf16(hi[0] * s, hi[1] * s);
        }
        uint4* dst = reinterpret_cast<uint4*>(m.w + i * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// m_out [E+1] = m_in where it rises from 0 to at most R, else zeros and the flag; m_in NULL: 0, R.  By one workgroup.
__device__ __forceinline__ void write_segments(const Segments& g) {
    bool bad = false;
    for (int i = threadIdx.x; g.in && i <= g.E; i += kThreads) bad |= i == 0 ? g.in[0] != 0 : g.in[i] < g.in[i - 1] || g.in[i] > g.R;
    bad = __syncthreads_or(bad);
    for (int i = threadIdx.x; i <= g.E; i += kThreads) g.out[i] = bad ? 0 : g.in ? g.in[i] : i == 0 ? 0 : g.R;
    if (bad && threadIdx.x == 0 && g.status) atomicOr(g.status, kDevBadIndptr);
}
__global__ __launch_bounds__(kThreads) void segments_kernel(Segments g) { write_segments(g); }

// Transpose of codes [E, N, K] to [E, K, N] and of their scales, a 128 x 128 square a workgroup, by
// way of LDS (row stride 132: a column's bytes meet different banks).  seg (out NULL: none) is written along
// with it, which saves a launch.
constexpr int kLd = 132;
__global__ __launch_bounds__(kThreads) void transpose_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                                                             int N, int K, uint8_t* __restrict__ codes_t,
                                                             float* __restrict__ scales_t, Segments seg) {
    __shared__ uint32_t tile[kB * kLd / 4];
    const int t = threadIdx.x, bn = blockIdx.x / (K / kB), bk = blockIdx.x - bn * (K / kB);
    const int64_t e = blockIdx.y;
    if (seg.out && blockIdx.x == 0 && e == 0) write_segments(seg);
    const uint8_t* src = codes + (e * N + (int64_t)bn * kB) * K + bk * kB;
    uint8_t* dst = codes_t + (e * K + bk * kB) * N + bn * kB;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 32 * r + (t >> 3), c = t & 7;
        const uint4 v = *reinterpret_cast<const uint4*>(src + (int64_t)row * K + 16 * c);
        uint32_t* p = tile + row * (kLd / 4) + 4 * c;
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    }
    __syncthreads();
    // thread: the 4 x 16 bytes of columns 4 c .. 4 c + 3, rows 16 g .. 16 g + 15
    const int c = t & 31, g = t >> 5;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = tile[(16 * g + i) * (kLd / 4) + c];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = (w[4 * q] >> (8 * j) & 0xFF) | (w[4 * q + 1] >> (8 * j) & 0xFF) << 8 |
                   (w[4 * q + 2] >> (8 * j) & 0xFF) << 16 | (w[4 * q + 3] >> (8 * j) & 0xFF) << 24;
        *reinterpret_cast<uint4*>(dst + (int64_t)(4 * c + j) * N + 16 * g) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (t == 0) scales_t[(e * (K / kB) + bk) * (N / kB) + bn] = scales[(e * (N / kB) + bn) * (K / kB) + bk];
}

bool shapes_ok(const Block128Pair& g) {
    for (const Block128Matrix& m : g.m)
        if (m.w && (m.E <= 0 || m.N <= 0 || m.K <= 0 || m.N % kB != 0 || m.K % kB != 0)) return false;
    return true;
}
int grid_of(int64_t n, int64_t most) { return (int)(n < 1 ? 1 : n < most ? n : most); }

}  // namespace

hipError_t launch_block128_rows(const uint16_t* v, int64_t rows, int K, uint8_t* codes, float* scales, bool block_major,
                                const int32_t* rows_dev, hipStream_t s) {
    if (rows < 0 || K <= 0 || K % kB != 0 || (rows_dev && !block_major)) return hipErrorInvalidValue;
    if (rows == 0) return hipSuccess;
    if (block_major) {
        const int64_t wgs = (rows + 15) / 16 * ((K / kB + 3) / 4);
        if (wgs > 0x7FFFFFFF) return hipErrorInvalidValue;
        hipLaunchKernelGGL(rows_block_major_kernel, dim3((unsigned)wgs), dim3(kThreads), 0, s, v, rows, K / kB, rows_dev, codes, scales);
    } else {
        const int64_t wgs = (rows * (K / 8) + kThreads - 1) / kThreads;
        hipLaunchKernelGGL(rows_kernel, dim3(grid_of(wgs, 65536)), dim3(kThreads), 0, s, v, rows * (K / kB), codes, scales);
    }
    return hipGetLastError();
}

hipError_t launch_block128_rows_f32(const float* v, int64_t rows, int K, uint8_t* codes, float* scales, hipStream_t s) {
    if (rows < 0 || K <= 0 || K % kB != 0) return hipErrorInvalidValue;
    if (rows == 0) return hipSuccess;
    const int64_t wgs = (rows * (K / 8) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(rows_f32_kernel, dim3(grid_of(wgs, 65536)), dim3(kThreads), 0, s, v, rows * (K / kB), codes, scales);
    return hipGetLastError();
}

hipError_t launch_block128_pack(Block128Pair g, hipStream_t s) {
    if (!shapes_ok(g)) return hipErrorInvalidValue;
    for (Block128Matrix& m : g.m) m.units = m.w ? (int64_t)m.E * (m.N / kB) * (m.K / kB) : 0;
    hipLaunchKernelGGL(squares_kernel, dim3(grid_of(g.m[0].units + g.m[1].units, 1 << 20)), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_block128_expand(Block128Pair g, hipStream_t s) {
    if (!shapes_ok(g)) return hipErrorInvalidValue;
    for (Block128Matrix& m : g.m) m.units = m.w ? (int64_t)m.E * m.N * (m.K / 16) : 0;
    const int64_t wgs = (g.m[0].units + g.m[1].units + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(expand_kernel, dim3(grid_of(wgs, 1 << 20)), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_segments(const Segments& g, hipStream_t s) {
    if (g.E <= 0 || g.E > 256 || g.R < 0 || (!g.in && g.E != 1)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(segments_kernel, dim3(1), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_block128_transpose(const uint8_t* codes, const float* scales, int E, int N, int K, uint8_t* codes_t,
                                     float* scales_t, const Segments& seg, hipStream_t s) {
    if (seg.out && (seg.E <= 0 || seg.E > 256 || seg.R < 0 || (!seg.in && seg.E != 1))) return hipErrorInvalidValue;
    if (E <= 0 || N <= 0 || K <= 0 || N % kB != 0 || K % kB != 0 || E > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL(transpose_kernel, dim3(K / kB * (N / kB), E), dim3(kThreads), 0, s, codes, scales, N, K, codes_t, scales_t, seg);
    return hipGetLastError();
}

}  // namespace moe
