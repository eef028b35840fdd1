// decode_block128.hip -- weight-streaming path for weights in E4M3 with one FP32 scale per 128 x 128
// (block128.hip), up to 256 rows: the expert layer's decode (T*k <= 256) and a product of few rows.
//
// The same quantities as on the grouped-GEMM path (gemm_block128.hip): rows in E4M3 with a scale per
// 128, sums of 128 products by one v_mfma_f32_16x16x128_f8f6f4 (the layer's W13: by four BF16 instructions, exact), times
// their scales added in FP32.  Here the weights are the instruction's rows: a wave takes 16 weight rows x 128 of K (2 KiB) with two
// 16-byte loads a lane, and up to 16 rows of the batch are its columns.  Lane (n, q) of either operand
// holds bytes 16 q .. + 15 and 64 + 16 q .. + 15 of the 128 (the instruction's order of K is free as long
// as both agree).  The time is that of streaming the weights.
//
// Several tokens: one launch sorts the entries by expert and quantizes x; W13 leaves a in FP32, since
// a block of it is the work of several workgroups; a launch quantizes it; W2 and the combine follow.
// One token: two launches, whose workgroups quantize x and a for themselves.
//
// d = 2048, I = 768, k = 8: one token 13.3 us a call in a graph for 25 + 13 MB (traced, 8.1 to 9.5 and 6.3 to 6.8), a round trip of loads
// each; 32 tokens of 68 experts W13 39.9 us (5.4 TB/s), W2 21.2 (5.1 TB/s), the three small launches 4.6-5.5 each.  A product
// of one row of 4096 x 4096: 5.6 us.
#include "block128.h"
#include "decode_common.h"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
constexpr int kNonTemporal = 2;      // the nt bit of a buffer load

__device__ __forceinline__ i32x8_t join(i32x4_t a, i32x4_t b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
__device__ __forceinline__ f32x4_t mma128(i32x8_t a, i32x8_t b) {
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}
// The same to FP32's precision: E4M3 values are BF16 numbers, and the BF16 instruction keeps their products whole (error
// 2^-26.7 of the sums in rms, against 2^-16 of the instruction above, which drops what lies below 2^-13 of the largest of eight
// products).  W13 takes it: of a's elements whose sums are off by 2^-16, 2^-9.3 fall on the other side of a border between
// their E4M3 codes, and with few rows a single one can be 3e-3 of y.  The weights' loads hide most of it (one token in a
// graph 12.9 -> 13.3 us, 32 tokens of 68 experts 68.6 -> 69.4).
__device__ __forceinline__ bf16x8_t to_bf16(int a, int b) {
    auto two = [](int w, auto high) { return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, decltype(high)::value)); };
    const i32x4_t v = {two(a, std::false_type()), two(a, std::true_type()), two(b, std::false_type()), two(b, std::true_type())};
    return __builtin_bit_cast(bf16x8_t, v);
}
__device__ __forceinline__ f32x4_t mma128_exact(i32x8_t a, i32x8_t b) {
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16(a[2 * i], a[2 * i + 1]), to_bf16(b[2 * i], b[2 * i + 1]), s, 0, 0, 0);
    return s;
}
template <bool kExact> __device__ __forceinline__ f32x4_t mma(i32x8_t a, i32x8_t b) {
    if constexpr (kExact) return mma128_exact(a, b);
    else return mma128(a, b);
}
__device__ __forceinline__ i32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t lane_offset, int offset, int policy) {
    return policy ? __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, lane_offset, offset, kNonTemporal))
                  : __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, lane_offset, offset, 0));
}
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16 weight rows x 128 of K as an operand, from two loads of whole lines: lane (n, q) has loaded bytes 16 q + 64 (n / 8) .. of row
// n % 8 (r0) and of row 8 + n % 8 (r1); lanes n and n ^ 8 exchange one of them.  (Loads of 64 bytes of each of 16 rows, two of
// which share a line: layer of 32 tokens of 68 experts 81 us against 69, one token in a graph 13.4 against 12.9, both
// without W13's exact sums.)
__device__ __forceinline__ i32x8_t join_lines(i32x4_t r0, i32x4_t r1) {
    i32x4_t a, b;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        a[z] = __builtin_amdgcn_update_dpp(r0[z], r1[z], 0x128, 0xF, 0xC, false);       // row_ror:8, to lanes n >= 8
        b[z] = __builtin_amdgcn_update_dpp(r1[z], r0[z], 0x128, 0xF, 0x3, false);       // to lanes n < 8
    }
    return join(a, b);
}
// this lane's byte of the first of those loads, in a matrix of rows of K bytes; the second's is 8 K further
__device__ __forceinline__ uint32_t line_offset(int K) {
    const int lane = threadIdx.x & 63;
    return (uint32_t)(lane & 7) * K + 16u * (lane >> 4) + 64u * (lane >> 3 & 1);
}

// Rows of up to 16 consecutive entries of one expert; what the first launch leaves for the others.
struct Groups {
    int n, pad[3];
    int4 g[kMaxDecodeRows];          // expert, first entry, entries
    int ent[kMaxDecodeRows];         // the entry's row
};
static_assert(sizeof(Groups) <= kBlock128GroupBytes, "room in the workspaces");

// rows of x in 8 bits: blocks of 128 counted over all rows, 16 lanes each, from `first` in steps of `step`
__device__ __forceinline__ void quantize_rows(const uint16_t* x, int64_t blocks, int64_t first, int64_t step, uint8_t* xq, float* xs) {
    for (int64_t i = first; i < blocks * 16; i += step) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + i * 8);
        const float s = block_scale(max16(bf16_amax_bits(v)));
        *reinterpret_cast<uint2*>(xq + i * 8) = block_codes8(v, s, block_inverse(s));
        if ((i & 15) == 0) xs[i >> 4] = s;
    }
}

// First launch of several tokens: workgroup 0 sorts the entries and sets the routing flags, the others
// quantize x [T, d].
__global__ __launch_bounds__(kThreads) void decode8_prepare(DecodeArgs g) {
    __shared__ Sorted sm;
    if (blockIdx.x > 0) {
        quantize_rows(g.x, (int64_t)g.T * (g.d / 128), (int64_t)(blockIdx.x - 1) * kThreads + threadIdx.x,
                      (int64_t)(gridDim.x - 1) * kThreads, g.xq, g.xs);
        return;
    }
    sort_entries(sm, g, true);
    Groups* out = static_cast<Groups*>(g.groups);
    const int tid = threadIdx.x;
    if (tid == 0) out->n = sm.groups;
    if (tid < sm.groups) {
        const int e = sm.group[tid] & 255, first = sm.pfx[e] + (sm.group[tid] >> 8) * kRows, left = sm.pfx[e + 1] - first;
        out->g[tid] = make_int4(e, first, left < kRows ? left : kRows, 0);
    }
    if (tid < sm.pfx[256]) out->ent[tid] = sm.ent[tid];
}

// The same for a product's rows, which are in expert order already: m_indptr (NULL: one matrix) is
// checked to rise from 0 to at most R; where it does not, there are no groups and the flag is set.
__global__ __launch_bounds__(kThreads) void product_prepare(Block128RowsArgs g) {
    __shared__ int at[257], sums[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x > 0) {
        int rows = g.m_indptr ? g.m_indptr[g.E] : g.R;
        rows = rows < 0 ? 0 : rows < g.R ? rows : g.R;
        quantize_rows(g.x, (int64_t)rows * (g.K / 128), (int64_t)(blockIdx.x - 1) * kThreads + tid,
                      (int64_t)(gridDim.x - 1) * kThreads, g.xq, g.xs);
        return;
    }
    for (int i = tid; i <= g.E; i += kThreads) at[i] = g.m_indptr ? g.m_indptr[i] : i == 0 ? 0 : g.R;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i <= g.E; i += kThreads) bad |= i == 0 ? at[0] != 0 : at[i] < at[i - 1] || at[i] > g.R;
    bad = __syncthreads_or(bad);
    Groups* out = static_cast<Groups*>(g.groups);
    const int count = !bad && tid < g.E ? at[tid + 1] - at[tid] : 0, own = (count + kRows - 1) / kRows;
    int incl = own;
    for (int off = 1; off < MOE_WAVE; off <<= 1) {
        const int v = __shfl_up(incl, off, MOE_WAVE);
        if (lane >= off) incl += v;
    }
    if (lane == MOE_WAVE - 1) sums[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += sums[w];
    for (int i = 0; i < own; ++i)
        out->g[incl - own + i] = make_int4(tid, at[tid] + i * kRows, count - i * kRows < kRows ? count - i * kRows : kRows, 0);
    if (tid == kThreads - 1) {
        out->n = incl;
        if (bad && g.status) atomicOr(g.status, kDevBadIndptr);
    }
    out->ent[tid] = tid;
}

// One group of entries times kTiles tiles of 16 weight rows: this wave's share s0 .. s1 of K's S steps.
// Tile t's rows start at row0(t) of the expert's matrix; rows 16 n of one tile lie in one square.
// ro, so: this lane's byte offsets of its row of codes and scales (kNoRow: none).
template <int kTiles> struct Operands8 {
    i32x4_t c[kTiles][2], x[2];
    float xs, ws[kTiles];
};
template <int kTiles, bool kExact, typename Row0>
__device__ __forceinline__ void tile_products(f32x4_t (&acc)[kTiles], __amdgpu_buffer_rsrc_t codes, const float* scales,
                                              Row0&& row0, int K, __amdgpu_buffer_rsrc_t rows, __amdgpu_buffer_rsrc_t row_scales,
                                              uint32_t ro, uint32_t so, int s0, int s1) {
    constexpr int kDepth = kTiles == 1 ? 4 : 2;          // operand sets, all but one on their way (kAhead of run_items at most)
    const int lane = threadIdx.x & 63, S = K / 128;
    uint32_t co = line_offset(K);
    ro += 16u * (lane >> 4);
    auto load = [&](Operands8<kTiles>& w, int s) {
        if (s >= s1) co = ro = so = kNoRow;              // past the last step: no memory is read
        const int at = s < s1 ? s : s0;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) w.c[t][h] = load16(codes, co, (row0(t) + 8 * h) * K + 128 * s, kNonTemporal);
#pragma unroll
        for (int h = 0; h < 2; ++h) w.x[h] = load16(rows, ro, 128 * s + 64 * h, 0);
        w.xs = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_scales, so, 4 * s, 0));
#pragma unroll
        for (int t = 0; t < kTiles; ++t) w.ws[t] = scales[row0(t) / 128 * S + at];
    };
    auto products = [&](const Operands8<kTiles>& w) {
        const i32x8_t x = join(w.x[0], w.x[1]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const f32x4_t p = mma<kExact>(join_lines(w.c[t][0], w.c[t][1]), x);
            const float f = w.xs * w.ws[t];
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[t][z] = __builtin_fmaf(p[z], f, acc[t][z]);
        }
    };
    if (s0 >= s1) return;
    Operands8<kTiles> w[kDepth];
#pragma unroll
    for (int u = 0; u < kDepth - 1; ++u) load(w[u], s0 + u);
    for (int s = s0; s < s1; s += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            if (s + u >= s1) return;
            load(w[(u + kDepth - 1) % kDepth], s + u + kDepth - 1);
            products(w[u]);
        }
    }
}

// The items (group, kTiles tiles) of this workgroup: its number in the launch and every (number of
// workgroups)-th.  Its four waves take a quarter of K each; their partial sums meet in LDS, where
// store(entries, how many, item of the group, part, lane) adds them in wave order.
template <int kTiles> struct Partials8 {
    f32x4_t p[2][kWaves][kTiles][MOE_WAVE];
};
template <int kTiles>
__device__ __forceinline__ f32x4_t sum_waves(const f32x4_t (&p)[kWaves][kTiles][MOE_WAVE], int t) {
    const int lane = threadIdx.x & 63;
    f32x4_t s = p[0][t][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += p[w][t][lane];
    return s;
}
template <int kTiles, bool kExact, typename Row0, typename Row, typename Store>
__device__ __forceinline__ void run_items(const Groups* groups, Partials8<kTiles>& part, const uint8_t* codes, const float* scales,
                                          int N, int K, int per, const uint8_t* rows, const float* row_scales, uint32_t nrows,
                                          Row0&& row0, Row&& row, Store&& store) {
    const int lane = threadIdx.x & 63, col = lane & 15, S = K / 128;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
    // The loads ahead of tile_products pass the last step by up to kAhead, at kNoRow: with their scalar offsets inside the range,
    // they are past its end whether it counts these or not.  Lanes with a row stay within the rows.
    constexpr uint32_t kAhead = 4;
    const __amdgpu_buffer_rsrc_t rr = rows_rsrc(rows, nrows * (uint32_t)K + 128u * kAhead);
    const __amdgpu_buffer_rsrc_t sr = rows_rsrc(row_scales, (nrows * (uint32_t)S + kAhead) * 4u);
    const int items = __builtin_amdgcn_readfirstlane(groups->n) * per;
    int half = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int q = item / per, blk = item - q * per;
        const int e = __builtin_amdgcn_readfirstlane(groups->g[q].x), first = __builtin_amdgcn_readfirstlane(groups->g[q].y);
        const int M = __builtin_amdgcn_readfirstlane(groups->g[q].z);
        const uint32_t r = col < M ? (uint32_t)row(groups->ent[first + col]) : 0u;
        f32x4_t acc[kTiles] = {};
        tile_products<kTiles, kExact>(acc, rows_rsrc(codes + (size_t)e * N * K, (uint32_t)N * (uint32_t)K),
                              scales + (size_t)e * (N / 128) * S, [&](int t) { return row0(blk, t); }, K, rr, sr,
                              col < M ? r * (uint32_t)K : kNoRow, col < M ? r * (uint32_t)S * 4u : kNoRow, s0, s1);
        // one barrier: the other half is written next, and read only after the next barrier
#pragma unroll
        for (int t = 0; t < kTiles; ++t) part.p[half][wave][t][lane] = acc[t];
        __syncthreads();
        store(col < M ? groups->ent[first + col] : -1, blk, part.p[half]);
        half ^= 1;
    }
}

constexpr int kTiles = 4, kWGs = 4;

// a [entry, I] in FP32: an item is 32 outputs, tiles 0 and 1 their gate rows, 2 and 3 their up rows
template <int kAct>
__global__ __launch_bounds__(kThreads, kWGs) void decode8_w13(DecodeArgs g) {
    __shared__ Partials8<kTiles> part;
    const int wave = threadIdx.x >> 6, quad = (threadIdx.x & 63) >> 4, I = g.I, k = g.k;
    run_items<kTiles, true>(static_cast<const Groups*>(g.groups), part, reinterpret_cast<const uint8_t*>(g.w13),
                      reinterpret_cast<const float*>(g.w13_scale), 2 * I, g.d, I / 32, g.xq, g.xs, (uint32_t)g.T,
                      [&](int blk, int t) { return (t >> 1) * I + 32 * blk + 16 * (t & 1); },
                      [&](int entry) { return entry / k; },
                      [&](int entry, int blk, const f32x4_t (&p)[kWaves][kTiles][MOE_WAVE]) {
        if (wave >= 2) return;
        const f32x4_t gate = sum_waves<kTiles>(p, wave), up = sum_waves<kTiles>(p, 2 + wave);
        if (entry < 0) return;
        f32x4_t v;
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] = act_f<kAct>(gate[z]) * up[z];
        *reinterpret_cast<f32x4_t*>(g.a32 + (size_t)entry * I + 32 * blk + 16 * wave + 4 * quad) = v;
    });
}

// o [entry, d] in FP32
__global__ __launch_bounds__(kThreads, kWGs) void decode8_w2(DecodeArgs g) {
    __shared__ Partials8<kTiles> part;
    const int wave = threadIdx.x >> 6, quad = (threadIdx.x & 63) >> 4, d = g.d;
    run_items<kTiles, false>(static_cast<const Groups*>(g.groups), part, reinterpret_cast<const uint8_t*>(g.w2),
                      reinterpret_cast<const float*>(g.w2_scale), d, g.I, d / 64, g.aq, g.as, (uint32_t)(g.T * g.k),
                      [](int blk, int t) { return 64 * blk + 16 * t; }, [](int entry) { return entry; },
                      [&](int entry, int blk, const f32x4_t (&p)[kWaves][kTiles][MOE_WAVE]) {
        const f32x4_t v = sum_waves<kTiles>(p, wave);
        if (entry >= 0) *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(g.o) + (size_t)entry * d + 64 * blk + 16 * wave + 4 * quad) = v;
    });
}

// y [row, N] in BF16.  kT = 1 where items of 64 weight rows would be fewer than the compute units
template <int kT>
__global__ __launch_bounds__(kThreads, kWGs) void product_rows(Block128RowsArgs g) {
    __shared__ Partials8<kT> part;
    const int wave = threadIdx.x >> 6, quad = (threadIdx.x & 63) >> 4, N = g.N;
    run_items<kT, false>(static_cast<const Groups*>(g.groups), part, g.w, g.ws, N, g.K, N / (16 * kT), g.xq, g.xs, (uint32_t)g.R,
                  [](int blk, int t) { return 16 * (kT * blk + t); }, [](int entry) { return entry; },
                  [&](int entry, int blk, const f32x4_t (&p)[kWaves][kT][MOE_WAVE]) {
        if (wave >= kT) return;
        const f32x4_t v = sum_waves<kT>(p, wave);
        if (entry >= 0)
            *reinterpret_cast<uint2*>(g.y + (size_t)entry * N + 16 * (kT * blk + wave) + 4 * quad) =
                make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    });
}

// ---- one token

// 4 blocks of a row in 8 bits, into this wave's 512 bytes of LDS; returns the scale of the lane's block
// (lanes 16 j .. 16 j + 15: block j)
__device__ __forceinline__ float stage_bf16(const uint4 v, char* at) {
    const float s = block_scale(max16(bf16_amax_bits(v)));
    *reinterpret_cast<uint2*>(at + 8 * (threadIdx.x & 63)) = block_codes8(v, s, block_inverse(s));
    return s;
}
__device__ __forceinline__ float stage_f32(f32x4_t a, f32x4_t b, char* at) {
    uint32_t top = 0;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        const uint32_t ma = __float_as_uint(a[z]) & 0x7FFFFFFFu, mb = __float_as_uint(b[z]) & 0x7FFFFFFFu;
        top = top > ma ? top : ma;
        top = top > mb ? top : mb;
    }
    const float s = block_scale(max16(top)), inv = block_inverse(s);
    *reinterpret_cast<uint2*>(at + 8 * (threadIdx.x & 63)) =
        make_uint2(block_codes4(a[0], a[1], a[2], a[3], s, inv), block_codes4(b[0], b[1], b[2], b[3], s, inv));
    return s;
}
__device__ __forceinline__ float of_block(float s, int j) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s), 16 * j));
}

// kT tiles of 16 weight rows times one row in BF16: this wave's share s0 .. s1 of K's steps, kChunk at a time.
// The row's piece is loaded before the weights, so that it is quantized while they are on their way (loads
// come back in order).  Every column of the instruction is the row.  row0(t): tile t's first row; scale(t): the
// scales of its squares along K.
template <int kT, int kChunk, bool kExact, typename Row0, typename Scale>
__device__ __forceinline__ void one_row(f32x4_t (&acc)[kT], __amdgpu_buffer_rsrc_t codes, Row0&& row0, Scale&& scale, int K,
                                        __amdgpu_buffer_rsrc_t xr, char* stage, int s0, int s1) {
    static_assert(kChunk % 4 == 0, "a load of the row is four blocks");
    const int lane = threadIdx.x & 63, quad = lane >> 4;
    const uint32_t co = line_offset(K);
    for (int s = s0; s < s1; s += kChunk) {
        i32x4_t c[kT][kChunk][2], x[kChunk / 4];
        float f[kT][kChunk];
        // past s1 a row's pieces belong to the next wave, or lie past the resource's end: not used.  (The whole offset is the
        // lane's, which a resource's range is checked against whether it counts the scalar offset or not.)
#pragma unroll
        for (int h = 0; h < kChunk / 4; ++h) x[h] = load16(xr, 16u * lane + 256u * (s + 4 * h), 0, 0);
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (s + j < s1)
#pragma unroll
                for (int t = 0; t < kT; ++t) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) c[t][j][h] = load16(codes, co, (row0(t) + 8 * h) * K + 128 * (s + j), kNonTemporal);
                    f[t][j] = scale(t)[s + j];
                }
        float xs[kChunk / 4];
#pragma unroll
        for (int h = 0; h < kChunk / 4; ++h) xs[h] = stage_bf16(__builtin_bit_cast(uint4, x[h]), stage + 512 * h);
        wave_fence();
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
            if (s + j < s1) {
                const char* b = stage + 128 * j + 16 * quad;
                const i32x8_t xv = join(*reinterpret_cast<const i32x4_t*>(b), *reinterpret_cast<const i32x4_t*>(b + 64));
                const float sx = of_block(xs[j / 4], j & 3);
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    const f32x4_t p = mma<kExact>(join_lines(c[t][j][0], c[t][j][1]), xv);
                    const float ff = sx * f[t][j];
#pragma unroll
                    for (int z = 0; z < 4; ++z) acc[t][z] = __builtin_fmaf(p[z], ff, acc[t][z]);
                }
            }
        wave_fence();
    }
}

// A workgroup per (slot, 16 outputs), its four waves a quarter of K each.
template <int kAct>
__global__ __launch_bounds__(kThreads, 3) void decode8_w13_one(DecodeArgs g) {
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    __shared__ __attribute__((aligned(16))) char stage[kWaves][512];
    int par = 0;
    if (blockIdx.x == 0 && blockIdx.y == 0) decode_flags_one_token(g);
    const int slot = blockIdx.y, e = g.ids[slot];
    if ((unsigned)e >= (unsigned)g.E) return;
    const int lane = threadIdx.x & 63, quad = lane >> 4, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int d = g.d, S = d / 128, i0 = 16 * blockIdx.x;
    const size_t matrix = (size_t)2 * g.I * d;
    const float* ws = reinterpret_cast<const float*>(g.w13_scale) + (size_t)e * (2 * g.I / 128) * S + i0 / 128 * S;
    f32x4_t acc[2] = {};
    one_row<2, 4, true>(acc, rows_rsrc(reinterpret_cast<const uint8_t*>(g.w13) + e * matrix, (uint32_t)matrix),
                  [&](int t) { return t * g.I + i0; }, [&](int t) { return ws + t * (g.I / 128 * S); }, d,
                  rows_rsrc(g.x, (uint32_t)d * 2u), stage[wave], S * wave / kWaves, S * (wave + 1) / kWaves);
    const f32x4_t gate = reduce_waves<true>(acc[0], red, par), uv = reduce_waves<true>(acc[1], red, par);
    if (threadIdx.x < MOE_WAVE && (lane & 15) == 0) {
        f32x4_t v;
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] = act_f<kAct>(gate[z]) * uv[z];
        *reinterpret_cast<f32x4_t*>(g.a32 + (size_t)slot * g.I + i0 + 4 * quad) = v;
    }
}

// One row through one matrix: a workgroup for 16 outputs.
__global__ __launch_bounds__(kThreads, 3) void product_one(Block128RowsArgs g) {
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    __shared__ __attribute__((aligned(16))) char stage[kWaves][1024];
    int par = 0;
    const int lane = threadIdx.x & 63, quad = lane >> 4, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int K = g.K, S = K / 128, n0 = 16 * blockIdx.x;
    const float* ws = g.ws + n0 / 128 * S;
    f32x4_t acc[1] = {};
    one_row<1, 8, false>(acc, rows_rsrc(g.w, (uint32_t)g.N * (uint32_t)K), [&](int) { return n0; }, [&](int) { return ws; }, K,
                  rows_rsrc(g.x, (uint32_t)K * 2u), stage[wave], S * wave / kWaves, S * (wave + 1) / kWaves);
    const f32x4_t v = reduce_waves<true>(acc[0], red, par);
    if (threadIdx.x < MOE_WAVE && (lane & 15) == 0)
        *reinterpret_cast<uint2*>(g.y + n0 + 4 * quad) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// W2 of all k experts and the combine, 8 output features per workgroup: rows 0 .. 7 of the instruction
// are those features of expert 2 p, rows 8 .. 15 of expert 2 p + 1; even columns are a_2p, odd ones
// a_2p+1 (half of the results belong to no expert and are not used).
__global__ __launch_bounds__(kThreads, 2) void decode8_w2_one(DecodeArgs g) {
    constexpr int kChunk = 8;
    __shared__ __attribute__((aligned(16))) char stage[kWaves][2][128 * kChunk];
    __shared__ float ov[kMaxTopK][8];
    __shared__ float sc[kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 63, row16 = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int d = g.d, I = g.I, k = g.k, S = I / 128, npair = (k + 1) / 2;
    const float score = tid < k ? g.scores[tid] : 0.f;
    const __amdgpu_buffer_rsrc_t ar = rows_rsrc(g.a32, (uint32_t)k * I * 4u);
    auto expert = [&](int j) {
        const int e = j < k ? __builtin_amdgcn_readfirstlane(g.ids[j]) : -1;
        return (unsigned)e < (unsigned)g.E ? e : -1;
    };
    for (int nb = blockIdx.x; nb < d / 8; nb += gridDim.x) {
        const int n0 = nb * 8;
        for (int p = wave; p < npair; p += kWaves) {
            const int ex = expert(2 * p), ey = expert(2 * p + 1);
            const int vx = ex >= 0 ? ex : 0, vy = ey >= 0 ? ey : 0;
            const uint8_t* w2 = reinterpret_cast<const uint8_t*>(g.w2) + (size_t)n0 * I + line_offset(I);
            const uint8_t* codes[2] = {w2 + (size_t)vx * d * I, w2 + (size_t)vy * d * I};
            const float* w2s = reinterpret_cast<const float*>(g.w2_scale);
            const float* wsx = w2s + ((size_t)vx * (d / 128) + n0 / 128) * S;
            const float* wsy = w2s + ((size_t)vy * (d / 128) + n0 / 128) * S;
            // a row of no valid expert was not written: zeros
            const uint32_t ax = ex >= 0 ? (uint32_t)(2 * p * I) * 4u + 32u * lane : kNoRow;
            const uint32_t ay = ey >= 0 ? (uint32_t)((2 * p + 1) * I) * 4u + 32u * lane : kNoRow;
            f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
            // kChunk steps at a time; a's pieces are loaded before the weights, as in one_row
            for (int s = 0; s < S; s += kChunk) {
                i32x4_t c[kChunk][2], a[kChunk / 4][4];
                float fx[kChunk], fy[kChunk];
                // (a load's blocks past S are another row's, or what follows a in the workspace: not used)
#pragma unroll
                for (int q = 0; q < kChunk / 4; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        a[q][h] = load16(ar, s + 4 * q < S ? ax + 16u * h : kNoRow, 512 * (s + 4 * q), 0);
                        a[q][2 + h] = load16(ar, s + 4 * q < S ? ay + 16u * h : kNoRow, 512 * (s + 4 * q), 0);
                    }
#pragma unroll
                for (int j = 0; j < kChunk; ++j)
                    if (s + j < S) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            c[j][h] = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(codes[h] + 128 * (s + j)));
                        fx[j] = wsx[s + j];
                        fy[j] = wsy[s + j];
                    }
                float sx[kChunk / 4], sy[kChunk / 4];
#pragma unroll
                for (int q = 0; q < kChunk / 4; ++q) {
                    sx[q] = stage_f32(__builtin_bit_cast(f32x4_t, a[q][0]), __builtin_bit_cast(f32x4_t, a[q][1]), stage[wave][0] + 512 * q);
                    sy[q] = stage_f32(__builtin_bit_cast(f32x4_t, a[q][2]), __builtin_bit_cast(f32x4_t, a[q][3]), stage[wave][1] + 512 * q);
                }
                wave_fence();
#pragma unroll
                for (int j = 0; j < kChunk; ++j)
                    if (s + j < S) {
                        const char* b = stage[wave][row16 & 1] + 128 * j + 16 * quad;
                        const f32x4_t r = mma128(join_lines(c[j][0], c[j][1]), join(*reinterpret_cast<const i32x4_t*>(b),
                                                                              *reinterpret_cast<const i32x4_t*>(b + 64)));
                        const float f = quad < 2 ? fx[j] * of_block(sx[j / 4], j & 3) : fy[j] * of_block(sy[j / 4], j & 3);
#pragma unroll
                        for (int z = 0; z < 4; ++z) acc[z] = __builtin_fmaf(r[z], f, acc[z]);
                    }
                wave_fence();
            }
            // column 0's rows 0 .. 7, column 1's rows 8 .. 15
            if (row16 == quad >> 1) {
                const int j = 2 * p + row16;
                if (j < k)
#pragma unroll
                    for (int z = 0; z < 4; ++z) ov[j][4 * (quad & 1) + z] = (row16 ? ey : ex) >= 0 ? acc[z] : 0.f;
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

template <class K> hipError_t launch_items(K kernel, const DecodeArgs& g, int per, int num_cu, hipStream_t s) {
    const int R = g.T * g.k, groups = R < g.E + R / kRows ? R : g.E + R / kRows;   // at most
    const int items = groups * per, cap = kWGs * num_cu;
    hipLaunchKernelGGL(kernel, dim3(items < cap ? items : cap), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}
template <int kAct> hipError_t launch_w13(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T == 1) {
        hipLaunchKernelGGL(decode8_w13_one<kAct>, dim3(g.I / 16, g.k), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    const int pieces = (g.T * (g.d / 8) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(decode8_prepare, dim3(1 + (pieces < 1024 ? pieces : 1024)), dim3(kThreads), 0, s, g);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_items(decode8_w13<kAct>, g, g.I / 32, num_cu, s);
}

}  // namespace

hipError_t launch_decode8_w13(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T * g.k > kMaxDecodeRows || g.E > 256 || g.d % 128 != 0 || g.I % 128 != 0) return hipErrorInvalidValue;
    if (g.act == kActGeGLU) return launch_w13<kActGeGLU>(g, num_cu, s);
    if (g.act == kActReGLU) return launch_w13<kActReGLU>(g, num_cu, s);
    return launch_w13<kActSwiGLU>(g, num_cu, s);
}

hipError_t launch_decode8_w2(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T == 1) {
        if (g.k > kMaxTopK) return hipErrorInvalidValue;
        const int cap = 3 * num_cu, grid = g.d / 8;
        hipLaunchKernelGGL(decode8_w2_one, dim3(grid < cap ? grid : cap), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    hipError_t e = launch_block128_rows_f32(g.a32, (int64_t)g.T * g.k, g.I, g.aq, g.as, s);
    if (e == hipSuccess) e = launch_items(decode8_w2, g, g.d / 64, num_cu, s);
    return e != hipSuccess ? e : launch_decode4_combine(g, s);
}

hipError_t launch_block128_few_rows(const Block128RowsArgs& g, int num_cu, hipStream_t s) {
    if (g.R <= 0) return hipSuccess;
    if (g.R > kMaxDecodeRows || g.E <= 0 || g.E > 256 || g.N % 128 != 0 || g.K % 128 != 0) return hipErrorInvalidValue;
    if (g.R == 1 && !g.m_indptr) {
        hipLaunchKernelGGL(product_one, dim3(g.N / 16), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    const int pieces = (g.R * (g.K / 8) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(product_prepare, dim3(1 + (pieces < 1024 ? pieces : 1024)), dim3(kThreads), 0, s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int groups = g.R < g.E + g.R / kRows ? g.R : g.E + g.R / kRows, cap = kWGs * num_cu;   // at most
    if (groups * (g.N / 64) >= num_cu) {
        const int items = groups * (g.N / 64);
        hipLaunchKernelGGL(product_rows<4>, dim3(items < cap ? items : cap), dim3(kThreads), 0, s, g);
    } else {
        const int items = groups * (g.N / 16);
        hipLaunchKernelGGL(product_rows<1>, dim3(items < cap ? items : cap), dim3(kThreads), 0, s, g);
    }
    return hipGetLastError();
}

}  // namespace moe
