// decode_mxfp4.hip -- weight-streaming path for expert weights in MXFP4 (mxfp4.hip's layout),
// T*k <= 256 routed rows.
//
// The same launches as with BF16 weights (decode.hip): W13 with the activation, then for one
// token W2 with the combine, else W2 and a combine.  a is rounded to BF16, the operand type of
// the W2 products, and its remainder, rounded too, is an operand row of its own: 16 bits of a, so
// that a token's y is as exact beside others as alone.  The experts' outputs o stay in FP32 until
// the one rounding of y.  The time is that of streaming 4.25 bits
// for each weight of the active experts: 128 experts of d = 2048, I = 768, k = 8, one token 5.2 and
// 4.7 us for 13.4 and 6.7 MB, where starting and the chain of loads are what is left; 32 tokens on
// 59 experts 22.0, 15.5 and (combine) 4.5 us for 99 and 49 MB (4.5 and 3.2 TB/s).  The remainders
// cost W2 2.1 us of that.
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

// One token: acc += A * B over the tiles s0 .. s1 - 1 of a row tile, with kRowsUsed operand rows
// (1 or 4).  codes and words point at this lane's piece of the first tile; row(r): byte offset
// of operand row r in ars (kNoRow: zeros).  The rows come through LDS (`stage`, this wave's own),
// 64 consecutive pieces a load: as MFMA operands straight from memory, with 60 of 64 lanes
// masked, they are four loads for each load of codes.
template <int kRowsUsed, int B> struct Stage4 {
    static constexpr int kRow = B * 256 + 16;          // bytes; padded: the rows' pieces meet different banks
    char b[kRowsUsed * kRow];
};
template <int kRowsUsed, int B, typename Row>
__device__ __forceinline__ f32x4_t mma_tiles(const uint8_t* codes, const uint32_t* words, int groups,
                                             __amdgpu_buffer_rsrc_t ars, Row&& row, Stage4<kRowsUsed, B>& stage, int s0, int s1) {
    static_assert(B % 4 == 0, "whole loads of a row");
    constexpr int kLoads = kRowsUsed * B / 4;          // of 1 KiB
    const int lane = threadIdx.x & 63;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    const char* mine = stage.b + (lane & (kRowsUsed - 1)) * Stage4<kRowsUsed, B>::kRow + 64 * (lane >> 4);
    for (int s = s0; s < s1; s += B) {
        u32x4_t c[B], x[kLoads];
        uint32_t sb[(B + 3) / 4];
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s + j < s1) c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes + (size_t)(s + j) * 1024));
#pragma unroll
        for (int j = 0; j < B; j += 4)
            if (s + j < s1) sb[j / 4] = scale_bytes(words, s + j, groups);
        // past s1 a row's pieces belong to the next wave's tiles, or the resource's end: not used
#pragma unroll
        for (int p = 0; p < kLoads; ++p) {
            const int at = p % (B / 4) * 1024 + lane * 16;
            x[p] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ars, row(p / (B / 4)) + 256u * s + at, 0, 0));
        }
#pragma unroll
        for (int p = 0; p < kLoads; ++p)
            *reinterpret_cast<u32x4_t*>(stage.b + p / (B / 4) * Stage4<kRowsUsed, B>::kRow + p % (B / 4) * 1024 + lane * 16) = x[p];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < B; ++j)
            if (s + j < s1) {
                const float f = __uint_as_float(((sb[j / 4] >> (8 * (j & 3))) & 0xFFu) << 23);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc = mma_quarter(*reinterpret_cast<const bf16x8_t*>(mine + 256 * j + 16 * i), c[j][i], f, acc);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    return acc;
}

// a[entry][i0 + n] = act(g) u in BF16, from one W13 tile's D: lane l holds rows 4 (l >> 4) + z
// of column n = l & 15, gate columns 0..7 and up columns 8..15.  The remainder goes T*k rows further.
template <int kAct>
__device__ __forceinline__ void store_a(const DecodeArgs& g, const int* ent, int M, int i0, f32x4_t acc, bool lead) {
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
    float up[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) up[z] = __shfl_down(acc[z], 8, 16);
    if (lead && n < 8) {
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int mm = 4 * kq + z;
            if (mm < M) {
                const float v = act_f<kAct>(acc[z]) * up[z];
                const uint32_t hi = f32_to_bf16(v);
                uint16_t* at = g.a + (size_t)ent[mm] * g.I + i0 + n;
                *at = (uint16_t)hi;
                at[(size_t)g.T * g.k * g.I] = (uint16_t)f32_to_bf16(v - bf16_to_f32(hi));
            }
        }
    }
}

// One token: a workgroup per (slot, row tile), its four waves a quarter of K each: every load of
// the launch is in flight at once, and the partial sums meet in LDS.
constexpr int kOneWGs = 3;
template <int kAct>
__global__ __launch_bounds__(kThreads, kOneWGs) void decode4_w13_one(DecodeArgs g) {
    __shared__ f32x4_t red[2][kWaves][MOE_WAVE];
    __shared__ __attribute__((aligned(16))) Stage4<1, 4> stage[kWaves];
    int par = 0;
    if (blockIdx.x == 0 && blockIdx.y == 0) decode_flags_one_token(g);
    const int slot = blockIdx.y, e = g.ids[slot];
    if ((unsigned)e >= (unsigned)g.E) return;
    const int lane = threadIdx.x & 63;
    const int S = g.d / 128, groups = (S + 3) / 4, w = threadIdx.x >> 6;
    const int s0 = __builtin_amdgcn_readfirstlane(S * w / kWaves), s1 = __builtin_amdgcn_readfirstlane(S * (w + 1) / kWaves);
    const size_t tile = (size_t)e * (g.I / 8) + blockIdx.x;
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(g.w13) + tile * S * 1024 + lane * 16;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(g.w13_scale) + tile * groups * 64 + lane;
    const f32x4_t acc = reduce_waves<true>(
        mma_tiles(codes, words, groups, rows_rsrc(g.x, (uint32_t)g.d * 2u), [](int) { return 0u; }, stage[w], s0, s1), red, par);
    store_a<kAct>(g, &slot, 1, blockIdx.x * 8, acc, threadIdx.x < MOE_WAVE);
}

// More tokens: a workgroup's item is (group of entries of one expert, kTiles row tiles), its four
// waves a quarter of K each.  A step is one tile along K: kTiles loads of codes, and four of the routed rows
// that all the tiles share.  Those four are what bounds the kernel when few tiles share them:
// they occupy the address unit as long as four loads of codes.  W13 and W2 at 32 tokens of the
// 128-expert layer, 59 experts active (99 and 49 MB):
//   (W2 without the remainders of a)
//   a wave for each tile over all of K            32.2 and 18.1 us
//   a wave for two, four tiles over all of K      23.6 and 14.0, 25.1 and 13.0
//   four, eight tiles and a quarter of K a wave   21.4 and 13.2, 21.9 and 14.0
// While a step's products run, the next step's operands are in flight, in one of two sets of
// registers that take turns (a copy from one to the other would wait for the loads); a third
// set costs a workgroup a CU and is slower (23.0 and 13.1 us); eight tiles with K in two shares are
// too (64 experts: 22.0 against 19.1 us for W13, 11.7 against 11.4 for W2's six steps).
constexpr int kTiles = 4, kDepth = 2, kWGs = 4;
static_assert(kTiles % kWaves == 0, "a wave adds up whole tiles");
constexpr int kNonTemporal = 2;      // the nt bit of a buffer load
template <int kSets> struct Operands4 {
    u32x4_t c[kTiles];               // codes
    uint32_t sb[kTiles];             // scales, a byte for each of four tiles along K
    bf16x8_t a[kSets][4];            // routed rows
};
struct Partials4 {
    f32x4_t p[2][kWaves][kTiles][MOE_WAVE];
};
// One 16-row group (rows at byte offset ao of ars, kNoRow: none) times the item's tiles: this
// wave's share of K.  codes and words: of the item's first row tile.  kSets = 2: plus the rows
// set_bytes further, the remainders.
template <int kSets>
__device__ __forceinline__ void tile_products(f32x4_t (&acc)[kTiles], const void* codes_base, const void* words_base,
                                              __amdgpu_buffer_rsrc_t ars, uint32_t ao, int set_bytes, int S, int s0, int s1) {
    const int lane = threadIdx.x & 63, groups = (S + 3) / 4;
    // uniform bases and offsets in scalar registers, one 32-bit lane offset each
    const __amdgpu_buffer_rsrc_t codes = rows_rsrc(codes_base, (uint32_t)(kTiles * S) * 1024u);
    const __amdgpu_buffer_rsrc_t words = rows_rsrc(words_base, (uint32_t)(kTiles * groups) * 256u);
    ao += 64u * (lane >> 4);
    uint32_t co = lane * 16, so = lane * 4;
    auto load = [&](Operands4<kSets>& w, int s) {
        if (s >= s1) co = so = ao = kNoRow;              // past the last step: no memory is read
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            w.c[t] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(codes, co, (t * S + s) * 1024, kNonTemporal));
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            w.sb[t] = __builtin_amdgcn_raw_buffer_load_b32(words, so, (t * groups + (s >> 2)) * 256, 0);
#pragma unroll
        for (int h = 0; h < kSets; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w.a[h][i] = __builtin_bit_cast(
                    bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(ars, ao + 16u * i, 256 * s + h * set_bytes, 0));
    };
    auto products = [&](const Operands4<kSets>& w, int s) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const float x = __uint_as_float(((w.sb[t] >> (8 * (s & 3))) & 0xFFu) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < kSets; ++h) acc[t] = mma_quarter(w.a[h][i], w.c[t][i], x, acc[t]);
        }
    };
    Operands4<kSets> w[kDepth];
#pragma unroll
    for (int u = 0; u < kDepth - 1; ++u) load(w[u], s0 + u);
    for (int s = s0; s < s1; s += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            if (s + u >= s1) return;
            load(w[(u + kDepth - 1) % kDepth], s + u + kDepth - 1);
            products(w[u], s + u);
        }
    }
}

// The routed entries sorted by expert, in groups of at most 16 entries of one expert.
constexpr int kRows = 16, kHalf = 8;
struct Sorted4 {
    int cnt[256];                    // entries per expert, a byte for each of the four waves
    int ids[kMaxDecodeRows];         // for the routing flags
    int pfx[257];                    // entries of expert e: ent[pfx[e] .. pfx[e + 1])
    int ent[kMaxDecodeRows];         // ascending within an expert
    uint16_t group[256 + kMaxDecodeRows / kRows];   // expert | number of the group << 8, ascending
    int wsum[kWaves];
    int groups;
};
// Every workgroup sorts for itself; the one with `report` sets the routing flags.  An entry's rank
// among its expert's comes from a ballot for each bit of the id, which finds the wave's entries
// of the same expert, and the counts of the waves before.  (Comparing with every earlier entry,
// up to 255, made W13 and W2 of 32 tokens 4.3 and 8.2 us longer.)
__device__ __forceinline__ void sort_entries(Sorted4& sm, const DecodeArgs& g, bool report) {
    static_assert(kThreads == 256 && kMaxDecodeRows == 256, "a thread for each expert and entry");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, R = g.T * g.k;
    const int id = tid < R ? g.ids[tid] : -1;
    const int e = (unsigned)id < (unsigned)g.E ? id : -1;
    sm.cnt[tid] = 0;
    if (report) sm.ids[tid] = e;
    __syncthreads();
    uint64_t same = __ballot(e >= 0);
#pragma unroll
    for (int bit = 1; bit < 256; bit <<= 1) {
        const uint64_t ones = __ballot((e & bit) != 0);
        same &= (e & bit) != 0 ? ones : ~ones;
    }
    const int rank = __popcll(same & lanemask_lt());
    if (e >= 0 && rank == 0) atomicAdd(&sm.cnt[e], (int)((uint32_t)__popcll(same) << (8 * wave)));   // at most 64
    if (report && tid < R) {
        int bad = e >= 0 ? 0 : kDevIdOutOfRange;
        const int t = tid / g.k, j = tid - t * g.k;
        for (int jj = 0; jj < j; ++jj)
            if (e >= 0 && sm.ids[t * g.k + jj] == e) bad |= kDevIdDuplicate;
        if (bad) atomicOr(g.status, bad);
    }
    __syncthreads();
    // thread tid for expert tid: prefix sums of the entries and (in the upper half) the groups
    auto bytes = [](uint32_t w) { return (int)((w & 0xFF) + (w >> 8 & 0xFF) + (w >> 16 & 0xFF) + (w >> 24)); };
    const int count = bytes((uint32_t)sm.cnt[tid]);
    const int own = count | (count + kRows - 1) / kRows << 16;
    int incl = own;
    for (int off = 1; off < MOE_WAVE; off <<= 1) {
        const int v = __shfl_up(incl, off, MOE_WAVE);
        if (lane >= off) incl += v;
    }
    if (lane == MOE_WAVE - 1) sm.wsum[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += sm.wsum[w];
    const int before = incl - own;
    sm.pfx[tid] = before & 0xFFFF;
    for (int i = 0; i < own >> 16; ++i) sm.group[(before >> 16) + i] = (uint16_t)(tid | i << 8);
    if (tid == 255) {
        sm.pfx[256] = incl & 0xFFFF;
        sm.groups = incl >> 16;
    }
    __syncthreads();
    if (e >= 0) {
        const uint32_t earlier = wave > 0 ? (uint32_t)sm.cnt[e] & ((1u << (8 * wave)) - 1) : 0u;
        sm.ent[sm.pfx[e] + bytes(earlier) + rank] = tid;
    }
    __syncthreads();
}

// The items (group of entries, kTiles row tiles) of this workgroup, its number in the launch and
// every (number of workgroups)-th; store(entries, how many, row tile, sums) by the wave that has
// added up the tile's four partial sums, in wave order.  row(entry): byte offset of its operand
// row.  kRest: every row has a remainder rest_bytes further.  Those of up to 8 entries are operand rows
// 8 .. 15 of the same loads and MFMAs, and store adds the two halves of the sums; groups of more
// entries have a second set of operands.  (W2 in groups of 8 entries throughout: 256 entries of 8
// experts, d = 4096, I = 1024, 50.8 us a call against 48.4; without remainders 43.5.)
template <bool kRest, typename Row, typename Store>
__device__ __forceinline__ void run_items(const Sorted4& sm, Partials4& part, const void* codes, const void* words,
                                          __amdgpu_buffer_rsrc_t ars, int rest_bytes, int nblk, int S, Row&& row, Store&& store) {
    const int lane = threadIdx.x & 63, n = lane & 15, word_bytes = (S + 3) / 4 * 256;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int s0 = S * wave / kWaves, s1 = S * (wave + 1) / kWaves;
    const int per = nblk / kTiles, items = __builtin_amdgcn_readfirstlane(sm.groups) * per;
    int half = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int q = item / per, blk = (item - q * per) * kTiles;
        const int group = __builtin_amdgcn_readfirstlane((int)sm.group[q]), e = group & 255, m0 = (group >> 8) * kRows;
        const int first = __builtin_amdgcn_readfirstlane(sm.pfx[e]) + m0;
        const int left = __builtin_amdgcn_readfirstlane(sm.pfx[e + 1]) - first, M = left < kRows ? left : kRows;
        const size_t tile = (size_t)e * nblk + blk;
        const bool both = kRest && M <= kHalf;
        const int m = both ? n % kHalf : n;
        const uint32_t ao = m < M ? row(sm.ent[first + m]) + (m < n ? (uint32_t)rest_bytes : 0u) : kNoRow;
        f32x4_t acc[kTiles] = {};
        const uint8_t* c0 = static_cast<const uint8_t*>(codes) + tile * S * 1024;
        const uint8_t* w0 = static_cast<const uint8_t*>(words) + tile * word_bytes;
        if (!kRest || both) tile_products<1>(acc, c0, w0, ars, ao, 0, S, s0, s1);
        else tile_products<2>(acc, c0, w0, ars, ao, rest_bytes, S, s0, s1);
        // one barrier: the other half is written next, and read only after the next barrier
#pragma unroll
        for (int t = 0; t < kTiles; ++t) part.p[half][wave][t][lane] = acc[t];
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kTiles; t += kWaves) {
            f32x4_t sum = part.p[half][0][t + wave][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) sum += part.p[half][w][t + wave][lane];
            store(sm.ent + first, M, blk + t + wave, sum);
        }
        half ^= 1;
    }
}

template <int kAct>
__global__ __launch_bounds__(kThreads, kWGs) void decode4_w13(DecodeArgs g) {
    __shared__ Sorted4 sm;
    __shared__ Partials4 part;
    sort_entries(sm, g, blockIdx.x == 0);
    run_items<false>(sm, part, g.w13, g.w13_scale, rows_rsrc(g.x, (uint32_t)g.T * g.d * 2u), 0, g.I / 8, g.d / 128,
                     [&](int entry) { return (uint32_t)(entry / g.k * g.d) * 2u; },
                     [&](const int* ent, int M, int tile, f32x4_t sum) { store_a<kAct>(g, ent, M, tile * 8, sum, true); });
}

__global__ __launch_bounds__(kThreads, kWGs) void decode4_w2(DecodeArgs g) {
    __shared__ Sorted4 sm;
    __shared__ Partials4 part;
    sort_entries(sm, g, false);
    float* o = reinterpret_cast<float*>(g.o);
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4, d = g.d, set = g.T * g.k * g.I * 2;
    run_items<true>(sm, part, g.w2, g.w2_scale, rows_rsrc(g.a, 2u * set), set, d / 16, g.I / 128,
                    [&](int entry) { return (uint32_t)(entry * g.I) * 2u; },
                    [&](const int* ent, int M, int tile, f32x4_t sum) {
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const float rest = __shfl_xor(sum[z], 32, MOE_WAVE);       // rows 8 .. 15 at rows 0 .. 7
            if (4 * kq + z < M) o[(size_t)ent[4 * kq + z] * d + tile * 16 + n] = M <= kHalf ? sum[z] + rest : sum[z];
        }
    });
}

// One token: W2 of all k experts and the combine, 8 output features per workgroup.  As in the
// BF16 kernel, experts 2p and 2p + 1 share one MFMA: columns 0..7 are rows n0 .. n0 + 7 of
// expert 2p, columns 8..15 the same rows of expert 2p + 1, A row 0 is a_2p and row 1 a_2p+1, rows
// 2 and 3 their remainders.
__global__ __launch_bounds__(kThreads, 1) void decode4_w2_one(DecodeArgs g) {
    __shared__ __attribute__((aligned(16))) Stage4<4, 8> stage[kWaves];
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
            auto row = [&](int r) {
                return (r & 1 ? vy : vx) ? (uint32_t)((2 * p + (r & 1) + (r & 2 ? k : 0)) * I) * 2u : kNoRow;
            };
            const f32x4_t acc = mma_tiles(codes, words, groups, rows_rsrc(g.a, (uint32_t)k * I * 4u), row, stage[wave], 0, S);
            if (kq == 0) {
                if (n < 8 && 2 * p < k) ov[2 * p][n] = vx ? acc[0] + acc[2] : 0.f;
                if (n >= 8 && 2 * p + 1 < k) ov[2 * p + 1][n - 8] = vy ? acc[1] + acc[3] : 0.f;
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

// y[t] = sum_j s[t][j] o[t*k + j] in FP32, j ascending from +0.0; four features a thread.  Entries
// of invalid ids add nothing (no product has written their o)
__global__ __launch_bounds__(MOE_WAVE) void decode4_combine(DecodeArgs g) {
    const int t = blockIdx.y, n = (blockIdx.x * MOE_WAVE + threadIdx.x) * 4;
    if (n >= g.d) return;
    const float* o = reinterpret_cast<const float*>(g.o) + (size_t)t * g.k * g.d + n;
    f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int j = 0; j < g.k; ++j) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(o + (size_t)j * g.d);
        const float s = g.scores[t * g.k + j];
        const bool valid = (unsigned)g.ids[t * g.k + j] < (unsigned)g.E;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = valid ? __builtin_fmaf(s, v[i], y[i]) : y[i];
    }
    *reinterpret_cast<uint2*>(g.y + (size_t)t * g.d + n) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// a workgroup for each item, as far as they fit the chip together (nblk a multiple of kTiles)
template <class K> hipError_t launch_items(K kernel, const DecodeArgs& g, int nblk, int num_cu, hipStream_t s) {
    const int R = g.T * g.k, groups = R < g.E + R / kRows ? R : g.E + R / kRows;   // at most
    const int items = groups * (nblk / kTiles), cap = kWGs * num_cu;
    hipLaunchKernelGGL(kernel, dim3(items < cap ? items : cap), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}
template <int kAct> hipError_t launch_w13(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T > 1) return launch_items(decode4_w13<kAct>, g, g.I / 8, num_cu, s);
    hipLaunchKernelGGL(decode4_w13_one<kAct>, dim3(g.I / 8, g.k), dim3(kThreads), 0, s, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode4_w13(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T * g.k > kMaxDecodeRows || g.d % 128 != 0 || g.I % 128 != 0) return hipErrorInvalidValue;
    if (g.act == kActGeGLU) return launch_w13<kActGeGLU>(g, num_cu, s);
    if (g.act == kActReGLU) return launch_w13<kActReGLU>(g, num_cu, s);
    return launch_w13<kActSwiGLU>(g, num_cu, s);
}

hipError_t launch_decode4_w2(const DecodeArgs& g, int num_cu, hipStream_t s) {
    if (g.T * g.k <= 0) return hipSuccess;
    if (g.T == 1) {
        if (g.k > kMaxTopK) return hipErrorInvalidValue;
        const int cap = 3 * num_cu, grid = g.d / 8;
        hipLaunchKernelGGL(decode4_w2_one, dim3(grid < cap ? grid : cap), dim3(kThreads), 0, s, g);
        return hipGetLastError();
    }
    const hipError_t e = launch_items(decode4_w2, g, g.d / 16, num_cu, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(decode4_combine, dim3((g.d / 4 + MOE_WAVE - 1) / MOE_WAVE, g.T), dim3(MOE_WAVE), 0, s, g);
    return hipGetLastError();
}

}  // namespace moe
