// decode_common.h -- what the weight-streaming kernels of small batches share (BF16 weights in
// decode.hip, 4-bit weights in decode_mxfp4.hip, 8-bit weights with a scale per 128 in
// decode_block128.hip): one token's routing flags, the row resource, the sum over a K split and the
// routed entries in expert order.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / MOE_WAVE;

// Routing flags for the one-token path (block 0 only): ids out of range or repeated.
__device__ void decode_flags_one_token(const DecodeArgs& g) {
    const int j = threadIdx.x;
    if (j < g.k) {
        const int e = g.ids[j];
        int bad = (unsigned)e < (unsigned)g.E ? 0 : kDevIdOutOfRange;
        for (int jj = 0; jj < j; ++jj)
            if (bad == 0 && g.ids[jj] == e) bad |= kDevIdDuplicate;
        if (bad) atomicOr(g.status, bad);
    }
}

// Raw buffer resource over `bytes` bytes at base (a uniform kernel argument).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kNoRow = 0x80000000u;   // beyond every resource: reads zeros

// K split: the four waves' partial sums added in wave order; the total is valid in
// wave 0.  red is double-buffered by the caller (`par`), so one barrier per call
// suffices: a buffer is rewritten only after the next call's barrier, which wave 0
// reaches after it has read the buffer.
template <bool kSplit>
__device__ __forceinline__ f32x4_t reduce_waves(f32x4_t acc, f32x4_t (*red)[kWaves][MOE_WAVE], int& par) {
    if (!kSplit) return acc;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    red[par][wave][lane] = acc;
    __syncthreads();
    f32x4_t s = red[par][0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[par][w][lane];
    par ^= 1;
    return s;
}

// The routed entries sorted by expert, in groups of at most 16 entries of one expert.
constexpr int kRows = 16;
struct Sorted {
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
__device__ __forceinline__ void sort_entries(Sorted& sm, const DecodeArgs& g, bool report) {
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

}  // namespace
}  // namespace moe
