// decode_common.h -- what the weight-streaming kernels of small batches share (BF16 weights in
// decode.hip, 4-bit weights in decode_mxfp4.hip): one token's routing flags, the row resource and
// the sum over a K split.
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

}  // namespace
}  // namespace moe
