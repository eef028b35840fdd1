// decode_common.h -- what the weight-streaming kernels of small batches share (BF16 weights in
// decode.hip, 4-bit weights in decode_mxfp4.hip): routed entries sorted by expert in LDS,
// work items, the row resource and the sum over a K split.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / MOE_WAVE;

struct DecodeSmem {
    int ids[kMaxDecodeRows];       // expert of entry q = t*k + j (-1 when invalid)
    int cnt[256];                  // routed rows per expert
    int pfx[257];                  // entries of expert e: ent[pfx[e] .. pfx[e+1])
    int slot_expert[256];          // i-th active expert (ascending id)
    int ent[kMaxDecodeRows];       // entries grouped by expert (ascending id), ascending
    int wsum[kWaves];
    int wact[kWaves];
    int n_active;
};

// Counts, active experts, the entries sorted by expert, and routing flags, from ids;
// every workgroup of a launch runs it (block 0 reports the flags).  Threads 0 .. 255 do
// the work; a larger workgroup's other threads only take part in its barriers.
__device__ void decode_setup(DecodeSmem& sm, const int32_t* __restrict__ ids, int T, int k, int E,
                             int32_t* status, bool report) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const bool worker = tid < 256;
    const int R = T * k;
    if (worker) sm.cnt[tid] = 0;
    __syncthreads();
    int my_e = -1;
    if (worker && tid < R) {
        const int e = ids[tid];
        const bool ok = (unsigned)e < (unsigned)E;
        my_e = ok ? e : -1;
        if (ok) atomicAdd(&sm.cnt[e], 1);
        if (report) {
            int bad = ok ? 0 : kDevIdOutOfRange;
            const int t = tid / k, j = tid - t * k;
            for (int jj = 0; jj < j; ++jj)
                if (ok && ids[t * k + jj] == e) bad |= kDevIdDuplicate;
            if (bad) atomicOr(status, bad);
        }
    }
    if (worker && tid < R) sm.ids[tid] = my_e;
    __syncthreads();
    // active experts in ascending id (ballot ranks) and the exclusive prefix of the
    // counts over the expert ids (wave scans plus the wave totals)
    int c = 0, incl = 0;
    bool active = false;
    uint64_t b = 0;
    if (worker) {
        c = sm.cnt[tid];
        active = tid < E && c > 0;
        b = __ballot(active);
        incl = c;
        for (int off = 1; off < MOE_WAVE; off <<= 1) {
            const int v = __shfl_up(incl, off, MOE_WAVE);
            if (lane >= off) incl += v;
        }
        if (lane == MOE_WAVE - 1) sm.wsum[wave] = incl;
        if (lane == 0) sm.wact[wave] = __popcll(b);
    }
    __syncthreads();
    if (worker) {
        int pre = 0, pre_act = 0;
        for (int w = 0; w < wave; ++w) { pre += sm.wsum[w]; pre_act += sm.wact[w]; }
        if (active) sm.slot_expert[pre_act + __popcll(b & lanemask_lt())] = tid;
        sm.pfx[tid] = pre + incl - c;
        if (tid == 255) sm.pfx[256] = pre + incl;
        if (tid == 0) {
            int nact = 0;
            for (int w = 0; w < 4; ++w) nact += sm.wact[w];
            sm.n_active = nact;
        }
    }
    __syncthreads();
    // entry q goes after the entries q' < q of its expert
    if (my_e >= 0) {
        int rank = 0;
        for (int q = 0; q < tid; ++q) rank += sm.ids[q] == my_e;
        sm.ent[sm.pfx[my_e] + rank] = tid;
    }
    __syncthreads();
}

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

// One token: the k expert ids into sm.slot_expert (the slots are the entries), so that
// an item reads its expert from LDS and not from global memory, whose wait would also
// wait for the previous item's stores.
__device__ __forceinline__ void one_token_slots(DecodeSmem& sm, const DecodeArgs& g) {
    if ((int)threadIdx.x < g.k) sm.slot_expert[threadIdx.x] = g.ids[threadIdx.x];
    __syncthreads();
}

// The expert, routed-row count and first entry of active slot `slot`; false when the
// slot's expert id is invalid (one-token path: the slot is the entry itself).  The values
// are uniform over the wave (the workgroup, with a K split), and kept in scalar registers.
__device__ __forceinline__ bool slot_info(const DecodeArgs& g, const DecodeSmem& sm, bool one, int slot,
                                          int& e, int& M, int& e0) {
    if (one) {
        e = __builtin_amdgcn_readfirstlane(sm.slot_expert[slot]);
        M = 1;
        e0 = slot;
        return (unsigned)e < (unsigned)g.E;
    }
    e = __builtin_amdgcn_readfirstlane(sm.slot_expert[slot]);
    e0 = __builtin_amdgcn_readfirstlane(sm.pfx[e]);
    M = __builtin_amdgcn_readfirstlane(sm.pfx[e + 1]) - e0;
    return true;
}

// Walks this wave's items (kSplit: this workgroup's): its global wave (workgroup) id,
// then every (number of waves (workgroups))-th item after it.  For each item,
// f(slot, block).  (A shared work counter would balance better, but one atomic per
// item on one address serialises: thousands per launch.)
template <bool kSplit, class F>
__device__ __forceinline__ void for_items(int items, int nblk, F f) {
    const int nw = kSplit ? (int)gridDim.x : (int)gridDim.x * kWaves;
    const int first = kSplit ? (int)blockIdx.x
                             : (int)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    items = __builtin_amdgcn_readfirstlane(items);
    for (int item = first; item < items; item += nw) {
        const int slot = item / nblk;
        f(slot, item - slot * nblk);
    }
}

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
