// norm.hip -- the norms before and after the routed expert layer with its gate and residual,
// forward and backward, on gfx950.
//
//   n = y                                  or  y q w_post,  q = 1 / sqrt(mean_c y^2 + eps)
//   z = x + alpha gate n                   (gate: 1, one a channel or one a token)
//   h = z r w_pre,                         r = 1 / sqrt(mean_c z^2 + eps), z as stored
// one pass over the rows: x and y are read once, z and h written once.  Backward, from the
// gradients dz (of z by way of the stream) and dh:
//   G  = dz + r (w_pre dh) - z r^3 mean_c(w_pre dh z),         dx = G
//   dn = alpha gate G,     dgate = sum (over tokens or channels) alpha G n
//   dy = q (w_post dn) - y q^3 mean_c(w_post dn y)             (dn itself without w_post)
//   dw_pre = sum_t dh z r,  dw_post = sum_t dn y q
// G is not rounded between the two norms.  r and q are computed again from z and y, which the
// backward reads anyway: their sums ride along in the first of a row's two reductions.
//
// A row belongs to kW waves, each lane with kC pieces of 8 channels (16 bytes of BF16), so
// that it stays in registers between the reductions; kW is the fewest waves that hold d.  The
// vectors over channels are loaded once per workgroup, which walks several rows.  Memory
// bound: the least traffic is 4 (forward) and 6 (backward) passes over [T, d]; 8192 x 2048 in
// BF16, post norm, gate and pre norm: forward 23.6 us (5.7 TB/s), backward 37.7 us (5.3 TB/s)
// and 4.8 us for the column sums' second stage.  Stores past the caches gain the forward 2 us
// here, cost it 4 us of 36 at 4099 x 4096 with an FP32 stream, and slow whoever reads h next.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

struct Vec8 { float v[8]; };

__device__ __forceinline__ Vec8 ld8(const uint16_t* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    return {{bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y), bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w)}};
}
__device__ __forceinline__ Vec8 ld8(const float* p) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
    return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
// rounds to the stored type and returns the stored values
__device__ __forceinline__ Vec8 st8(uint16_t* p, const Vec8& x) {
    const uint4 u = make_uint4(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]), pack_bf16(x.v[4], x.v[5]),
                               pack_bf16(x.v[6], x.v[7]));
    *reinterpret_cast<uint4*>(p) = u;
    return {{bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y), bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w)}};
}
__device__ __forceinline__ Vec8 st8(float* p, const Vec8& x) {
    const f32x4_t a = {x.v[0], x.v[1], x.v[2], x.v[3]}, b = {x.v[4], x.v[5], x.v[6], x.v[7]};
    *reinterpret_cast<f32x4_t*>(p) = a;
    *reinterpret_cast<f32x4_t*>(p + 4) = b;
    return x;
}
__device__ __forceinline__ Vec8 ld8_or(const float* p, int c, bool in, float other) {
    if (p && in) return ld8(p + c);
    return {{other, other, other, other, other, other, other, other}};
}
__device__ __forceinline__ Vec8 zero8() { return {{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}}; }

// 8 channels as they lie in memory.  A row's pieces are all loaded, from a place that exists
// whatever the lane, before the first is unpacked: an unpacked load on one side of a branch
// would be waited for there, one piece after the other.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
    uint4 u = {0, 0, 0, 0};
    __device__ __forceinline__ void load(const uint16_t* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void keep(bool in) { u = {in ? u.x : 0, in ? u.y : 0, in ? u.z : 0, in ? u.w : 0}; }
    __device__ __forceinline__ Vec8 get() const {
        return {{bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y), bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w)}};
    }
};
template <> struct Raw8<float> {
    f32x4_t a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4_t*>(p);
        b = *reinterpret_cast<const f32x4_t*>(p + 4);
    }
    __device__ __forceinline__ void keep(bool in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = in ? a[i] : 0.0f;
            b[i] = in ? b[i] : 0.0f;
        }
    }
    __device__ __forceinline__ Vec8 get() const { return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}}; }
};

// v plus its value kBy lanes further in the row of 16
template <int kBy> __device__ __forceinline__ float plus_rotated(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + kBy, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = plus_rotated<1>(plus_rotated<2>(plus_rotated<4>(plus_rotated<8>(v))));
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// kN sums over the kW waves of a row: every lane takes the sum of one wave, and rotations by
// kW / 2, .., 1 add them in the same order in all lanes.  One barrier: `red` has two halves used
// in turn, and a half is written again only after the barrier of the reduction in between.
template <int kN, int kW, int kGroups>
__device__ __forceinline__ void row_sums(float (&v)[kN], float (*red)[kGroups][kW][kN], int& half) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = wave_sum(v[i]);
    if constexpr (kW > 1) {
        const int w = (threadIdx.x >> 6) % kW, grp = (threadIdx.x >> 6) / kW;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < kN; ++i) red[half][grp][w][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            v[i] = red[half][grp][threadIdx.x % kW][i];
            if constexpr (kW >= 16) v[i] = plus_rotated<8>(v[i]);
            if constexpr (kW >= 8) v[i] = plus_rotated<4>(v[i]);
            if constexpr (kW >= 4) v[i] = plus_rotated<2>(v[i]);
            v[i] = plus_rotated<1>(v[i]);
        }
        half ^= 1;
    }
}

constexpr int kFwdThreads = 256;
template <typename TRes, int kW, int kC>
__global__ __launch_bounds__(64 * kW > kFwdThreads ? 64 * kW : kFwdThreads) void norm_kernel(NormArgs g) {
    constexpr int kThr = 64 * kW > kFwdThreads ? 64 * kW : kFwdThreads;
    constexpr int kGroups = kThr / (64 * kW);
    __shared__ float red[2][kGroups][kW][1];
    int half = 0;
    const int grp = threadIdx.x / (64 * kW), lt = threadIdx.x % (64 * kW);
    const int d = g.d;
    const float inv_d = 1.0f / (float)d;
    const TRes* x = static_cast<const TRes*>(g.x);
    TRes* z = static_cast<TRes*>(g.z);
    Vec8 wa[kC], wp[kC];                               // alpha gate w_post, w_pre
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int col = 8 * (lt + c * 64 * kW);
        const bool in = col < d;
        wa[c] = ld8_or(g.w_post, col, in, 1.0f);
        const Vec8 gt = ld8_or(g.gate_kind == kGateChannel ? g.gate : nullptr, col, in, 1.0f);
        wp[c] = ld8_or(g.w_pre, col, in, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) wa[c].v[i] *= g.alpha * gt.v[i];
    }
    for (int64_t t0 = (int64_t)blockIdx.x * kGroups; t0 < g.T; t0 += (int64_t)gridDim.x * kGroups) {
        const int64_t t = t0 + grp;
        const bool row = t < g.T;                       // groups past T only take part in barriers
        Vec8 xv[kC], yv[kC];
        float ss[1] = {0.0f};
        Raw8<TRes> rx[kC];
        Raw8<uint16_t> ry[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int col = 8 * (lt + c * 64 * kW);
            const int64_t at = row && col < d ? t * d + col : 0;
            rx[c].load(x + at);
            if (g.y) ry[c].load(g.y + at);
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const bool in = row && 8 * (lt + c * 64 * kW) < d;
            rx[c].keep(in);
            ry[c].keep(in);
            xv[c] = rx[c].get();
            yv[c] = ry[c].get();
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] += yv[c].v[i] * yv[c].v[i];
        }
        float f = 1.0f;
        if (g.w_post) {
            row_sums<1, kW, kGroups>(ss, red, half);
            f = __builtin_amdgcn_rsqf(ss[0] * inv_d + g.eps);
        }
        if (g.gate_kind == kGateToken && row) f *= g.gate[t];
        float sz[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int col = 8 * (lt + c * 64 * kW);
            if (g.y) {
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[c].v[i] += yv[c].v[i] * f * wa[c].v[i];
                if (row && col < d) xv[c] = st8(z + t * d + col, xv[c]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sz[0] += xv[c].v[i] * xv[c].v[i];
        }
        if (g.w_pre) {
            row_sums<1, kW, kGroups>(sz, red, half);
            const float r = __builtin_amdgcn_rsqf(sz[0] * inv_d + g.eps);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int col = 8 * (lt + c * 64 * kW);
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[c].v[i] *= r * wp[c].v[i];
                if (row && col < d) st8(g.h + t * d + col, xv[c]);
            }
        }
    }
}

// the parameters' gradients of column c from its sum: a_pre (which 0) or a_out (1) of
// norm_grad_kernel
__device__ __forceinline__ void finish_column(const NormGradArgs& g, int which, int c, float sum) {
    if (which == 0) {
        g.dw_pre[c] = sum;
        return;
    }
    const bool channel = g.gate_kind == kGateChannel;
    if (g.w_post) g.dw_post[c] = channel ? g.gate[c] * sum : sum;
    if (channel) g.dgate[c] = g.w_post ? g.w_post[c] * sum : sum;
}
// the same of columns c .. c + 7
__device__ __forceinline__ void finish_columns(const NormGradArgs& g, int which, int c, const Vec8& sum) {
    if (which == 0) {
        st8(g.dw_pre + c, sum);
        return;
    }
    const bool channel = g.gate_kind == kGateChannel;
    Vec8 w = ld8_or(g.w_post, c, true, 1.0f), gt = ld8_or(channel ? g.gate : nullptr, c, true, 1.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w.v[i] *= sum.v[i];
        gt.v[i] *= sum.v[i];
    }
    if (g.w_post) st8(g.dw_post + c, gt);
    if (channel) st8(g.dgate + c, w);
}

// Workgroups of 512 threads, two a CU, so that one loads while the other waits at a barrier.  What
// stays of a row from its first reduction on stays packed (8 registers for h and y instead of 16),
// and only one sum is left for the second (dgate_t and the mean of w_post dn y differ by a
// factor), so that the next row's loads fit besides the second workgroup: 8192 x 2048 in BF16
// 37.7 us (39.0 without them; one workgroup of 1024 threads 37.1), 4099 x 4096 with an FP32 stream
// 56.6 us (57.4; 58.4), 5.6 and 5.6 TB/s of what they move, the partial sums of 8 and 17 MB among it.
// One rule for both: what 1024 threads gain at the first they lose at the second.  Past d = 8192 a lane
// holds 16 channels, for which 128 registers are too few (19 spilled, 47 with an FP32 stream):
// 2048 x 16384 takes 118 and 180 us, 3.4 TB/s.
constexpr int kBwdThreads = 512;
template <int kW> constexpr int bwd_threads() { return 64 * kW > kBwdThreads ? 64 * kW : kBwdThreads; }
template <typename TRes, int kW, int kC>
__global__ __launch_bounds__(bwd_threads<kW>(), 4) void norm_grad_kernel(NormGradArgs g) {
    constexpr int kThr = bwd_threads<kW>(), kGroups = kThr / (64 * kW), kCols = 512 * kW;
    __shared__ float red1[2][kGroups][kW][3];
    __shared__ float red2[2][kGroups][kW][1];
    __shared__ __attribute__((aligned(16))) float cols[kGroups > 1 ? kThr * 8 : 4];
    int half1 = 0, half2 = 0;
    const int grp = threadIdx.x / (64 * kW), lt = threadIdx.x % (64 * kW);
    const int d = g.d;
    const float inv_d = 1.0f / (float)d;
    const TRes* dz = static_cast<const TRes*>(g.dz);
    const TRes* z = static_cast<const TRes*>(g.z);
    TRes* dx = static_cast<TRes*>(g.dx);
    const bool pre = g.w_pre != nullptr, post = g.w_post != nullptr;
    // a_pre: sum_t dh z r;  a_out: sum_t alpha gate_t G y q (gate_t: of a gate per token, else 1),
    // from which a gate per channel and w_post give dw_post = gate a_out, dgate = w_post a_out
    Vec8 wg[kC], wp[kC], a_pre[kC], a_out[kC];          // wg: w_post times the gate per channel
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const int col = 8 * (lt + c * 64 * kW);
        const bool in = col < d;
        wg[c] = ld8_or(g.w_post, col, in, 1.0f);
        const Vec8 gt = ld8_or(g.gate_kind == kGateChannel ? g.gate : nullptr, col, in, 1.0f);
        wp[c] = ld8_or(g.w_pre, col, in, 0.0f);
        a_pre[c] = a_out[c] = zero8();
#pragma unroll
        for (int i = 0; i < 8; ++i) wg[c].v[i] *= gt.v[i];
    }
    const int64_t step = (int64_t)gridDim.x * kGroups;
    struct Row {
        Raw8<TRes> dz[kC], z[kC];
        Raw8<uint16_t> h[kC], y[kC];
    };
    auto load = [&](Row& w, int64_t t) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int col = 8 * (lt + c * 64 * kW);
            const int64_t at = t < g.T && col < d ? t * d + col : 0;
            if (dz) w.dz[c].load(dz + at);
            if (pre) {
                w.z[c].load(z + at);
                w.h[c].load(g.dh + at);
            }
            if (g.y) w.y[c].load(g.y + at);
        }
    };
    // the next row's loads are out while this one's sums and stores run, where its 16 to 24
    // registers are there
    constexpr bool kAhead = kC == 1;
    Row next;
    if constexpr (kAhead) load(next, (int64_t)blockIdx.x * kGroups + grp);
    for (int64_t t0 = (int64_t)blockIdx.x * kGroups; t0 < g.T; t0 += step) {
        const int64_t t = t0 + grp;
        const bool row = t < g.T;
        Row w;
        if constexpr (kAhead) w = next;
        else load(w, t);
        float s[3] = {0.0f, 0.0f, 0.0f};               // sums of z^2, w_pre dh z, y^2
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const bool in = row && 8 * (lt + c * 64 * kW) < d;
            w.dz[c].keep(in); w.z[c].keep(in); w.h[c].keep(in); w.y[c].keep(in);
            const Vec8 zv = w.z[c].get(), hv = w.h[c].get(), yv = w.y[c].get();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[0] += zv.v[i] * zv.v[i];
                s[1] += hv.v[i] * wp[c].v[i] * zv.v[i];
                s[2] += yv.v[i] * yv.v[i];
            }
        }
        if constexpr (kAhead) load(next, t + step);
        row_sums<3, kW, kGroups>(s, red1, half1);
        const float r = __builtin_amdgcn_rsqf(s[0] * inv_d + g.eps);
        const float q = post ? __builtin_amdgcn_rsqf(s[2] * inv_d + g.eps) : 1.0f;
        const float rz = r * (s[1] * inv_d) * r * r;   // in this order a row of zeros gives 0
        const float tg = g.alpha * (g.gate_kind == kGateToken && row ? g.gate[t] : 1.0f);
        const float tq = tg * q;
        float u[1] = {0.0f};                           // sum of w_post gate_c G y
        Vec8 G[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int col = 8 * (lt + c * 64 * kW);
            G[c] = w.dz[c].get();
            if (pre) {
                const Vec8 zv = w.z[c].get(), hv = w.h[c].get();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float hr = hv.v[i] * r;
                    a_pre[c].v[i] += hr * zv.v[i];
                    G[c].v[i] += wp[c].v[i] * hr - zv.v[i] * rz;
                }
            }
            if (row && col < d) st8(dx + t * d + col, G[c]);
            const Vec8 yv = w.y[c].get();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a_out[c].v[i] += G[c].v[i] * tq * yv.v[i];
                G[c].v[i] *= wg[c].v[i];
                u[0] += G[c].v[i] * yv.v[i];
            }
        }
        if (!g.y) continue;
        if (post || g.gate_kind == kGateToken) row_sums<1, kW, kGroups>(u, red2, half2);
        const float qy = post ? q * (tg * u[0] * inv_d) * q * q : 0.0f;
        if (g.gate_kind == kGateToken && row && lt == 0) g.dgate[t] = g.alpha * q * u[0];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            const int col = 8 * (lt + c * 64 * kW);
            const Vec8 yv = w.y[c].get();
#pragma unroll
            for (int i = 0; i < 8; ++i) G[c].v[i] = tq * G[c].v[i] - yv.v[i] * qy;
            if (row && col < d) st8(g.dy + t * d + col, G[c]);
        }
    }
    // column sums: the workgroup's row groups in order, then one partial row (with one workgroup
    // the sums themselves)
    const bool last = gridDim.x == 1;
    auto column = [&](const Vec8 (&a)[kC], int which) {
        float* dst = g.part + ((size_t)blockIdx.x * 2 + which) * d;
        if constexpr (kGroups > 1) {
            __syncthreads();
            st8(cols + threadIdx.x * 8, a[0]);
            __syncthreads();
            for (int c = threadIdx.x; c < kCols; c += kThr) {
                float v = cols[c];
#pragma unroll
                for (int u = 1; u < kGroups; ++u) v += cols[u * kCols + c];
                if (c >= d) continue;
                if (last) finish_column(g, which, c, v);
                else dst[c] = v;
            }
        } else {
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const int col = 8 * (lt + c * 64 * kW);
                if (col >= d) continue;
                if (last) finish_columns(g, which, col, a[c]);
                else st8(dst + col, a[c]);
            }
        }
    };
    static_assert(kGroups == 1 || kC == 1, "one piece per lane when a workgroup holds several rows");
    if (pre) column(a_pre, 0);
    if (g.y && (post || g.gate_kind == kGateChannel)) column(a_out, 1);
}

// The column sums over the workgroups' partial rows, in workgroup order within each of 64 slices
// and then over the slices: 64 columns per workgroup, four a thread.
constexpr int kSliceCols = 64, kSlices = 64;
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormGradArgs g, int blocks) {
    __shared__ f32x4_t p[kSlices][kSliceCols / 4];
    const int q = threadIdx.x % (kSliceCols / 4), slice = threadIdx.x / (kSliceCols / 4);
    const int which = blockIdx.y, c = blockIdx.x * kSliceCols + 4 * q;
    if (which == 1 ? !g.y || !(g.w_post || g.gate_kind == kGateChannel) : !g.w_pre) return;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (c < g.d)
#pragma unroll 4
        for (int b = slice; b < blocks; b += kSlices)
            v += *reinterpret_cast<const f32x4_t*>(g.part + ((size_t)b * 2 + which) * g.d + c);
    p[slice][q] = v;
    __syncthreads();
    const int col = blockIdx.x * kSliceCols + threadIdx.x;
    if (threadIdx.x >= kSliceCols || col >= g.d) return;
    float s = 0.0f;
    for (int u = 0; u < kSlices; ++u) s += reinterpret_cast<const float*>(&p[u][threadIdx.x >> 2])[threadIdx.x & 3];
    finish_column(g, which, col, s);
}

template <typename TRes, int kW, int kC>
void launch_norm_t(const NormArgs& g, int num_cu, hipStream_t s) {
    constexpr int thr = 64 * kW > kFwdThreads ? 64 * kW : kFwdThreads;
    const int groups = thr / (64 * kW);
    const int64_t rows = ((int64_t)g.T + groups - 1) / groups;
    // Half of the waves that fit a CU, with more rows each, but two workgroups: 8192 x 2048 in BF16
    // 23.6 us against 25.3 with all waves (28.3 with four times as many), 16384 x 4096 97 against
    // 103; 2048 x 7168, of 1024 threads a workgroup, 20.4 with two workgroups, 23.1 with one.
    const int64_t cap = (int64_t)num_cu * (1024 / thr > 2 ? 1024 / thr : 2);
    const int grid = (int)(rows < cap ? rows : cap);
    hipLaunchKernelGGL((norm_kernel<TRes, kW, kC>), dim3(grid), dim3(thr), 0, s, g);
}
template <typename TRes, int kW, int kC>
int launch_norm_grad_t(const NormGradArgs& g, hipStream_t s) {
    constexpr int thr = bwd_threads<kW>(), groups = thr / (64 * kW);
    const int64_t rows = ((int64_t)g.T + groups - 1) / groups;
    // two passes of one workgroup cost no more than the second launch that several need (33 rows
    // of 256 in two launches 5.9 us in a graph, 32 rows in four passes 7.3) and spare the host it
    constexpr int cap = kNormBlocks * kBwdThreads / thr;
    const int grid = (int)(rows <= 2 ? 1 : rows < cap ? rows : cap);
    hipLaunchKernelGGL((norm_grad_kernel<TRes, kW, kC>), dim3(grid), dim3(thr), 0, s, g);
    return grid;
}
template <typename TRes> void launch_norm_d(const NormArgs& g, int num_cu, hipStream_t s) {
    if (g.d <= 512) launch_norm_t<TRes, 1, 1>(g, num_cu, s);
    else if (g.d <= 1024) launch_norm_t<TRes, 2, 1>(g, num_cu, s);
    else if (g.d <= 2048) launch_norm_t<TRes, 4, 1>(g, num_cu, s);
    else if (g.d <= 4096) launch_norm_t<TRes, 8, 1>(g, num_cu, s);
    else if (g.d <= 8192) launch_norm_t<TRes, 16, 1>(g, num_cu, s);
    else launch_norm_t<TRes, 16, 2>(g, num_cu, s);
}
template <typename TRes> int launch_norm_grad_d(const NormGradArgs& g, hipStream_t s) {
    if (g.d <= 512) return launch_norm_grad_t<TRes, 1, 1>(g, s);
    if (g.d <= 1024) return launch_norm_grad_t<TRes, 2, 1>(g, s);
    if (g.d <= 2048) return launch_norm_grad_t<TRes, 4, 1>(g, s);
    if (g.d <= 4096) return launch_norm_grad_t<TRes, 8, 1>(g, s);
    if (g.d <= 8192) return launch_norm_grad_t<TRes, 16, 1>(g, s);
    return launch_norm_grad_t<TRes, 16, 2>(g, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& g, bool f32, int num_cu, hipStream_t s) {
    if (g.T == 0) return hipSuccess;
    if (g.d % 8 != 0 || g.d > kNormMaxD) return hipErrorInvalidValue;
    if (f32) launch_norm_d<float>(g, num_cu, s);
    else launch_norm_d<uint16_t>(g, num_cu, s);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs& g, bool f32, hipStream_t s) {
    if (g.d % 8 != 0 || g.d > kNormMaxD) return hipErrorInvalidValue;
    const int blocks = f32 ? launch_norm_grad_d<float>(g, s) : launch_norm_grad_d<uint16_t>(g, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || blocks == 1 || !(g.w_pre || g.w_post || g.gate_kind == kGateChannel)) return e;
    const dim3 grid((g.d + kSliceCols - 1) / kSliceCols, 2);
    hipLaunchKernelGGL(norm_columns_kernel, grid, dim3(1024), 0, s, g, blocks);
    return hipGetLastError();
}

}  // namespace moe
