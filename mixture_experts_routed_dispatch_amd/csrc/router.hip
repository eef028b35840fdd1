// router.hip -- the router in front of the routed expert layer, on gfx950: logits -> expert
// ids, scores, per-expert counts, probability sums and the balance loss, and the gradient.
//
// With z = logits[t], s = softmax(z) or sigmoid(z), p_e = s_e / sum_e' s_e' (softmax: p = s):
//   ids      the k experts of the largest key, descending, ties to the lowest index; the key
//            is z_e itself, or s_e + bias_e when a selection bias is given
//   scores   scale s_j, divided by the sum of the chosen s with `normalize`
//   counts_e tokens that chose e;  P_e = sum_t p_te  (rows that the mask leaves out count
//            nowhere; N = sum counts / k rows remain)
//   loss     coef E / (k N^2) sum_e counts_e P_e
// Gradient, with r_j the derivative by way of the scores (v_j = s_j / sum of the chosen s,
// g_j = scale dscores_j):  normalize: ds_j = (g_j - sum_i g_i v_i) / sum_i s_i, else ds_j = g_j,
// and b_e = dloss coef E counts_e / (k N^2) by way of P:
//   softmax  dz_e = p_e (b_e - D) + [e chosen] p_e ds_e,   D = sum_e p_e b_e + sum_j p_j ds_j
//   sigmoid  dz_e = ((b_e - sum p b) / sum s + [e chosen] ds_e) s_e (1 - s_e)
//
// A row of E <= 256 logits is held by 16 lanes (kV = 4, 8 or 16 consecutive logits each), so
// that a wave works on four rows and every reduction over a row stays within 16 lanes, where
// DPP rotations do it without LDS.  The k largest are taken one at a time: each lane's
// maximum, the row's maximum, the lowest lane that has it, and there the first of its
// logits.  Keys are compared as unsigned integers that order like the floats (NaN below
// everything, -0 as +0), so that ties and infinities need no case of their own.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 16;         // rows in flight per workgroup
constexpr int kWide = 1024;                  // threads of the workgroups of large batches

template <int kCtrl> __device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
// over the 16 lanes of a row: rotations by 8, 4, 2, 1; every lane gets the same bits
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
    uint32_t o;
    o = dpp<0x128>(v); v = v > o ? v : o;
    o = dpp<0x124>(v); v = v > o ? v : o;
    o = dpp<0x122>(v); v = v > o ? v : o;
    o = dpp<0x121>(v); v = v > o ? v : o;
    return v;
}
__device__ __forceinline__ float row_max(float v) {
    v = __builtin_fmaxf(v, __uint_as_float(dpp<0x128>(__float_as_uint(v))));
    v = __builtin_fmaxf(v, __uint_as_float(dpp<0x124>(__float_as_uint(v))));
    v = __builtin_fmaxf(v, __uint_as_float(dpp<0x122>(__float_as_uint(v))));
    return __builtin_fmaxf(v, __uint_as_float(dpp<0x121>(__float_as_uint(v))));
}
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(dpp<0x128>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x124>(__float_as_uint(v)));
    v += __uint_as_float(dpp<0x122>(__float_as_uint(v)));
    return v + __uint_as_float(dpp<0x121>(__float_as_uint(v)));
}

// unsigned key that orders like the float: NaN 1, then -inf .. +inf; 0 stays free for
// logits that are taken or past E
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return f != f ? 1u : u;
}
__device__ __forceinline__ float key_value(uint32_t u) {
    return __uint_as_float(u ^ ((u & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t order_key64(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f + 0.0);
    const uint64_t u = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
    return f != f ? 1ull : u;
}

// e^x with the hardware exp2 (about 1 ulp, plus |x| 2^-24 from the argument)
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(1.4426950408889634f * x); }
// sigmoid(z) and 1 - sigmoid(z), neither by a cancelling difference
__device__ __forceinline__ void sigmoid2(float z, float& s, float& c) {
    const float e = exp_f(-__builtin_fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    s = z >= 0.0f ? r : er;
    c = z >= 0.0f ? er : r;
    if (z != z) s = c = z;
}

__device__ __forceinline__ float ld_logit(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// kV logits from index i0 of the row at element offset `row`; -inf past E.  vec: rows start
// on, and E is a multiple of, the widest piece used here (16 bytes, 8 for kV = 4 in BF16).
template <int kV, bool kF32>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int i0, int E, bool vec, float z[kV]) {
    if (vec) {
        if constexpr (kF32) {
#pragma unroll
            for (int c = 0; c < kV; c += 4) {
                f32x4_t v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (i0 + c < E) v = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + row + i0 + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[c + i] = v[i];
            }
        } else if constexpr (kV == 4) {
            uint2 v = make_uint2(0xFF80FF80u, 0xFF80FF80u);
            if (i0 < E) v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + row + i0);
            z[0] = bf16lo(v.x); z[1] = bf16hi(v.x); z[2] = bf16lo(v.y); z[3] = bf16hi(v.y);
        } else {
#pragma unroll
            for (int c = 0; c < kV; c += 8) {
                uint4 v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
                if (i0 + c < E) v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + row + i0 + c);
                z[c] = bf16lo(v.x); z[c + 1] = bf16hi(v.x); z[c + 2] = bf16lo(v.y); z[c + 3] = bf16hi(v.y);
                z[c + 4] = bf16lo(v.z); z[c + 5] = bf16hi(v.z); z[c + 6] = bf16lo(v.w); z[c + 7] = bf16hi(v.w);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) z[i] = i0 + i < E ? ld_logit(p, row + i0 + i, kF32) : -INFINITY;
    }
}

template <int kV, bool kF32>
__device__ __forceinline__ void store_row(void* p, int64_t row, int i0, int E, bool vec, const float z[kV]) {
    if (vec) {
        if constexpr (kF32) {
#pragma unroll
            for (int c = 0; c < kV; c += 4)
                if (i0 + c < E) {
                    const f32x4_t v = {z[c], z[c + 1], z[c + 2], z[c + 3]};
                    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + row + i0 + c) = v;
                }
        } else if constexpr (kV == 4) {
            if (i0 < E)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + row + i0) =
                    make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
        } else {
#pragma unroll
            for (int c = 0; c < kV; c += 8)
                if (i0 + c < E)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + row + i0 + c) =
                        make_uint4(pack_bf16(z[c], z[c + 1]), pack_bf16(z[c + 2], z[c + 3]),
                                   pack_bf16(z[c + 4], z[c + 5]), pack_bf16(z[c + 6], z[c + 7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i0 + i < E) {
                if constexpr (kF32) static_cast<float*>(p)[row + i0 + i] = z[i];
                else static_cast<uint16_t*>(p)[row + i0 + i] = (uint16_t)f32_to_bf16(z[i]);
            }
    }
}

// Scores of a row: s (softmax: p), and the factor that makes them probabilities (softmax: 1).
// A row of -inf alone gives zeros; a NaN or +inf logit gives NaN as the formula does.
// zmax is the row's maximum and inv the reciprocal of its sum of e^(z - zmax).
template <int kV, bool kSig>
__device__ __forceinline__ void row_scores(const float z[kV], float s[kV], float& zmax, float& inv) {
    if constexpr (kSig) {
        float sum = 0.0f;
        zmax = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float c;
            sigmoid2(z[i], s[i], c);
            sum += s[i];
        }
        sum = row_sum(sum);
        inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    } else {
        float m = z[0];
#pragma unroll
        for (int i = 1; i < kV; ++i) m = __builtin_fmaxf(m, z[i]);
        zmax = row_max(m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            s[i] = zmax == -INFINITY && z[i] == z[i] ? 0.0f : exp_f(z[i] - zmax);
            sum += s[i];
        }
        sum = row_sum(sum);
        inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int i = 0; i < kV; ++i) s[i] *= inv;
    }
}
// the score of one logit of that row, the same bits as row_scores gives it
template <bool kSig> __device__ __forceinline__ float one_score(float z, float zmax, float inv) {
    if constexpr (kSig) {
        float s, c;
        sigmoid2(z, s, c);
        return s;
    } else {
        return (zmax == -INFINITY && z == z ? 0.0f : exp_f(z - zmax)) * inv;
    }
}

// the k largest of the row's keys, one a round; sel[0 .. k) gets their indices.  Taken keys
// become 0.  Returns the last one's key.
template <int kV>
__device__ __forceinline__ uint32_t take_top(uint32_t key[kV], int k, int i0, int* sel) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, grp = lane >> 4;
    uint32_t m = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t mine = key[0];
#pragma unroll
        for (int i = 1; i < kV; ++i) mine = mine > key[i] ? mine : key[i];
        m = row_max_u32(mine);
        const uint64_t b = __ballot(mine == m);
        const uint32_t half = grp & 2 ? (uint32_t)(b >> 32) : (uint32_t)b;
        const uint32_t field = (grp & 1 ? half >> 16 : half) & 0xFFFFu;
        int li = 0;
#pragma unroll
        for (int i = kV - 1; i >= 0; --i) li = key[i] == m ? i : li;
        if (l16 == __builtin_ctz(field)) sel[j] = i0 + li;
        else li = -1;
#pragma unroll
        for (int i = 0; i < kV; ++i) key[i] = li == i ? 0u : key[i];
    }
    return m;
}
// the same in 64 bits: s + bias computed and compared in double
template <int kV, bool kSig>
__device__ __forceinline__ void take_top_exact(const float z[kV], const float bias[kV], int E, int k, int i0, float zmax,
                                            int* sel) {
    const int l16 = threadIdx.x & 15;
    double s[kV];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        if constexpr (kSig) s[i] = 1.0 / (1.0 + exp(-(double)z[i]));
        else s[i] = zmax == -INFINITY && z[i] == z[i] ? 0.0 : exp((double)z[i] - (double)zmax);
        sum += s[i];
    }
    if constexpr (!kSig) {
        for (int o = 8; o; o >>= 1) sum += __shfl_xor(sum, o, 16);
        const double d = sum == 0.0 ? 1.0 : sum;
#pragma unroll
        for (int i = 0; i < kV; ++i) s[i] /= d;
    }
    uint64_t key[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) key[i] = i0 + i < E ? order_key64(s[i] + (double)bias[i]) : 0ull;
    for (int j = 0; j < k; ++j) {
        uint64_t m = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (key[i] > m) { m = key[i]; at = i0 + i; }
        if (m == 0) at = 1 << 20;
        for (int o = 8; o; o >>= 1) {
            const uint64_t om = __shfl_xor((unsigned long long)m, o, 16);
            const int oa = __shfl_xor(at, o, 16);
            if (om > m || (om == m && oa < at)) { m = om; at = oa; }
        }
        if (l16 == 0) sel[j] = at;
#pragma unroll
        for (int i = 0; i < kV; ++i) if (i0 + i == at) key[i] = 0ull;
    }
}

// LDS writes of one wave, read by its other lanes
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// keys that FP32 rounding may have brought into a wrong order lie this close (relative to
// the larger of 1 and the key): a score is off by at most 3e-7 and the sum's rounding adds
// 6e-8 of the key, so two keys by less than 7.2e-7
constexpr float kNear = 2e-6f;

// N and sum counts_e P_e from one expert per thread, e < 256, and the loss from them
__device__ __forceinline__ void write_loss(const RouterArgs& g, int count, float psum, double (*part)[2]) {
    double a = (double)count * (double)psum, n = (double)count;
    for (int o = 32; o; o >>= 1) { a += __shfl_xor(a, o, 64); n += __shfl_xor(n, o, 64); }
    if ((threadIdx.x & 63) == 0 && threadIdx.x < 256) { part[threadIdx.x >> 6][0] = a; part[threadIdx.x >> 6][1] = n; }
    __syncthreads();
    if (threadIdx.x == 0 && g.loss) {
        a = n = 0.0;
        for (int w = 0; w < 4; ++w) { a += part[w][0]; n += part[w][1]; }
        n /= g.k;
        *g.loss = n > 0.0 ? (float)((double)g.coef * g.E / (g.k * n * n) * a) : 0.0f;
    }
}

template <int kThr, int kV, bool kF32, bool kSig, bool kBias>
__global__ __launch_bounds__(kThr) void route_kernel(RouterArgs g) {
    constexpr int kR = kThr / 16;
    __shared__ int sel[kR][kMaxTopK];
    __shared__ int cnt[256];
    __shared__ float sums[kThr / MOE_WAVE][256];
    __shared__ double part[4][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = tid & 15, row = tid >> 4;
    const int E = g.E, k = g.k, i0 = l16 * kV;
    if (tid < 256) cnt[tid] = 0;
    __syncthreads();
    float acc[kV], bias[kBias ? kV : 1];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        acc[i] = 0.0f;
        if constexpr (kBias) bias[i] = i0 + i < E ? g.bias[i0 + i] : 0.0f;
    }
    // rows past T repeat row T - 1 and write nothing (their lanes take part in every DPP step)
    for (int64_t t0 = (int64_t)blockIdx.x * kR; t0 < g.T; t0 += (int64_t)gridDim.x * kR) {
        const bool in = t0 + row < g.T;
        const int64_t t = in ? t0 + row : g.T - 1;
        const bool live = in && (!g.mask || g.mask[t]);
        float z[kV], s[kV], zmax, inv;
        load_row<kV, kF32>(g.logits, t * E, i0, E, g.vec, z);
        row_scores<kV, kSig>(z, s, zmax, inv);
        uint32_t key[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const bool here = i0 + i < E;
            if constexpr (kBias) key[i] = here ? order_key(s[i] + bias[i]) : 0u;
            else key[i] = here ? order_key(z[i]) : 0u;
            if (live && here) acc[i] += kSig ? s[i] * inv : s[i];
        }
        const uint32_t last = take_top<kV>(key, k, i0, sel[row]);
        wave_fence();
        if constexpr (kBias) {
            // is every neighbour in the order, and everything left behind the last one,
            // either further off than FP32 rounding reaches, or the same logit and bias
            // (a true tie, which the index has settled)?
            bool near = false;
            const int e_last = sel[row][k - 1];
            const float z_last = ld_logit(g.logits, t * E + e_last, kF32), b_last = g.bias[e_last];
            const float k_last = key_value(last);
            const float floor_key = k_last - kNear * __builtin_fmaxf(1.0f, __builtin_fabsf(k_last));
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (key[i] != 0u && !(key_value(key[i]) < floor_key))
                    near |= !(z[i] == z_last && bias[i] == b_last);
            for (int j = l16; j + 1 < k; j += 16) {
                const int ea = sel[row][j], eb = sel[row][j + 1];
                const float za = ld_logit(g.logits, t * E + ea, kF32), zb = ld_logit(g.logits, t * E + eb, kF32);
                const float ba = g.bias[ea], bb = g.bias[eb];
                const float ka = one_score<kSig>(za, zmax, inv) + ba, kb = one_score<kSig>(zb, zmax, inv) + bb;
                near |= !(ka - kb > kNear * __builtin_fmaxf(1.0f, __builtin_fabsf(ka))) && !(za == zb && ba == bb);
            }
            if (__ballot(near)) {
                wave_fence();
                take_top_exact<kV, kSig>(z, bias, E, k, i0, zmax, sel[row]);
                wave_fence();
            }
        }
        // lane j writes the j-th (and j + 16-th) expert of its row
        float sc[2] = {0.0f, 0.0f}, total = 0.0f;
        int id[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = l16 + 16 * h;
            id[h] = j < k ? sel[row][j] : 0;
            if (j < k) {
                sc[h] = one_score<kSig>(ld_logit(g.logits, t * E + id[h], kF32), zmax, inv);
                total += sc[h];
            }
        }
        total = row_sum(total);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = l16 + 16 * h;
            if (j < k && in) {
                float w = sc[h];
                if (g.normalize) w = total == 0.0f ? 0.0f : w / total;
                g.ids[t * k + j] = live ? id[h] : j;
                g.scores[t * k + j] = live ? w * g.scale : 0.0f;
                if (live && g.part_counts) atomicAdd(&cnt[id[h]], 1);
            }
        }
        wave_fence();                                   // sel is rewritten by the next rows
    }
    if (!g.part_counts) return;
    // the rows' probabilities added over the wave's four rows, then the workgroup's waves
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        acc[i] += __shfl_xor(acc[i], 16, 64);
        acc[i] += __shfl_xor(acc[i], 32, 64);
        if (lane < 16) sums[wave][i0 + i] = acc[i];
    }
    __syncthreads();
    int c = 0;
    float p = 0.0f;
    if (tid < E) {
        c = cnt[tid];
        for (int w = 0; w < kThr / MOE_WAVE; ++w) p += sums[w][tid];
    }
    if (gridDim.x == 1) {
        if (tid < E) {
            if (g.counts) g.counts[tid] = c;
            if (g.psum) g.psum[tid] = p;
        }
        write_loss(g, c, p, part);
    } else if (tid < g.stride) {
        g.part_counts[(size_t)blockIdx.x * g.stride + tid] = c;
        g.part_sums[(size_t)blockIdx.x * g.stride + tid] = p;
    }
}

// the workgroups' partial counts and sums, in workgroup order within 16 slices, then the slices
constexpr int kFinalThreads = 1024;
__global__ __launch_bounds__(kFinalThreads) void route_final_kernel(RouterArgs g, int blocks) {
    __shared__ f32x4_t ps[16][64];
    __shared__ int4 cs[16][64];
    __shared__ double part[4][2];
    const int tid = threadIdx.x, q = tid & 63, slice = tid >> 6;
    f32x4_t p = {0.f, 0.f, 0.f, 0.f};
    int4 c = make_int4(0, 0, 0, 0);
    if (4 * q < g.stride) {
#pragma unroll 8
        for (int b = slice; b < blocks; b += 16) {
            p += *reinterpret_cast<const f32x4_t*>(g.part_sums + (size_t)b * g.stride + 4 * q);
            const int4 v = *reinterpret_cast<const int4*>(g.part_counts + (size_t)b * g.stride + 4 * q);
            c.x += v.x; c.y += v.y; c.z += v.z; c.w += v.w;
        }
    }
    ps[slice][q] = p;
    cs[slice][q] = c;
    __syncthreads();
    float sum = 0.0f;
    int count = 0;
    if (tid < g.E) {
        for (int s = 0; s < 16; ++s) {
            sum += reinterpret_cast<const float*>(&ps[s][tid >> 2])[tid & 3];
            count += reinterpret_cast<const int*>(&cs[s][tid >> 2])[tid & 3];
        }
        if (g.counts) g.counts[tid] = count;
        if (g.psum) g.psum[tid] = sum;
    }
    write_loss(g, count, sum, part);
}

template <int kV, bool kF32, bool kSig>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouterGradArgs g) {
    __shared__ float extra[kRows][16 * kV];               // p_j ds_j (softmax), ds_j (sigmoid) of the chosen
    __shared__ double part[kThreads / MOE_WAVE];
    const int tid = threadIdx.x, l16 = tid & 15, row = tid >> 4;
    const int E = g.E, k = g.k, i0 = l16 * kV;
    // b_e of this lane's experts
    float bal[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) bal[i] = 0.0f;
    if (g.dloss) {
        double n = tid < E ? (double)g.counts[tid] : 0.0;
        for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o, 64);
        if ((tid & 63) == 0) part[tid >> 6] = n;
        __syncthreads();
        n = 0.0;
        for (int w = 0; w < kThreads / MOE_WAVE; ++w) n += part[w];
        n /= k;
        const double f = n > 0.0 ? (double)*g.dloss * g.coef * E / (k * n * n) : 0.0;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i0 + i < E) bal[i] = (float)(f * g.counts[i0 + i]);
    }
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < g.T; t0 += (int64_t)gridDim.x * kRows) {
        const bool in = t0 + row < g.T;
        const int64_t t = in ? t0 + row : g.T - 1;
        const bool live = !g.mask || g.mask[t];
        float z[kV], s[kV], zmax, inv;
        load_row<kV, kF32>(g.logits, t * E, i0, E, g.vec, z);
        int id[2];
        float gj[2], zj[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = l16 + 16 * h;
            id[h] = j < k ? g.ids[t * k + j] : -1;
            if ((unsigned)id[h] >= (unsigned)E) id[h] = -1;
            gj[h] = id[h] >= 0 && g.dscores ? g.dscores[t * k + j] * g.scale : 0.0f;
            zj[h] = id[h] >= 0 ? ld_logit(g.logits, t * E + id[h], kF32) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) extra[row][i0 + i] = 0.0f;
        row_scores<kV, kSig>(z, s, zmax, inv);
        float sj[2], total = 0.0f, dot = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sj[h] = id[h] >= 0 ? one_score<kSig>(zj[h], zmax, inv) : 0.0f;
            total += sj[h];
        }
        total = row_sum(total);
        float vj[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            vj[h] = total == 0.0f ? 0.0f : sj[h] / total;  // IEEE: exactly 1 for one expert a token
            dot += gj[h] * vj[h];
        }
        dot = row_sum(dot);
        float own = 0.0f;
        wave_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float r;
            if (g.normalize) {
                // softmax: p_j ds_j = v_j (g_j - dot), whose sum over j is zero
                r = kSig ? (total == 0.0f ? 0.0f : (gj[h] - dot) / total) : vj[h] * (gj[h] - dot);
            } else {
                r = kSig ? gj[h] : sj[h] * gj[h];
                own += kSig ? 0.0f : r;
            }
            if (id[h] >= 0) extra[row][id[h]] = r;
        }
        wave_fence();
        float pb = own;
#pragma unroll
        for (int i = 0; i < kV; ++i) pb += (kSig ? s[i] * inv : s[i]) * bal[i];
        pb = row_sum(pb);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const float x = extra[row][i0 + i];
            if constexpr (kSig) {
                float ss, c;
                sigmoid2(z[i], ss, c);
                z[i] = ((bal[i] - pb) * inv + x) * ss * c;
            } else {
                z[i] = s[i] * (bal[i] - pb) + x;
            }
            if (!live) z[i] = 0.0f;
        }
        if (in) store_row<kV, kF32>(g.dlogits, t * E, i0, E, g.vec, z);
        wave_fence();                                   // extra is rewritten by the next rows
    }
}

// Workgroups of 1024 threads once there are more rows than one pass of the smaller ones over
// the chip: the same rows in flight with a quarter of the partial sums.
bool wide_blocks(int64_t T) { return T > (int64_t)kRouterBlocks * kRows; }

// logits per lane, and whether rows are made of aligned pieces of the widest load
int per_lane(int E) { return E <= 64 ? 4 : E <= 128 ? 8 : 16; }
bool aligned_rows(const void* a, const void* b, int E, bool f32) {
    const int v = f32 ? 4 : per_lane(E) == 4 ? 4 : 8;
    const uintptr_t bytes = v * (f32 ? 4 : 2);
    return E % v == 0 && reinterpret_cast<uintptr_t>(a) % bytes == 0 && reinterpret_cast<uintptr_t>(b) % bytes == 0;
}

template <int kThr, int kV, bool kF32>
void launch_route_t(const RouterArgs& g, int grid, bool sig, hipStream_t s) {
    const dim3 gd(grid), bd(kThr);
    if (sig && g.bias) hipLaunchKernelGGL((route_kernel<kThr, kV, kF32, true, true>), gd, bd, 0, s, g);
    else if (sig) hipLaunchKernelGGL((route_kernel<kThr, kV, kF32, true, false>), gd, bd, 0, s, g);
    else if (g.bias) hipLaunchKernelGGL((route_kernel<kThr, kV, kF32, false, true>), gd, bd, 0, s, g);
    else hipLaunchKernelGGL((route_kernel<kThr, kV, kF32, false, false>), gd, bd, 0, s, g);
}
template <int kV, bool kF32>
void launch_route_v(const RouterArgs& g, int grid, bool sig, hipStream_t s) {
    if (wide_blocks(g.T)) launch_route_t<kWide, kV, kF32>(g, grid, sig, s);
    else launch_route_t<kThreads, kV, kF32>(g, grid, sig, s);
}
template <int kV>
void launch_route_grad_v(const RouterGradArgs& g, int grid, bool sig, bool f32, hipStream_t s) {
    const dim3 gd(grid), bd(kThreads);
    if (f32 && sig) hipLaunchKernelGGL((route_grad_kernel<kV, true, true>), gd, bd, 0, s, g);
    else if (f32) hipLaunchKernelGGL((route_grad_kernel<kV, true, false>), gd, bd, 0, s, g);
    else if (sig) hipLaunchKernelGGL((route_grad_kernel<kV, false, true>), gd, bd, 0, s, g);
    else hipLaunchKernelGGL((route_grad_kernel<kV, false, false>), gd, bd, 0, s, g);
}

}  // namespace

int router_blocks(int64_t T) {
    const int rows = wide_blocks(T) ? kWide / 16 : kRows;
    const int64_t b = (T + rows - 1) / rows;
    return (int)(b < 1 ? 1 : b < kRouterBlocks ? b : kRouterBlocks);
}

hipError_t launch_route(RouterArgs g, bool sigmoid, bool f32, hipStream_t s) {
    const bool stats = g.part_counts != nullptr;
    if (g.T == 0 && !stats) return hipSuccess;
    g.vec = aligned_rows(g.logits, g.logits, g.E, f32);
    g.stride = (g.E + 3) & ~3;
    const int grid = router_blocks(g.T);
    switch (per_lane(g.E) * 2 + (f32 ? 1 : 0)) {
        case 8: launch_route_v<4, false>(g, grid, sigmoid, s); break;
        case 9: launch_route_v<4, true>(g, grid, sigmoid, s); break;
        case 16: launch_route_v<8, false>(g, grid, sigmoid, s); break;
        case 17: launch_route_v<8, true>(g, grid, sigmoid, s); break;
        case 32: launch_route_v<16, false>(g, grid, sigmoid, s); break;
        default: launch_route_v<16, true>(g, grid, sigmoid, s); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !stats || grid == 1) return e;
    hipLaunchKernelGGL(route_final_kernel, dim3(1), dim3(kFinalThreads), 0, s, g, grid);
    return hipGetLastError();
}

hipError_t launch_route_grad(RouterGradArgs g, bool sigmoid, bool f32, hipStream_t s) {
    if (g.T == 0) return hipSuccess;
    g.vec = aligned_rows(g.logits, g.dlogits, g.E, f32);
    const int64_t b = ((int64_t)g.T + kRows - 1) / kRows;
    const int grid = (int)(b < 2048 ? b : 2048);
    switch (per_lane(g.E)) {
        case 4: launch_route_grad_v<4>(g, grid, sigmoid, f32, s); break;
        case 8: launch_route_grad_v<8>(g, grid, sigmoid, f32, s); break;
        default: launch_route_grad_v<16>(g, grid, sigmoid, f32, s); break;
    }
    return hipGetLastError();
}

}  // namespace moe
