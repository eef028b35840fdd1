// router.hip -- the router in front of the routed expert layer, on gfx950: logits -> expert
// ids, scores, per-expert counts, probability sums and the balance loss, and the gradient.
//
// With z = logits[t], s = softmax(z) or sigmoid(z), p_e = s_e / sum_e' s_e' (softmax: p = s):
//   ids      the k experts of the largest key, descending, ties to the lowest index; the key
//            is z_e itself, or s_e + bias_e when a selection bias is given (-inf where z_e is)
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
// A row of E <= 256 logits is held by 16 lanes (kV = 4, 8 or 16 logits each), so
// that a wave works on four rows and every reduction over a row stays within 16 lanes, where
// DPP rotations do it without LDS.
//
// The choice.  A bound that at least k keys reach and few do is the k-th largest of the 16 lanes'
// maxima for k <= 8 (of 256 random keys about 11 reach it for k = 8), or of their two largest each
// for k <= 20 (about 18 for k = 16).  Those candidates' indices go to LDS in ascending order, one or
// two to a lane, and each counts the ones before it, which is its place.  With larger k, or more than
// kCand candidates (ties, rows of one value), the row's maximum is taken k times; a bias then takes
// the last of those as the bound.  16384 x 256 in BF16 with sigmoid, bias and k = 8: 12.0 to 13.6 us
// (card to card), against 32.4 by taking the maximum 8 times; 800 vector instructions a wave issue for
// 6 us of it, the rest is the latency of one pass (its 9.5 MB take 1.9 us), in which the candidates'
// logits and then the chosen ones' are fetched again from memory.  k = 16 with the second launch
// 22.2 us, and 113 while all of k > 12 took the maxima and settled near keys for the whole row; k = 32,
// which takes the maxima, 214.
//
// With a bias the keys s + b have to be ordered as in exact arithmetic.  They are compared in
// FP32; where two that matter lie closer than FP32's error, they are computed again in 64
// bits: of the candidates only, or in the other way of all.
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

// what a key counts as in the choice: NaN as -inf
__device__ __forceinline__ float choice_key(float f) { return f != f ? -INFINITY : f; }
__device__ __forceinline__ double choice_key(double f) { return f != f ? -(double)INFINITY : f; }
// the score as it enters a biased key: a logit of -inf stays behind the others whatever its bias
template <typename T> __device__ __forceinline__ T key_score(T s, float z) { return z == -INFINITY ? -(T)INFINITY : s; }
// unsigned number that orders like the (choice) key; 0 stays free for logits that are taken
// or past E
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(choice_key(f) + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t u) {
    return __uint_as_float(u ^ ((u & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
// e^x with the hardware exp2 (about 1 ulp, plus |x| 2^-24 from the argument: what a row's sum and
// probabilities take, where e^x <= 1 makes it at most 0.4 2^-24 of the row's largest)
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(1.4426950408889634f * x); }
// the same without the argument's part, for scores, which may lie far below the maximum and are divided
// by one another: what the product loses to its rounding comes back as a factor 1 + ln 2 rest.  (For
// every e^x of a row it costs 16384 x 256 0.2 to 0.9 us, and the gradient 0.4 of 7.7.)
__device__ __forceinline__ float exp_exact_argument(float x) {
    const float t = 1.4426950408889634f * x;
    float rest = __builtin_fmaf(1.4426950408889634f, x, -t);
    rest = __builtin_fmaf(1.925962991e-8f, x, rest);              // log2 e less its 24 bits
    rest = __builtin_fabsf(t) < 256.0f ? rest : 0.0f;             // 0 or inf; no NaN from infinite x
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(0.6931471805599453f, rest, 1.0f);
}
// what a row's logits are taken relative to: its maximum, 0 for a row of -inf alone (so that its
// terms are e^-inf = 0)
__device__ __forceinline__ float base_of(float zmax) { return zmax == -INFINITY ? 0.0f : zmax; }

__device__ __forceinline__ float ld_logit(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// The logits of a lane: kV from index first(l16) on, the second 8 of 16 from the row's second half.
// So the 16 lanes' pieces follow one another, and rows of 129 to 255 fill all lanes too.
template <int kV> __device__ __forceinline__ int first(int l16) { return l16 * (kV < 8 ? kV : 8); }
// i-th of them relative to the first
__device__ __forceinline__ constexpr int ahead(int i) { return i + (i >= 8 ? 120 : 0); }

// A lane's kV logits of the row at element offset `row`; -inf past E.  vec: rows start
// on, and E is a multiple of, the widest piece used here (16 bytes, 8 for kV = 4 in BF16).
template <int kV, bool kF32>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int i0, int E, bool vec, float z[kV]) {
    if (vec) {
        if constexpr (kF32) {
#pragma unroll
            for (int c = 0; c < kV; c += 4) {
                f32x4_t v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (ahead(c) < E - i0) v = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + row + i0 + ahead(c));
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
                if (ahead(c) < E - i0) v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + row + i0 + ahead(c));
                z[c] = bf16lo(v.x); z[c + 1] = bf16hi(v.x); z[c + 2] = bf16lo(v.y); z[c + 3] = bf16hi(v.y);
                z[c + 4] = bf16lo(v.z); z[c + 5] = bf16hi(v.z); z[c + 6] = bf16lo(v.w); z[c + 7] = bf16hi(v.w);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) z[i] = ahead(i) < E - i0 ? ld_logit(p, row + i0 + ahead(i), kF32) : -INFINITY;
    }
}

template <int kV, bool kF32>
__device__ __forceinline__ void store_row(void* p, int64_t row, int i0, int E, bool vec, const float z[kV]) {
    if (vec) {
        if constexpr (kF32) {
#pragma unroll
            for (int c = 0; c < kV; c += 4)
                if (ahead(c) < E - i0) {
                    const f32x4_t v = {z[c], z[c + 1], z[c + 2], z[c + 3]};
                    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + row + i0 + ahead(c)) = v;
                }
        } else if constexpr (kV == 4) {
            if (i0 < E)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + row + i0) =
                    make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
        } else {
#pragma unroll
            for (int c = 0; c < kV; c += 8)
                if (ahead(c) < E - i0)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + row + i0 + ahead(c)) =
                        make_uint4(pack_bf16(z[c], z[c + 1]), pack_bf16(z[c + 2], z[c + 3]),
                                   pack_bf16(z[c + 4], z[c + 5]), pack_bf16(z[c + 6], z[c + 7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (ahead(i) < E - i0) {
                if constexpr (kF32) static_cast<float*>(p)[row + i0 + ahead(i)] = z[i];
                else static_cast<uint16_t*>(p)[row + i0 + ahead(i)] = (uint16_t)f32_to_bf16(z[i]);
            }
    }
}

// Scores of a row: s (softmax: p), and the factor that makes them probabilities (softmax: 1).
// A row of -inf alone gives zeros; a NaN or +inf logit gives NaN as the formula does.
// base as base_of (sigmoid: 0), inv the reciprocal of the row's sum.
template <int kV, bool kSig>
__device__ __forceinline__ void row_scores(const float z[kV], float s[kV], float& base, float& inv) {
    float sum = 0.0f;
    if constexpr (kSig) {
        base = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) sum += s[i] = sigmoid_f(z[i]);
    } else {
        float m = z[0];
#pragma unroll
        for (int i = 1; i < kV; ++i) m = __builtin_fmaxf(m, z[i]);
        base = base_of(row_max(m));
#pragma unroll
        for (int i = 0; i < kV; ++i) sum += s[i] = exp_f(z[i] - base);
    }
    sum = row_sum(sum);
    inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if constexpr (!kSig)
#pragma unroll
        for (int i = 0; i < kV; ++i) s[i] *= inv;
}
// the score of one logit of that row, with the argument of e^x in full
template <bool kSig> __device__ __forceinline__ float one_score(float z, float base, float inv) {
    if constexpr (kSig) return __builtin_amdgcn_rcpf(1.0f + exp_exact_argument(-z));
    else return exp_exact_argument(z - base) * inv;
}

// the k largest of the row's keys, one a round; sel[0 .. k) gets their indices.  Taken keys
// become 0.  Returns the last one's key.
template <int kV>
__device__ __forceinline__ uint32_t take_top(uint32_t key[kV], int k, int i0, int* sel) {
    uint32_t m = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t mine = key[0];
#pragma unroll
        for (int i = 1; i < kV; ++i) mine = mine > key[i] ? mine : key[i];
        m = row_max_u32(mine);
        int at = 1 << 20;                               // the first of them in this lane, then in the row
#pragma unroll
        for (int i = kV - 1; i >= 0; --i) at = key[i] == m ? ahead(i) : at;
        at += i0;
        const int best = (int)~row_max_u32(~(uint32_t)at);
        if (at == best) sel[j] = best;
#pragma unroll
        for (int i = 0; i < kV; ++i) key[i] = ahead(i) == best - i0 ? 0u : key[i];
    }
    return m;
}
// s + bias in 64 bits.  zmax and sum: the row's maximum (0 for a row of -inf alone) and its sum
// of e^(z - zmax) (softmax)
template <bool kSig> __device__ __forceinline__ double exact_key(float z, float b, float zmax, double sum) {
    double s;
    if constexpr (kSig) s = 1.0 / (1.0 + exp(-(double)z));
    else s = exp((double)z - (double)zmax) / sum;
    return choice_key(key_score(s, z) + (double)b);
}
template <int kV, bool kSig>
__device__ __forceinline__ double exact_sum(const void* logits, int64_t row, int i0, int E, float& zmax, bool f32) {
    zmax = 0.0f;
    if constexpr (kSig) return 1.0;
    float top = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < kV; ++i)
        if (ahead(i) < E - i0) top = __builtin_fmaxf(top, ld_logit(logits, row + i0 + ahead(i), f32));
    top = row_max(top);
    zmax = top == -INFINITY ? 0.0f : top;
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < kV; ++i) {
        const float z = ahead(i) < E - i0 ? ld_logit(logits, row + i0 + ahead(i), f32) : -INFINITY;
        sum += exp((double)z - (double)zmax);
    }
    for (int o = 8; o; o >>= 1) sum += __shfl_xor(sum, o, 16);
    return sum == 0.0 ? 1.0 : sum;
}
// the k largest by keys in 64 bits, each computed when it is compared (rare: few registers
// matter more than time)
template <int kV, bool kSig>
__device__ __forceinline__ void take_top_exact(const RouterArgs& g, int64_t row, int i0, bool f32, int* sel) {
    float zmax;
    const double sum = exact_sum<kV, kSig>(g.logits, row, i0, g.E, zmax, f32);
    uint32_t taken = 0;
    for (int j = 0; j < g.k; ++j) {
        double m = -(double)INFINITY;
        int at = 1 << 20;
#pragma unroll 1
        for (int i = 0; i < kV; ++i) {
            const int e = i0 + ahead(i);
            if (e >= g.E || (taken >> i & 1)) continue;
            const double key = exact_key<kSig>(ld_logit(g.logits, row + e, f32), g.bias[e], zmax, sum);
            if (key > m || at == 1 << 20) { m = key; at = e; }
        }
        for (int o = 8; o; o >>= 1) {
            const double om = __shfl_xor(m, o, 16);
            const int oa = __shfl_xor(at, o, 16);
            if (oa != 1 << 20 && (at == 1 << 20 || om > m || (om == m && oa < at))) { m = om; at = oa; }
        }
        if ((threadIdx.x & 15) == 0) sel[j] = at;
#pragma unroll
        for (int i = 0; i < kV; ++i) taken |= ahead(i) == at - i0 ? 1u << i : 0u;
    }
}

// LDS writes of one wave, read by its other lanes
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Keys that FP32 rounding may have brought into a wrong order lie this close (relative to the larger
// of 1 and the key).  With u = 2^-24, softmax: e^x is off by (3 |x| + 2) u, the row's sum by its 15 + 4
// additions and the terms' errors weighted with p (sum p |x| < 3.4 for 256 terms), 31 u, the
// reciprocal and the product by 2 u.  Two scores add up to at most 1, so all that is common to a row or
// relative to a score comes to 35 u in their difference, p |x| <= 0.4 to 3 u, and the rounding of two
// keys to 2 u of the key: 40 u = 2.4e-6.  (A row that rounds the same way in one lane reaches
// 8.8e-7; with sigmoid it is 10 u.)  The bound and two thirds of it:
constexpr float kNear = 4e-6f;

constexpr int kOneK = 8, kTwoK = 20;     // largest k with bounds from the lanes' first one and two
constexpr int kCand = 32;                // candidates a row, at most

// how many of the other 15 lanes' values are larger than v
template <int kN = 15> __device__ __forceinline__ void count_above(float v, int& above) {
    above += __uint_as_float(dpp<0x120 + kN>(__float_as_uint(v))) > v;
    if constexpr (kN > 1) count_above<kN - 1>(v, above);
}
// the same of two values a lane, which pass by one lane at a time (side by side they take 30
// registers)
template <int kN = 15>
__device__ __forceinline__ void count_above(float a, float b, float ra, float rb, int& above_a, int& above_b) {
    ra = __uint_as_float(dpp<0x121>(__float_as_uint(ra)));
    rb = __uint_as_float(dpp<0x121>(__float_as_uint(rb)));
    above_a += (ra > a) + (rb > a);
    above_b += (ra > b) + (rb > b);
    if constexpr (kN > 1) count_above<kN - 1>(a, b, ra, rb, above_a, above_b);
}
// A bound that at least k of the row's keys reach: the k-th largest of the lanes' largest keys, or
// of their two largest.  It is the smallest of those with fewer than k above it.
template <int kV> __device__ __forceinline__ float bound_of(const float key[kV], int k) {
    if (__builtin_expect(k <= kOneK, 1)) {
        float a = key[0];
#pragma unroll
        for (int i = 1; i < kV; ++i) a = __builtin_fmaxf(a, key[i]);
        a = choice_key(a);
        int above = 0;
        count_above(a, above);
        return -row_max(above < k ? -a : -INFINITY);
    }
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        b = key[i] > a ? a : __builtin_fmaxf(b, key[i]);
        a = __builtin_fmaxf(a, key[i]);
    }
    int above_a = 0, above_b = a > b;
    count_above(a, b, a, b, above_a, above_b);
    return -row_max(above_b < k ? -b : above_a < k ? -a : -INFINITY);
}
// Indices of the row's candidates, which reach the bound, into list, ascending; returns how many
// there are (more than kCand: the list is not to be used).  slack: how far below the bound a key
// still counts.
template <int kV>
__device__ __forceinline__ int find_candidates(const float key[kV], float bound, int i0, int E, float slack, int* list) {
    bound -= slack * __builtin_fmaxf(1.0f, __builtin_fabsf(bound));
    if (!(bound > -INFINITY)) bound = -INFINITY;        // +inf gives NaN: then every key counts
    uint32_t m = 0;                                     // a NaN key is a candidate, which counts as -inf
#pragma unroll
    for (int i = kV - 1; i >= 0; --i) m = m + m + !(key[i] < bound);
    auto exist = [&](int room) { return room > 7 ? 0xFFu : room > 0 ? (1u << room) - 1 : 0u; };
    uint32_t all = exist(E - i0);
    if constexpr (kV == 16) all |= exist(E - i0 - 128) << 8;
    m &= all;
    // candidates of the lanes below, of each half of the row: row_shr, 0 past the row
    const uint32_t n = (uint32_t)__builtin_popcount(m & 0xFF) | (uint32_t)__builtin_popcount(m >> 8) << 16;
    uint32_t incl = n;
    incl += dpp<0x111>(incl);
    incl += dpp<0x112>(incl);
    incl += dpp<0x114>(incl);
    incl += dpp<0x118>(incl);
    const uint32_t total = row_max_u32(incl);           // the last lane's, in both halves
    const int sum = (int)((total & 0xFFFF) + (total >> 16));
    int pos = (int)((incl - n) & 0xFFFF);
    // where the second half's go less where they would go if they followed the lane's first ones
    const int jump = kV == 16 ? (int)((total & 0xFFFF) + (incl >> 16) - (n >> 16) - (incl & 0xFFFF)) : 0;
    while (__ballot(m != 0)) {
        if (m) {
            const int i = __builtin_ctz(m), at = pos + (i < 8 ? 0 : jump);
            if (at < kCand) list[at] = i0 + ahead(i);
            ++pos;
            m &= m - 1;
        }
    }
    return sum;
}

// Where each candidate of a row (n of them, kH to a lane) comes in the order: id and place of this
// lane's ones; place >= k: not chosen.  With a bias FP32 keys order the candidates only
// where every other key is further off than kNear; otherwise (a tie too, and among infinite keys,
// whose differences say nothing) 64 bits do.
template <int kH, int kV, bool kF32, bool kSig, bool kBias>
__device__ __forceinline__ void place_candidates(const RouterArgs& g, int64_t t, int i0, int n, float base, float inv,
                                                 const int* list, float* keys, double* keys64, int (&id)[2],
                                                 int (&place)[2]) {
    const int l16 = threadIdx.x & 15;
    const int64_t row = t * g.E;
    float own[kH];
    id[1] = 0;
    place[1] = g.k;
#pragma unroll
    for (int h = 0; h < kH; ++h) {
        const int c = l16 + 16 * h;
        id[h] = c < n ? list[c] : 0;
        const float z = ld_logit(g.logits, row + id[h], kF32);
        own[h] = choice_key(kBias ? key_score(one_score<kSig>(z, base, inv), z) + g.bias[id[h]] : z);
        keys[c] = c < n ? own[h] : NAN;                 // compares with nothing
        place[h] = c < n ? 0 : g.k;
    }
    wave_fence();
    int close[kH] = {};                                 // keys within kNear, the own one among them
#pragma unroll
    for (int c = 0; c < 16 * kH; c += 4) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&keys[c]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int h = 0; h < kH; ++h) {
                if constexpr (kBias) {
                    place[h] += v[u] > own[h];
                    close[h] += __builtin_fabsf(v[u] - own[h]) <= kNear * __builtin_fmaxf(1.0f, __builtin_fabsf(own[h]));
                } else {
                    place[h] += v[u] > own[h] || (v[u] == own[h] && c + u < l16 + 16 * h);
                }
            }
    }
    if constexpr (kBias) {
        bool near = false;
#pragma unroll
        for (int h = 0; h < kH; ++h) near |= (close[h] > 1 || __builtin_fabsf(own[h]) == INFINITY) && place[h] < g.k;
        if (__builtin_expect(!__ballot(near), 1)) return;
        float zmax;
        const double sum = exact_sum<kV, kSig>(g.logits, row, i0, g.E, zmax, kF32);
        double own64[kH];
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            const int c = l16 + 16 * h;
            own64[h] = exact_key<kSig>(ld_logit(g.logits, row + id[h], kF32), g.bias[id[h]], zmax, sum);
            keys64[c] = c < n ? own64[h] : (double)NAN;
            place[h] = c < n ? 0 : g.k;
        }
        wave_fence();
#pragma unroll 1
        for (int c = 0; c < 16 * kH; ++c) {
            const double v = keys64[c];
#pragma unroll
            for (int h = 0; h < kH; ++h) place[h] += v > own64[h] || (v == own64[h] && c < l16 + 16 * h);
        }
    }
}

// the loss from sum counts_e P_e and sum counts_e
__device__ __forceinline__ float loss_value(const RouterArgs& g, double a, double n) {
    n /= g.k;
    return n > 0.0 ? (float)((double)g.coef * g.E / (g.k * n * n) * a) : 0.0f;
}
// those sums from one expert per thread, e < 256, and the loss
__device__ __forceinline__ void write_loss(const RouterArgs& g, int count, float psum, double (*part)[2]) {
    double a = (double)count * (double)psum, n = (double)count;
    for (int o = 32; o; o >>= 1) { a += __shfl_xor(a, o, 64); n += __shfl_xor(n, o, 64); }
    if ((threadIdx.x & 63) == 0 && threadIdx.x < 256) { part[threadIdx.x >> 6][0] = a; part[threadIdx.x >> 6][1] = n; }
    __syncthreads();
    if (threadIdx.x == 0 && g.loss) {
        a = n = 0.0;
        for (int w = 0; w < 4; ++w) { a += part[w][0]; n += part[w][1]; }
        *g.loss = loss_value(g, a, n);
    }
}

template <int kThr, int kV, bool kF32, bool kSig, bool kBias>
__global__ __launch_bounds__(kThr) void route_kernel(RouterArgs g) {
    constexpr int kR = kThr / 16;
    __shared__ int sel[kR][kCand];
    __shared__ __attribute__((aligned(16))) float keys[kR][kCand];
    __shared__ double keys64[kBias ? kR : 1][kCand];
    __shared__ int cnt[256];
    __shared__ float sums[kThr / MOE_WAVE][256];
    __shared__ double part[4][2];
    static_assert(kMaxTopK <= kCand, "sel holds a row's choice too");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = tid & 15, row = tid >> 4;
    const int E = g.E, k = g.k, i0 = first<kV>(l16);
    if (tid < 256) cnt[tid] = 0;
    __syncthreads();
    float acc[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = 0.0f;
    // rows past T repeat row T - 1 and write nothing (their lanes take part in every DPP step)
    for (int64_t t0 = (int64_t)blockIdx.x * kR; t0 < g.T; t0 += (int64_t)gridDim.x * kR) {
        const bool in = t0 + row < g.T;
        const int64_t t = in ? t0 + row : g.T - 1;
        const bool live = in && (!g.mask || g.mask[t]);
        float z[kV], s[kV], base, inv;
        load_row<kV, kF32>(g.logits, t * E, i0, E, g.vec, z);
        row_scores<kV, kSig>(z, s, base, inv);
        if (live) {
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] += kSig ? s[i] * inv : s[i];
        }
        if constexpr (kBias) {
#pragma unroll
            for (int i = 0; i < kV; ++i) s[i] = key_score(s[i], z[i]);
            load_row<kV, true>(g.bias, 0, i0, E, g.bias_vec, z);
#pragma unroll
            for (int i = 0; i < kV; ++i) z[i] += s[i];  // keys from here on
        }
        int n = kCand + 1;
        if (k <= kTwoK) n = find_candidates<kV>(z, bound_of<kV>(z, k), i0, E, kBias ? kNear : 0.0f, sel[row]);
        // the ways marked unlikely lie behind the usual one, which a wave walks through once: in their
        // places between its parts they cost 16384 rows 0.5 to 1 us of instruction fetches
        bool placed = !__ballot(n > kCand);
        uint32_t last = 0;                              // the k-th largest key, where the maxima were taken
        if (__builtin_expect(!placed, 0)) {
            uint32_t key[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) key[i] = ahead(i) < E - i0 ? order_key(z[i]) : 0u;
            wave_fence();
            last = take_top<kV>(key, k, i0, sel[row]);
            wave_fence();
            if constexpr (kBias) {
                // that key is the best bound; the candidates go to 64 bits only if they have to
                int* list = reinterpret_cast<int*>(keys[row]);
                n = find_candidates<kV>(z, key_value(last), i0, E, kNear, list);
                placed = !__ballot(n > kCand);
                wave_fence();
                if (placed) {
                    sel[row][l16] = list[l16];
                    sel[row][l16 + 16] = list[l16 + 16];
                }
                wave_fence();
            }
        }
        if (__builtin_expect(placed, 1)) {
            wave_fence();
            double* k64 = keys64[kBias ? row : 0];
            int id[2], place[2];
            if (__builtin_expect(__ballot(n > 16) != 0, 0))
                place_candidates<2, kV, kF32, kSig, kBias>(g, t, i0, n, base, inv, sel[row], keys[row], k64, id, place);
            else
                place_candidates<1, kV, kF32, kSig, kBias>(g, t, i0, n, base, inv, sel[row], keys[row], k64, id, place);
            wave_fence();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (place[h] < k) sel[row][place[h]] = id[h];
            wave_fence();
        } else {
            if constexpr (kBias) {
                // is every neighbour in the order, and everything around the last one, either
                // further off than FP32 rounding reaches, or the same logit and bias (a true
                // tie, which the index has settled)?
                bool near = false;
                const int e_last = sel[row][k - 1];
                const float z_last = ld_logit(g.logits, t * E + e_last, kF32), b_last = g.bias[e_last];
                const float k_last = key_value(last);
                const float reach = kNear * __builtin_fmaxf(1.0f, __builtin_fabsf(k_last));
#pragma unroll 1
                for (int i = 0; i < kV; ++i) {
                    const int e = i0 + ahead(i);
                    if (e >= E) continue;
                    const float zi = ld_logit(g.logits, t * E + e, kF32), bi = g.bias[e];
                    const float ki = choice_key(key_score(one_score<kSig>(zi, base, inv), zi) + bi);
                    near |= __builtin_fabsf(ki - k_last) <= reach && !(zi == z_last && bi == b_last);
                }
                for (int j = l16; j + 1 < k; j += 16) {
                    const int ea = sel[row][j], eb = sel[row][j + 1];
                    const float za = ld_logit(g.logits, t * E + ea, kF32), zb = ld_logit(g.logits, t * E + eb, kF32);
                    const float ba = g.bias[ea], bb = g.bias[eb];
                    const float ka = choice_key(key_score(one_score<kSig>(za, base, inv), za) + ba);
                    const float kb = choice_key(key_score(one_score<kSig>(zb, base, inv), zb) + bb);
                    near |= !(ka - kb > kNear * __builtin_fmaxf(1.0f, __builtin_fabsf(ka))) && !(za == zb && ba == bb);
                }
                if (__ballot(near)) {
                    wave_fence();
                    take_top_exact<kV, kSig>(g, t * E, i0, kF32, sel[row]);
                    wave_fence();
                }
            }
        }
        // sel holds the choice in order: lane j takes the j-th (and j + 16-th), so that the sum
        // of the scores does not depend on how the row's choice was found
        int id[2];
        float sc[2], total = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = l16 + 16 * h;
            id[h] = j < k ? sel[row][j] : 0;
            sc[h] = j < k ? one_score<kSig>(ld_logit(g.logits, t * E + id[h], kF32), base, inv) : 0.0f;
            total += sc[h];
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
        wave_fence();                                   // sel and keys are rewritten by the next rows
    }
    if (!g.part_counts) return;
    // the rows' probabilities added over the wave's four rows, then the workgroup's waves
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        acc[i] += __shfl_xor(acc[i], 16, 64);
        acc[i] += __shfl_xor(acc[i], 32, 64);
        if (lane < 16) sums[wave][i0 + ahead(i)] = acc[i];
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
        if (blockIdx.x == 0 && tid == 0) *g.ticket = 0;
        g.part_counts[(size_t)blockIdx.x * g.stride + tid] = c;
        g.part_sums[(size_t)blockIdx.x * g.stride + tid] = p;
    }
}

// Counts, sums and loss from the workgroups' partial rows: 16 experts per workgroup, a thread
// four of them in every 64th row, then the lanes and the waves in a fixed order.  The loss
// needs every expert: each workgroup leaves its share, and the last one to do so (a ticket that
// route_kernel has cleared) adds the shares in order.  5.6 us for the 512 KB of 256 workgroups and
// experts (one workgroup for all of it: 7.4 us).
__global__ __launch_bounds__(kThreads) void route_final_kernel(RouterArgs g, int blocks) {
    __shared__ float ps[4][16];
    __shared__ int cs[4][16];
    const int tid = threadIdx.x, q = tid & 3, col = 16 * blockIdx.x + 4 * q;
    f32x4_t p = {0.f, 0.f, 0.f, 0.f};
    int4 c = make_int4(0, 0, 0, 0);
    if (col < g.stride)
#pragma unroll
        for (int u = 0; u < kRouterBlocks / 64; ++u) {
            const int b = (tid >> 2) + 64 * u;
            if (b < blocks) {
                p += *reinterpret_cast<const f32x4_t*>(g.part_sums + (size_t)b * g.stride + col);
                const int4 v = *reinterpret_cast<const int4*>(g.part_counts + (size_t)b * g.stride + col);
                c.x += v.x; c.y += v.y; c.z += v.z; c.w += v.w;
            }
        }
    for (int o = 4; o < 64; o <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] += __shfl_xor(p[i], o, 64);
        c.x += __shfl_xor(c.x, o, 64); c.y += __shfl_xor(c.y, o, 64);
        c.z += __shfl_xor(c.z, o, 64); c.w += __shfl_xor(c.w, o, 64);
    }
    if ((tid & 63) < 4) {
        const int cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ps[tid >> 6][4 * q + i] = p[i];
            cs[tid >> 6][4 * q + i] = cc[i];
        }
    }
    __syncthreads();
    if (tid >= 16) return;
    const int e = 16 * blockIdx.x + tid;
    const float sum = ((ps[0][tid] + ps[1][tid]) + ps[2][tid]) + ps[3][tid];
    const int count = cs[0][tid] + cs[1][tid] + cs[2][tid] + cs[3][tid];
    if (e < g.E) {
        if (g.counts) g.counts[e] = count;
        if (g.psum) g.psum[e] = sum;
    }
    double a = e < g.E ? (double)count * (double)sum : 0.0, n = e < g.E ? (double)count : 0.0;
    for (int o = 8; o; o >>= 1) { a += __shfl_xor(a, o, 16); n += __shfl_xor(n, o, 16); }
    int ticket = 0;
    if (tid == 0) {
        __hip_atomic_store(&g.shares[2 * blockIdx.x], a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&g.shares[2 * blockIdx.x + 1], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        ticket = __hip_atomic_fetch_add(g.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__shfl(ticket, 0, 16) != (int)gridDim.x - 1 || !g.loss) return;
    // a lane for each share, so that their loads overlap
    const bool have = tid < (int)gridDim.x;
    a = have ? __hip_atomic_load(&g.shares[2 * tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    n = have ? __hip_atomic_load(&g.shares[2 * tid + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    for (int o = 8; o; o >>= 1) { a += __shfl_xor(a, o, 16); n += __shfl_xor(n, o, 16); }
    if (tid != 0) return;
    *g.loss = loss_value(g, a, n);
}

// A row is read, and its gradient written, once; the row's scores are computed again rather than
// kept.  8192 x 128 in FP32 5.2 us, 16384 x 256 in BF16 8.4 us (17.8 MB: 2.1 TB/s): as in the
// forward, the chain of reductions of one pass over the chip is most of it.
template <int kV, bool kF32, bool kSig>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouterGradArgs g) {
    constexpr int kStep = kV + 4;
    // of the chosen, by way of the scores: p_j ds_j (softmax), s_j (1 - s_j) ds_j (sigmoid)
    __shared__ __attribute__((aligned(16))) float extra[kRows][16 * kStep];
    __shared__ __attribute__((aligned(16))) float shared[16 * kStep];   // counts
    __shared__ int64_t part[kThreads / MOE_WAVE];
    const int tid = threadIdx.x, l16 = tid & 15, row = tid >> 4;
    const int E = g.E, k = g.k, i0 = first<kV>(l16);
    // b_e of this lane's experts
    float bal[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) bal[i] = 0.0f;
    // a row's logits, and this lane's chosen experts with g_j: loaded ahead of their use
    float z[kV], gj[2], zj[2];
    int id[2];
    auto load = [&](int64_t t0) {
        const int64_t t = t0 + row < g.T ? t0 + row : g.T - 1;
        load_row<kV, kF32>(g.logits, t * E, i0, E, g.vec, z);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = l16 + 16 * h;
            id[h] = j < k ? g.ids[t * k + j] : -1;
            if ((unsigned)id[h] >= (unsigned)E) id[h] = -1;
            gj[h] = id[h] >= 0 && g.dscores ? g.dscores[t * k + j] * g.scale : 0.0f;
            zj[h] = id[h] >= 0 ? ld_logit(g.logits, t * E + id[h], kF32) : 0.0f;
        }
    };
    load((int64_t)blockIdx.x * kRows);
    // where expert e's entry lies: by lane, as the lanes hold the logits
    auto slot = [](int e) { return kV == 16 ? (e >> 3 & 15) * kStep + (e >> 7) * 8 + (e & 7) : e / kV * kStep + e % kV; };
    const int x0 = l16 * kStep;                           // padded, so that the lanes' pieces meet few banks twice
    if (g.dloss) {
        // every count is read once by the workgroup and shared: reading kV of them per lane from
        // memory made 16384 x 256 take 14.0 us
        const int c = tid < E ? g.counts[tid] : 0;
        int64_t n = c;
        for (int o = 32; o; o >>= 1) n += __shfl_xor((long long)n, o, 64);
        if ((tid & 63) == 0) part[tid >> 6] = n;
        if (tid < 16 * kV) shared[slot(tid)] = (float)c;
        __syncthreads();
        n = 0;
        for (int w = 0; w < kThreads / MOE_WAVE; ++w) n += part[w];
        // coef E / (k N^2) with N = n / k
        const float f = n > 0 ? *g.dloss * g.coef * (float)(E * k) / (float)n / (float)n : 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) bal[i] = f * shared[x0 + i];
    }
    float* ex = &extra[row][0];
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < g.T; t0 += (int64_t)gridDim.x * kRows) {
        const bool in = t0 + row < g.T;
        const int64_t t = in ? t0 + row : g.T - 1;
        const bool live = !g.mask || g.mask[t];
#pragma unroll
        for (int i = 0; i < kV; ++i) ex[x0 + i] = 0.0f;
        // f: what dz_e is a multiple of, p (softmax) or s (1 - s) (sigmoid); pb: sum p b
        float f[kV], base = 0.0f, sum = 0.0f, pb = 0.0f;
        if constexpr (kSig) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                // e / (1 + e)^2 with e = e^-|z| does not cancel
                const float e = exp_f(-__builtin_fabsf(z[i])), r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
                const float s = z[i] >= 0.0f ? r : er;
                sum += s;
                pb += s * bal[i];
                f[i] = er * r;
            }
        } else {
            float m = z[0];
#pragma unroll
            for (int i = 1; i < kV; ++i) m = __builtin_fmaxf(m, z[i]);
            base = base_of(row_max(m));
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                f[i] = exp_f(z[i] - base);
                sum += f[i];
                pb += f[i] * bal[i];
            }
        }
        sum = row_sum(sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        pb = row_sum(pb) * inv;
        float sj[2], total = 0.0f, dot = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sj[h] = id[h] >= 0 ? one_score<kSig>(zj[h], base, inv) : 0.0f;
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
            // normalize: s_j ds_j = v_j (g_j - dot), whose sum over j is zero (1 / total alone may be too
            // large for a product)
            float r = g.normalize ? vj[h] * (gj[h] - dot) : sj[h] * gj[h];
            if constexpr (kSig) r *= one_score<true>(-zj[h], 0.0f, 0.0f);    // 1 - s_j does not cancel
            else own += r;
            if (id[h] >= 0) ex[slot(id[h])] = r;
        }
        wave_fence();
        if constexpr (!kSig) {
            if (!g.normalize) pb += row_sum(own);
        }
        float out[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) out[i] = f[i] * inv * (bal[i] - pb) + ex[x0 + i];
        if (!live) {
#pragma unroll
            for (int i = 0; i < kV; ++i) out[i] = 0.0f;
        }
        if (t0 + (int64_t)gridDim.x * kRows < g.T) load(t0 + (int64_t)gridDim.x * kRows);
        if (in) store_row<kV, kF32>(g.dlogits, t * E, i0, E, g.vec, out);
        wave_fence();                                   // extra is rewritten by the next rows
    }
}

// Up to kOneBlock rows go to one workgroup, which needs no second launch for its sums: 64 rows of
// 128 logits take 7.0 us in a graph (two passes, 128 rows, 11.3; 65 rows in two launches 8.4)
// and 2.7 us less of the host.  Workgroups of 1024 threads there, and once there are more rows
// than one pass of the smaller ones over the chip: the same rows in flight with a quarter of
// the partial sums.
constexpr int kOneBlock = 64;
bool wide_blocks(int64_t T) { return (T > kRows && T <= kOneBlock) || T > (int64_t)kRouterBlocks * kRows; }

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
    if (T <= kOneBlock) return 1;
    const int rows = wide_blocks(T) ? kWide / 16 : kRows;
    const int64_t b = (T + rows - 1) / rows;
    return (int)(b < 1 ? 1 : b < kRouterBlocks ? b : kRouterBlocks);
}

hipError_t launch_route(RouterArgs g, bool sigmoid, bool f32, hipStream_t s) {
    const bool stats = g.part_counts != nullptr;
    if (g.T == 0 && !stats) return hipSuccess;
    g.vec = aligned_rows(g.logits, g.logits, g.E, f32);
    g.bias_vec = aligned_rows(g.bias, g.bias, g.E, true);
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
    hipLaunchKernelGGL(route_final_kernel, dim3((g.E + 15) / 16), dim3(kThreads), 0, s, g, grid);
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
