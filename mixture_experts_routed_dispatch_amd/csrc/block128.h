// block128.h -- what the kernels on E4M3 codes with one FP32 scale per 128 share: a block's scale
// and the codes of its values.
#pragma once

#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

// The scale of a block from the bits of its largest magnitude (magnitudes of floats order like
// their bits, infinities and NaN above all): amax / 448 rounded once, at least 2^-100, which keeps
// the quotients' remainders below exact; NaN for a block that holds an infinity or NaN, so that
// what is computed from it is NaN.  With r = 1 / 448 rounded, the quotient a r plus its remainder times r
// is the correctly rounded one (Markstein's theorem; where a is too small for that the floor holds).
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    constexpr float r = 1.0f / 448.0f;
    const float a = __uint_as_float(amax_bits), q = a * r;
    const float s = __builtin_fmaxf(__builtin_fmaf(__builtin_fmaf(-q, 448.0f, a), r, q), 0x1p-100f);
    return amax_bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : s;
}
// 1 / s within an ulp, for block_quotient
__device__ __forceinline__ float block_inverse(float s) { return __builtin_amdgcn_rcpf(s); }

// v / s for |v| <= 448 s (1 + 2^-24), as a float that rounds to the same E4M3 value as the exact
// quotient does (nearest, ties to even).  q is within an ulp of the quotient.  Where it is not the
// quotient itself and its last bit is 0, it goes one ulp towards the quotient: E4M3 values and the
// midpoints between them have that bit 0, so none of them lies between the result and the
// quotient.  The sign of the remainder v - q s is that of the exact one, which fma rounds once.
__device__ __forceinline__ float block_quotient(float v, float s, float inv) {
    const float a = __builtin_fabsf(v);
    float q = a * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, a), inv, q);
    const float rest = __builtin_fmaf(-q, s, a);
    uint32_t b = __float_as_uint(q);
    b -= rest < 0.0f;                                  // (only where q > 0)
    b |= rest != 0.0f;
    return __builtin_copysignf(__uint_as_float(b), v);
}

// Codes of four values.  With a NaN scale they are any codes: what is multiplied with that scale is NaN whatever they are.
// v inv is within three of its own last places of the quotient (the reciprocal's ulp and a rounding), so that it
// rounds as the quotient does unless a midpoint between two E4M3 values is that near: from 2^-6 on, where these have
// three bits behind the point, one whose 20 last bits are 0x80000.  Such values, and smaller ones, are settled by
// block_quotient.  (Every value that way: a layer of 16384 x 4096 x 2048, 64 experts, 3658 us against 3612.)  What is above 448 by
// those last places rounds to it.
__device__ __forceinline__ uint32_t block_codes4(float a, float b, float c, float d, float s, float inv) {
    const float v[4] = {a, b, c, d};
    float q[4], least = INFINITY;
    uint32_t near = 0xFFFFFFFFu;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
        q[z] = v[z] * inv;
        const uint32_t t = (__float_as_uint(q[z]) << 12) - (0x7FFFCu << 12);
        near = near < t ? near : t;
        least = __builtin_fminf(least, __builtin_fabsf(q[z]));
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    if (__builtin_expect(near < 8u << 12 || least < 0x1p-6f, 0))
        return e4m3_pack4(block_quotient(a, s, inv), block_quotient(b, s, inv), block_quotient(c, s, inv),
                          block_quotient(d, s, inv));
    return (uint32_t)w;
}
// largest magnitude, as bits, of eight BF16 values
__device__ __forceinline__ uint32_t bf16_amax_bits(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = w[i] & 0x7FFF0000u, l = (w[i] << 16) & 0x7FFF0000u;
        hi = hi > h ? hi : h;
        lo = lo > l ? lo : l;
    }
    return hi > lo ? hi : lo;
}
__device__ __forceinline__ uint2 block_codes8(uint4 v, float s, float inv) {
    return make_uint2(block_codes4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y), s, inv),
                      block_codes4(bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w), s, inv));
}
// maximum over the 16 lanes of a DPP row, in all of them
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    auto turn = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xF, 0xF, true);
    };
    uint32_t o;
    o = turn(v, std::integral_constant<int, 0x128>()); v = v > o ? v : o;
    o = turn(v, std::integral_constant<int, 0x124>()); v = v > o ? v : o;
    o = turn(v, std::integral_constant<int, 0x122>()); v = v > o ? v : o;
    o = turn(v, std::integral_constant<int, 0x121>()); v = v > o ? v : o;
    return v;
}

}  // namespace
}  // namespace moe
