// block_api.cpp -- C entry points around the routed expert layer (include/moe.h): 4-bit
// weights, the router and the norms.  Checks of arguments and launches only.
#include <cmath>

#include "../../include/moe.h"
#include "kernels.h"
#include "plan.h"

using namespace moe;

static bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

extern "C" {

moe_status_t moe_prepare_weights(moe_plan_t p, const void* w13, const void* w2, uint8_t* w13_q,
                                 uint8_t* w13_s, uint8_t* w2_q, uint8_t* w2_s, void* stream) {
    if (!p || !w13 || !w2 || !w13_q || !w13_s || !w2_q || !w2_s) return MOE_ERR_INVALID_ARG;
    const moe_config_t& c = p->cfg;
    if (c.d % 128 != 0 || c.I % 128 != 0) return MOE_ERR_UNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (c.precision == MOE_MXFP4) {
        if (!aligned16(w13) || !aligned16(w2) || !aligned16(w13_q) || !aligned16(w13_s) || !aligned16(w2_q) || !aligned16(w2_s))
            return MOE_ERR_INVALID_ARG;
        const Mxfp4Args g{{mxfp4_w13(w13, w13_q, w13_s, c.E, c.I, c.d), mxfp4_w2(w2, w2_q, w2_s, c.E, c.I, c.d)}};
        if (launch_mxfp4_pack(g, s) != hipSuccess) return MOE_ERR_HIP;
        return MOE_OK;
    }
    if (c.precision == MOE_FP8_BLOCK128) {
        if (!aligned16(w13) || !aligned16(w2) || !aligned16(w13_q) || !aligned16(w13_s) || !aligned16(w2_q) || !aligned16(w2_s))
            return MOE_ERR_INVALID_ARG;
        const Block128Pair g{{block128(w13, w13_q, w13_s, c.E, 2 * c.I, c.d), block128(w2, w2_q, w2_s, c.E, c.d, c.I)}};
        return launch_block128_pack(g, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
    }
    // block-major scales (the layout the MXFP8 GEMMs copy from)
    if (launch_quantize_mxfp8(static_cast<const uint16_t*>(w13), (int64_t)c.E * 2 * c.I, c.d, w13_q, w13_s,
                              true, s) != hipSuccess)
        return MOE_ERR_HIP;
    if (launch_quantize_mxfp8(static_cast<const uint16_t*>(w2), (int64_t)c.E * c.d, c.I, w2_q, w2_s, true,
                              s) != hipSuccess)
        return MOE_ERR_HIP;
    return MOE_OK;
}

moe_status_t moe_expand_weights(moe_plan_t p, const moe_weights_t* w, void* w13, void* w2, void* stream) {
    if (!p || !w || !w13 || !w2 || !w->w13 || !w->w2 || !w->w13_scale || !w->w2_scale) return MOE_ERR_INVALID_ARG;
    const moe_config_t& c = p->cfg;
    if (c.precision != MOE_MXFP4 && c.precision != MOE_FP8_BLOCK128) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(w->w13) || !aligned16(w->w2) || !aligned16(w->w13_scale) || !aligned16(w->w2_scale) || !aligned16(w13) ||
        !aligned16(w2))
        return MOE_ERR_INVALID_ARG;
    if (c.precision == MOE_FP8_BLOCK128) {
        const Block128Pair b{{block128(w13, w->w13, w->w13_scale, c.E, 2 * c.I, c.d), block128(w2, w->w2, w->w2_scale, c.E, c.d, c.I)}};
        return launch_block128_expand(b, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
    }
    const Mxfp4Args g{{mxfp4_w13(w13, w->w13, w->w13_scale, c.E, c.I, c.d), mxfp4_w2(w2, w->w2, w->w2_scale, c.E, c.I, c.d)}};
    return launch_mxfp4_expand(g, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

static moe_status_t router_check(const moe_router_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->T < 0 || c->E <= 0 || c->k <= 0) return MOE_ERR_INVALID_ARG;
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if ((c->normalize != 0 && c->normalize != 1) || (c->logits_f32 != 0 && c->logits_f32 != 1)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->scale) || !std::isfinite(c->balance_coef)) return MOE_ERR_INVALID_ARG;
    if (c->groups < 0 || c->top_groups < 0 || c->group_top < 0) return MOE_ERR_INVALID_ARG;
    if (c->groups == 0 ? c->top_groups != 0 || c->group_top != 0
                       : c->top_groups < 1 || c->top_groups > c->groups || c->group_top < 1 || c->group_top > 2)
        return MOE_ERR_INVALID_ARG;
    if (c->E > kMaxExperts || c->k > c->E || c->k > kMaxTopK) return MOE_ERR_UNSUPPORTED;
    if (c->groups > 0) {
        // groups of one size, which hold the keys that rank them, and enough experts in the chosen ones
        if (c->groups > kMaxRouterGroups || c->E % c->groups != 0) return MOE_ERR_UNSUPPORTED;
        const int size = c->E / c->groups;
        if (c->group_top > size || c->k > c->top_groups * size) return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

// the loss' shares and ticket, in front of the partial counts and sums
constexpr size_t kRouterHead = 32 * sizeof(double) + 16;

size_t moe_router_workspace_bytes(const moe_router_config_t* c) {
    if (router_check(c) != MOE_OK) return 0;
    return (size_t)router_blocks(c->T) * ((c->E + 3) & ~3) * (sizeof(int32_t) + sizeof(float)) + kRouterHead;
}

moe_status_t moe_router_forward(const moe_router_config_t* c, const void* logits, const float* bias,
                                const uint8_t* mask, int32_t* ids, float* scores, int32_t* counts,
                                float* prob_sums, float* loss, void* workspace, size_t workspace_bytes, void* stream) {
    const moe_status_t st = router_check(c);
    if (st != MOE_OK) return st;
    if (c->T > 0 && (!logits || !ids || !scores)) return MOE_ERR_INVALID_ARG;
    RouterArgs g{};
    g.T = c->T; g.E = c->E; g.k = c->k; g.normalize = c->normalize;
    g.scale = c->scale; g.coef = c->balance_coef;
    g.logits = logits; g.bias = bias; g.mask = mask;
    g.ids = ids; g.scores = scores;
    g.groups = c->groups; g.top_groups = c->top_groups; g.group_top = c->group_top;
    g.counts = counts; g.psum = prob_sums; g.loss = loss;
    if (counts || prob_sums || loss) {
        if (!workspace || workspace_bytes < moe_router_workspace_bytes(c)) return MOE_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return MOE_ERR_INVALID_ARG;
        const size_t part = (size_t)router_blocks(c->T) * ((c->E + 3) & ~3);
        g.shares = static_cast<double*>(workspace);
        g.ticket = reinterpret_cast<int32_t*>(g.shares + 32);
        g.part_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + kRouterHead);
        g.part_counts = reinterpret_cast<int32_t*>(g.part_sums + part);
    }
    const hipError_t e = launch_route(g, c->score == MOE_SCORE_SIGMOID, c->logits_f32 != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status_t moe_router_backward(const moe_router_config_t* c, const float* dscores, const void* logits,
                                 const uint8_t* mask, const int32_t* ids, const int32_t* counts, const float* dloss,
                                 void* dlogits, void* stream) {
    const moe_status_t st = router_check(c);
    if (st != MOE_OK) return st;
    if (c->T > 0 && (!logits || !ids || !dlogits)) return MOE_ERR_INVALID_ARG;
    if (dloss && !counts) return MOE_ERR_INVALID_ARG;
    RouterGradArgs g{};
    g.T = c->T; g.E = c->E; g.k = c->k; g.normalize = c->normalize;
    g.scale = c->scale; g.coef = c->balance_coef;
    g.logits = logits; g.mask = mask; g.ids = ids; g.dscores = dscores;
    g.counts = counts; g.dloss = dloss; g.dlogits = dlogits;
    const hipError_t e = launch_route_grad(g, c->score == MOE_SCORE_SIGMOID, c->logits_f32 != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

static moe_status_t norm_check(const moe_norm_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->T < 0 || c->d <= 0) return MOE_ERR_INVALID_ARG;
    if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_TOKEN) return MOE_ERR_INVALID_ARG;
    if (c->residual_f32 != 0 && c->residual_f32 != 1) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->residual_scale) || !std::isnormal(c->eps) || c->eps < 0.0f) return MOE_ERR_INVALID_ARG;
    if (c->d % 8 != 0 || c->d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t moe_norm_workspace_bytes(const moe_norm_config_t* c) {
    if (norm_check(c) != MOE_OK) return 0;
    return sizeof(float) * (size_t)kNormBlocks * 2 * c->d;
}

moe_status_t moe_norm_forward(const moe_norm_config_t* c, const void* x, const void* y, const float* w_post,
                              const float* gate, const float* w_pre, void* z, void* h, void* stream) {
    const moe_status_t st = norm_check(c);
    if (st != MOE_OK) return st;
    if (c->T == 0) return MOE_OK;
    // without a block output there is nothing to norm, gate or add, and the stream stays x
    if (!y && (w_post || gate || z)) return MOE_ERR_INVALID_ARG;
    if (y && (gate != nullptr) != (c->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if ((w_pre != nullptr) != (h != nullptr) || (!y && !h)) return MOE_ERR_INVALID_ARG;
    if (!x || (y && !z)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) || !aligned16(z) || !aligned16(h) ||
        (c->gate == MOE_GATE_CHANNEL && !aligned16(gate)))
        return MOE_ERR_INVALID_ARG;
    NormArgs g{};
    g.T = c->T; g.d = c->d; g.gate_kind = y ? c->gate : MOE_GATE_NONE;
    g.eps = c->eps; g.alpha = c->residual_scale;
    g.x = x; g.y = static_cast<const uint16_t*>(y);
    g.w_post = w_post; g.gate = gate; g.w_pre = w_pre;
    g.z = z; g.h = static_cast<uint16_t*>(h);
    const hipError_t e = launch_norm(g, c->residual_f32 != 0, device_cus(), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status_t moe_norm_backward(const moe_norm_config_t* c, const void* dz, const void* dh, const void* z, const void* y,
                               const float* w_post, const float* gate, const float* w_pre, void* dx, void* dy,
                               float* dw_post, float* dgate, float* dw_pre, void* workspace, size_t workspace_bytes,
                               void* stream) {
    const moe_status_t st = norm_check(c);
    if (st != MOE_OK) return st;
    if (c->T == 0) {
        // no rows: the sums over them are zero
        hipStream_t s = static_cast<hipStream_t>(stream);
        float* sums[3] = {dw_post, c->gate == MOE_GATE_CHANNEL ? dgate : nullptr, dw_pre};
        for (float* p : sums)
            if (p && launch_fill_i32(reinterpret_cast<int32_t*>(p), c->d, 0, s) != hipSuccess) return MOE_ERR_HIP;
        return MOE_OK;
    }
    if (!y && (w_post || gate || dy)) return MOE_ERR_INVALID_ARG;
    if (y && (gate != nullptr) != (c->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if ((dw_post != nullptr) != (w_post != nullptr) || (dgate != nullptr) != (gate != nullptr) ||
        (dw_pre != nullptr) != (w_pre != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!y && !w_pre) return MOE_ERR_INVALID_ARG;
    if (!dx || (y && !dy) || (w_pre && (!dh || !z)) || (!w_pre && !dz)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dz) || !aligned16(dh) || !aligned16(z) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
        !aligned16(dx) || !aligned16(dy) || !aligned16(dw_post) || !aligned16(dw_pre) ||
        (c->gate == MOE_GATE_CHANNEL && (!aligned16(gate) || !aligned16(dgate))))
        return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe_norm_workspace_bytes(c)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_INVALID_ARG;
    NormGradArgs g{};
    g.T = c->T; g.d = c->d; g.gate_kind = y ? c->gate : MOE_GATE_NONE;
    g.eps = c->eps; g.alpha = c->residual_scale;
    g.dz = dz; g.dh = w_pre ? static_cast<const uint16_t*>(dh) : nullptr;
    g.z = w_pre ? z : nullptr; g.y = static_cast<const uint16_t*>(y);
    g.w_post = w_post; g.gate = gate; g.w_pre = w_pre;
    g.dx = dx; g.dy = static_cast<uint16_t*>(dy);
    g.dw_post = dw_post; g.dgate = dgate; g.dw_pre = dw_pre;
    g.part = static_cast<float*>(workspace);
    const hipError_t e = launch_norm_grad(g, c->residual_f32 != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
