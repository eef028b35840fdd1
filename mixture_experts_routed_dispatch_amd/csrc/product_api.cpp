// product_api.cpp -- C entry points of the products with weights in blocks of 128 (include/moe.h):
// checks of arguments, workspace layout and launches.
#include "../../include/moe.h"
#include "kernels.h"
#include "plan.h"

using namespace moe;

static bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
static bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

static moe_status_t product_check(const moe_product_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->R < 0 || c->N <= 0 || c->K <= 0 || c->E <= 0) return MOE_ERR_INVALID_ARG;
    if ((c->training != 0 && c->training != 1) || (c->wgrad_accumulate != 0 && c->wgrad_accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    if (c->wgrad_accumulate && !c->training) return MOE_ERR_UNSUPPORTED;
    if (c->N % 128 != 0 || c->K % 128 != 0 || c->E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
    // 32-bit offsets inside a matrix, and counts of rows and tiles
    if ((int64_t)c->N * c->K >= (1LL << 31) || c->R > kMaxProductRows) return MOE_ERR_UNSUPPORTED;
    // the weight gradients' operands along the rows, as in an MXFP8 layer's
    const int64_t wide = c->N > c->K ? c->N : c->K;
    if (c->training && wide * ((int64_t)c->R + (int64_t)kMxWgradPad * c->E) >= (1LL << 32)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

namespace {
struct Room {
    size_t q, qs, groups, starts, wt, wts, tp, tps, tq, tqs, part, bytes;
};
// Pieces into which the rows of a weight gradient are cut: as many as fill the chip with tiles of 256 x 256, of
// 1024 rows at least on average (8192 rows of 2048 x 2048, four pieces: all gradients 132 us against 149 with one)
int grad_pieces(const moe_product_config_t& c) {
    constexpr int kUnits = 256, kMost = 8, kRows = 1024;
    const int64_t tiles = (int64_t)c.E * ((c.N + 255) / 256) * ((c.K + 255) / 256), rows = c.R / c.E / kRows;
    int64_t n = kUnits / tiles;
    n = n < rows ? n : rows;
    return (int)(n < 1 ? 1 : n < kMost ? n : kMost);
}
Room room_of(const moe_product_config_t& c) {
    Room r{};
    size_t off = 0;
    auto take = [&](size_t n) { const size_t o = off; off = (off + n + 255) & ~size_t(255); return o; };
    const size_t R = (size_t)c.R, wide = (size_t)(c.training && c.N > c.K ? c.N : c.K);
    r.q = take(R * wide);                                // x, or dy
    r.qs = take(R * wide / 32);
    r.groups = take(kBlock128GroupBytes);
    if (c.training) {
        const size_t tokens = R + (size_t)kMxWgradPad * c.E, weights = (size_t)c.E * c.N * c.K;
        r.starts = take(sizeof(int32_t) * (c.E + 1));
        r.wt = take(weights);
        r.wts = take(weights / 4096);
        r.tp = take(tokens * c.K);
        r.tps = take(tokens * c.K / 32);
        r.tq = take(tokens * c.N);
        r.tqs = take(tokens * c.N / 32);
        const int pieces = grad_pieces(c);
        r.part = take(pieces > 1 ? sizeof(float) * pieces * weights : 0);
    }
    r.bytes = off;
    return r;
}
}  // namespace

extern "C" {

moe_status_t moe_quantize_block128(const void* v, int64_t rows, int32_t K, uint8_t* codes, float* scales, void* stream) {
    if (rows < 0 || K <= 0 || K % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!v || !codes || !scales)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(v) || !aligned16(codes) || !aligned4(scales)) return MOE_ERR_INVALID_ARG;
    const hipError_t e = launch_block128_rows(static_cast<const uint16_t*>(v), rows, K, codes, scales, false, nullptr,
                                              static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t moe_product_workspace_bytes(const moe_product_config_t* c) {
    return product_check(c) == MOE_OK ? room_of(*c).bytes : 0;
}

moe_status_t moe_product_prepare_weights(const moe_product_config_t* c, const void* w, uint8_t* w_q, float* w_s, void* stream) {
    const moe_status_t st = product_check(c);
    if (st != MOE_OK) return st;
    if (!w || !w_q || !w_s || !aligned16(w) || !aligned16(w_q) || !aligned4(w_s)) return MOE_ERR_INVALID_ARG;
    const Block128Pair g{{block128(w, w_q, w_s, c->E, c->N, c->K)}};
    return launch_block128_pack(g, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status_t moe_product_expand_weights(const moe_product_config_t* c, const uint8_t* w_q, const float* w_s, void* w, void* stream) {
    const moe_status_t st = product_check(c);
    if (st != MOE_OK) return st;
    if (!w || !w_q || !w_s || !aligned16(w) || !aligned16(w_q) || !aligned4(w_s)) return MOE_ERR_INVALID_ARG;
    const Block128Pair g{{block128(w, w_q, w_s, c->E, c->N, c->K)}};
    return launch_block128_expand(g, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status_t moe_product_forward(const moe_product_config_t* c, const void* x, const int32_t* m_indptr, const uint8_t* w_q,
                                 const float* w_s, void* y, int32_t* status, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    const moe_status_t st = product_check(c);
    if (st != MOE_OK) return st;
    if (c->R == 0) return MOE_OK;
    if (!x || !w_q || !w_s || !y || (!m_indptr && c->E != 1)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w_q) || !aligned4(w_s) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    const Room r = room_of(*c);
    if (!workspace || workspace_bytes < r.bytes) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* q = reinterpret_cast<uint8_t*>(ws + r.q);
    float* qs = reinterpret_cast<float*>(ws + r.qs);
    if (block128_few_rows(c->R, c->E)) {
        Block128RowsArgs g{};
        g.E = c->E; g.N = c->N; g.K = c->K; g.R = c->R;
        g.m_indptr = m_indptr; g.status = status;
        g.x = static_cast<const uint16_t*>(x); g.w = w_q; g.ws = w_s; g.y = static_cast<uint16_t*>(y);
        g.xq = q; g.xs = qs; g.groups = ws + r.groups;
        return launch_block128_few_rows(g, device_cus(), s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
    }
    if (launch_block128_rows(static_cast<const uint16_t*>(x), c->R, c->K, q, qs, true, m_indptr ? m_indptr + c->E : nullptr,
                             s) != hipSuccess)
        return MOE_ERR_HIP;
    Block128GemmArgs g{};
    g.E = c->E; g.K = c->K; g.Np = c->N; g.R = c->R;
    g.m_indptr = m_indptr; g.check = m_indptr != nullptr; g.status = status;
    g.pq = w_q; g.ps = w_s; g.qq = q; g.qs = qs;
    g.out = static_cast<uint16_t*>(y);
    return launch_gemm_block128(B128_PLAIN, g, device_cus(), s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status_t moe_product_backward(const moe_product_config_t* c, const void* dy, const void* x, const int32_t* m_indptr,
                                  const uint8_t* w_q, const float* w_s, void* dx, void* dw, int32_t* status, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    const moe_status_t st = product_check(c);
    if (st != MOE_OK) return st;
    if (!c->training) return MOE_ERR_STATE;
    if (c->R == 0 && !dw) return MOE_OK;                 // dx is empty (so that its pointer may be null)
    if (!dx && !dw) return MOE_ERR_INVALID_ARG;
    if (c->R > 0 && (!dy || (dw && !x) || (dx && (!w_q || !w_s)) || (!m_indptr && c->E != 1))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(w_q) || !aligned4(w_s) || !aligned16(dx) || !aligned16(dw))
        return MOE_ERR_INVALID_ARG;
    const Room r = room_of(*c);
    if (!workspace || workspace_bytes < r.bytes) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int cus = device_cus();
    auto codes = [&](size_t off) { return reinterpret_cast<uint8_t*>(ws + off); };
    auto scales = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    // no rows: every matrix' segment is empty, whatever m_indptr holds
    const int E = c->E, R = c->R;
    int32_t* starts = reinterpret_cast<int32_t*>(ws + r.starts);
    const Segments seg{m_indptr, starts, status, E, R};
    if (R == 0) {
        if (launch_fill_i32(starts, E + 1, 0, s) != hipSuccess) return MOE_ERR_HIP;
    } else if (!dx && launch_segments(seg, s) != hipSuccess) {
        return MOE_ERR_HIP;
    }
    if (dx && R > 0) {
        // dx = dy W: the matrices transposed, dy quantized along N
        if (launch_block128_transpose(w_q, w_s, E, c->N, c->K, codes(r.wt), scales(r.wts), seg, s) != hipSuccess)
            return MOE_ERR_HIP;
        if (dw) {                                        // with dy along the rows, for dw, from the same reads
            const RowsColumnsArgs both{static_cast<const uint16_t*>(dy), starts, R, E, c->N, codes(r.tq), codes(r.tqs),
                                       codes(r.q), scales(r.qs)};
            if (launch_rows_and_columns(both, s) != hipSuccess) return MOE_ERR_HIP;
        } else if (launch_block128_rows(static_cast<const uint16_t*>(dy), R, c->N, codes(r.q), scales(r.qs), true, starts + E,
                                        s) != hipSuccess) {
            return MOE_ERR_HIP;
        }
        Block128GemmArgs g{};
        g.E = E; g.K = c->N; g.Np = c->K; g.R = R;
        g.m_indptr = starts;
        g.pq = codes(r.wt); g.ps = scales(r.wts); g.qq = codes(r.q); g.qs = scales(r.qs);
        g.out = static_cast<uint16_t*>(dx);
        if (launch_gemm_block128(B128_PLAIN, g, cus, s) != hipSuccess) return MOE_ERR_HIP;
    }
    if (dw) {
        // dW_e = sum_r dy[r] x[r]^T: both operands along the rows, in MXFP8
        RowsColumnsArgs t{static_cast<const uint16_t*>(x), starts, R, E, c->K, codes(r.tp), codes(r.tps), nullptr, nullptr};
        if (launch_rows_and_columns(t, s) != hipSuccess) return MOE_ERR_HIP;
        if (!dx || R == 0) {
            t.v = static_cast<const uint16_t*>(dy); t.N = c->N; t.codes = codes(r.tq); t.scales = codes(r.tqs);
            if (launch_rows_and_columns(t, s) != hipSuccess) return MOE_ERR_HIP;
        }
        MxGemmArgs g{};
        g.T = R; g.k = 1; g.E = E; g.m_indptr = starts;
        g.Np = c->K; g.Nq = c->N;
        g.pq = codes(r.tp); g.ps = codes(r.tps); g.qq = codes(r.tq); g.qs = codes(r.tqs);
        g.out = static_cast<uint16_t*>(dw);
        g.accumulate = c->wgrad_accumulate;
        g.pieces = grad_pieces(*c);
        g.part = reinterpret_cast<float*>(ws + r.part);
        if (launch_gemm_mxfp8(MX_WGRAD, g, cus, s) != hipSuccess) return MOE_ERR_HIP;
    }
    return MOE_OK;
}

}  // extern "C"
