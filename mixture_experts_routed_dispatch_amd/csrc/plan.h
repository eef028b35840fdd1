// plan.h -- the plan behind moe_plan_t (internal to libmoe's host code).
#pragma once

#include <hip/hip_runtime.h>

#include <vector>

#include "../../include/moe.h"

constexpr size_t kMaxProfileRecords = 4096;
constexpr int kMaxExperts = 256;             // nvfp4moe README, "Limits"

struct moe_plan_s {
    moe_config_t cfg;
    int64_t R;
    bool decode;
    // workspace offsets (bytes)
    size_t off_status, off_m_indptr, off_gather, off_slots, off_probs;
    size_t off_a, off_o, off_h, off_dh, off_dxp, off_xg, off_dys, off_xq, off_xs, off_xsr, off_aq, off_as;
    // MXFP8 backward: dO and (dg, du) quantized along d and 2I (codes, block-major scales), and
    // the weight-gradient operands in the token layout (P and Q codes and scales)
    size_t off_doq, off_dos, off_dhq, off_dhs, off_tp, off_tps, off_tq, off_tqs;
    size_t tp_feat, tq_feat;           // features of the largest P / Q token-layout operand
    int64_t ntok;                      // token-layout rows: T*k + 128 E
    size_t off_part, off_split;        // split weight-gradient tiles: partial sums, descriptors
    size_t off_we;                     // MXFP4 on the grouped-GEMM path: a product's weights as BF16
    size_t a_bytes, o_bytes;           // of the regions of W13 outputs and expert outputs
    size_t off_mega;                   // mega decode: FP32 partial expert outputs [T*k, I / chunk, d]
    size_t ws_bytes;
    char* ws;
    size_t ws_size;
    int num_cu;
    bool have_saved_forward;
    bool h_aliased;                    // recompute_h: h occupies the dxp / xg / dys region
    bool dh_aliased;                   // BF16 training: dh occupies o's region (see below)
    int32_t* status_word;              // device status word of the last call (workspace or static scratch)
    // measurement-only event pairs around kernel stages (moe_profile)
    struct ProfRec { int stage; hipEvent_t a, b; };
    bool prof_on = false;
    std::vector<hipEvent_t> ev_free;
    std::vector<ProfRec> recs;

    template <class T> T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }

    hipEvent_t take_event() {
        hipEvent_t e = nullptr;
        if (!ev_free.empty()) { e = ev_free.back(); ev_free.pop_back(); return e; }
        if (hipEventCreate(&e) != hipSuccess) return nullptr;
        return e;
    }
    // returns a record index, or -1 when not recording
    int stage_begin(int stage, hipStream_t s) {
        if (!prof_on || recs.size() >= kMaxProfileRecords) return -1;
        ProfRec r{stage, take_event(), take_event()};
        if (!r.a || !r.b || hipEventRecord(r.a, s) != hipSuccess) {
            if (r.a) ev_free.push_back(r.a);
            if (r.b) ev_free.push_back(r.b);
            return -1;
        }
        recs.push_back(r);
        return (int)recs.size() - 1;
    }
    void stage_end(int idx, hipStream_t s) {
        if (idx >= 0) (void)hipEventRecord(recs[(size_t)idx].b, s);
    }
    ~moe_plan_s() {
        for (auto& r : recs) { (void)hipEventDestroy(r.a); (void)hipEventDestroy(r.b); }
        for (auto e : ev_free) (void)hipEventDestroy(e);
    }
};
