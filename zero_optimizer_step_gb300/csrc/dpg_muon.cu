// dpg_muon.cu -- the passes around the orthogonalisation (momentum of the
// reduced gradient, weight update) and the C entry points of the
// matrix-orthogonalising step.
//
// Both passes stream every byte once: 2R (or 4R) + 8 + 2 (or 4) bytes per
// element for the momentum, 10 + 2 per view for the update, with a handful of
// binary32 operations, so HBM bounds them.  One 8-element vector per thread in
// small CTAs (no grid-stride loop), as in the fused step: several CTAs at
// different points of their loads and stores keep DRAM busy.
//
// Measured (one GB300, whole calls): momentum of 28.3M elements, R = 8, bf16,
// 736 MB in 105 us (7.0 TB/s); 134M elements, fp32 update, 3758 MB in 529 us
// (7.1 TB/s); 42M elements, R = 4, fp32 gradients, 1090 MB in 149 us (7.3 TB/s).
// Update of 28.3M elements with four views, 510 MB in 76 us (6.7 TB/s); of 134M
// with one, 1610 MB in 230 us (7.0 TB/s).  A plain copy reaches 6.8.  Tiny calls are the host's 10 to 20 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dpg_host.h"
#include "dpg_ortho.h"

namespace dpg {

struct MomentumArgs {
    RsAdamArgs r;        // gradients, R, scale (1/G); the rest unused
    float* momentum;
    void* update;
    float mu, omu;       // mu, 1 - mu
    int32_t nesterov, out_f32;
    int64_t lo, hi;      // element range, multiples of 8
};

template <int RT, int MODE>
__global__ void __launch_bounds__(kChunkThreads) k_muon_momentum(const __grid_constant__ MomentumArgs a) {
    pdl_enter();
    const int64_t i = a.lo + (int64_t(blockIdx.x) * kChunkThreads + threadIdx.x) * kVec;
    if (i >= a.hi) return;
    float s[8], u[8];
    F8 m = ld_state_f8(a.momentum + i);
    reduce_vector<RT, MODE>(a.r, i, s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float g = __fmul_rn(__fmul_rn(s[j], a.r.scale), a.omu);
        m.v[j] = __fadd_rn(__fmul_rn(a.mu, m.v[j]), g);
        u[j] = a.nesterov ? __fadd_rn(g, __fmul_rn(a.mu, m.v[j])) : m.v[j];
    }
    st_f8(a.momentum + i, m);
    if (a.out_f32) {
        F8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x.v[j] = u[j];
        st_f8(static_cast<float*>(a.update) + i, x);
    } else {
        st_u4(static_cast<uint16_t*>(a.update) + i, narrow8(u));
    }
}

struct ApplyArgs {
    const ApplyItem* items;
    const double* scales;   // 2 per parameter
    const uint16_t* ortho;
    const int32_t* status;  // of the orthogonalisation; NULL: none has run
    float* master;
    void* views[DPG_MAX_VIEWS];
    int32_t n_views, rule, decay;
    float lr_wd;
    double lr;
};

__global__ void __launch_bounds__(kChunkThreads) k_muon_apply(const __grid_constant__ ApplyArgs a) {
    static_assert(kApplyChunk == kChunkThreads * kVec, "one vector per thread");
    pdl_enter();
    const ApplyItem it = a.items[blockIdx.x];
    // (an ordinary load, which L1 keeps: every CTA asking L2 for the word cost 1.3 %)
    const int32_t status = a.status ? *a.status : 0;
    const int e = int(threadIdx.x) * kVec;
    if (e >= it.count) return;
    const int64_t i = it.off + e;
    const float lrs = float(a.lr * __ldg(a.scales + 2 * it.param + a.rule));
    float o[8];
    F8 w = ld_state_f8(a.master + i);
    widen8(ld_grad_u4(a.ortho + i), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float x = w.v[j];
        if (a.decay) x = __fsub_rn(x, __fmul_rn(a.lr_wd, x));
        x = __fsub_rn(x, __fmul_rn(lrs, o[j]));
        if (e + j < it.count) w.v[j] = x;   // slots after the parameter are padding
    }
    // o is incomplete: weights and views stay as they are
    if (status != 0) return;
    st_f8(a.master + i, w);
    const uint4 p = narrow8(w.v);
    for (int k = 0; k < a.n_views; ++k) st_u4(static_cast<uint16_t*>(a.views[k]) + i, p);
}

using MomentumKernel = void (*)(MomentumArgs);

template <int MODE>
static MomentumKernel pick_momentum(int R) {
    switch (R) {
        case 1: return k_muon_momentum<1, MODE>;
        case 2: return k_muon_momentum<2, MODE>;
        case 4: return k_muon_momentum<4, MODE>;
        case 8: return k_muon_momentum<8, MODE>;
        default: return k_muon_momentum<0, MODE>;
    }
}

// Each constant in double, rounded once.
static int muon_check(const dpg_muon_hparams* hp, const char* who) {
    if (!hp) return fail(DPG_ERR_INVALID_ARG, "%s: hparams is NULL", who);
    if (!(hp->momentum >= 0.0 && hp->momentum < 1.0))
        return fail(DPG_ERR_INVALID_ARG, "%s: momentum must lie in [0, 1)", who);
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay))
        return fail(DPG_ERR_INVALID_ARG, "%s: lr and weight_decay must be finite", who);
    if (hp->scale_rule != DPG_SCALE_SPECTRAL && hp->scale_rule != DPG_SCALE_RMS)
        return fail(DPG_ERR_INVALID_ARG, "%s: scale_rule %d unknown", who, hp->scale_rule);
    return DPG_OK;
}

static int check_flat(const void* p, int32_t dtype, const char* name, const char* who) {
    if (dtype != DPG_BF16 && dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: dtype %d of %s unknown", who, dtype, name);
    if (!p) return fail(DPG_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
    if (!aligned(p, dtype == DPG_BF16 ? 16 : 32))
        return fail(DPG_ERR_MISALIGNED, "%s: %s misaligned", who, name);
    return DPG_OK;
}

// Checks a momentum call and fills `a`; *grid = 0: nothing to do.
static int momentum_args(Plan& p, const void* const* grads, int32_t grads_dtype,
                         const void* const* last, const int64_t* tokens, int32_t n_counts,
                         const dpg_muon_hparams* hp, float* momentum, void* update,
                         int32_t update_dtype, int32_t b0, int32_t b1, MomentumArgs& a, int* grid,
                         const char* who) {
    *grid = 0;
    if (b0 < 0 || b1 < b0 || b1 > p.n_buckets)
        return fail(DPG_ERR_INVALID_ARG, "%s: bucket range [%d, %d) outside [0, %d]", who, b0, b1,
                    p.n_buckets);
    if (grads_dtype != DPG_BF16 && grads_dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: grads_dtype %d unknown", who, grads_dtype);
    if (last && grads_dtype != DPG_F32)
        return fail(DPG_ERR_INVALID_ARG, "%s: last_micro_bf16 needs fp32 accumulation grads", who);
    int st = muon_check(hp, who);
    if (st != DPG_OK) return st;
    st = token_scale(tokens, n_counts, &a.r.scale);
    if (st != DPG_OK) return st;
    a.lo = p.bucket_offset[size_t(b0)];
    a.hi = p.bucket_offset[size_t(b1)];
    if (a.hi <= a.lo) return DPG_OK;
    st = check_flat(update, update_dtype, "update", who);
    if (st == DPG_OK) st = check_flat(momentum, DPG_F32, "momentum", who);
    if (st != DPG_OK) return st;
    if (!grads) return fail(DPG_ERR_INVALID_ARG, "%s: grads is NULL", who);
    for (int r = 0; r < p.R; ++r) {
        st = check_flat(grads[r], grads_dtype, "a gradient buffer", who);
        if (st == DPG_OK && last) st = check_flat(last[r], DPG_BF16, "a last microbatch", who);
        if (st != DPG_OK) return st;
        a.r.grads[r] = grads[r];
        a.r.last[r] = last ? last[r] : nullptr;
    }
    a.r.R = p.R;
    a.momentum = momentum;
    a.update = update;
    a.mu = float(hp->momentum);
    a.omu = float(1.0 - hp->momentum);
    a.nesterov = hp->nesterov != 0;
    a.out_f32 = update_dtype == DPG_F32;
    return grid_cover(((a.hi - a.lo) / kVec + kChunkThreads - 1) / kChunkThreads, grid, who);
}

static int launch_momentum(const MomentumArgs& a, int grid, int32_t grads_dtype, bool last,
                           cudaStream_t s, const char* who) {
    if (grid == 0) return DPG_OK;
    MomentumKernel k = grads_dtype == DPG_BF16 ? pick_momentum<kInBf16>(a.r.R)
                     : last ? pick_momentum<kInF32PlusBf16>(a.r.R) : pick_momentum<kInF32>(a.r.R);
    return launch_k(k, unsigned(grid), kChunkThreads, s, who, a);
}

static int apply_args(const Matrices& m, const void* ortho, const dpg_muon_hparams* hp, float* master,
                      void* const* views, int32_t n_views, ApplyArgs& a, const char* who) {
    int st = muon_check(hp, who);
    if (st != DPG_OK) return st;
    if (n_views < 0 || n_views > DPG_MAX_VIEWS)
        return fail(DPG_ERR_INVALID_ARG, "%s: n_views %d outside [0, %d]", who, n_views, DPG_MAX_VIEWS);
    if (m.apply_items.empty()) return DPG_OK;
    st = check_flat(ortho, DPG_BF16, "the orthogonalised update", who);
    if (st == DPG_OK) st = check_flat(master, DPG_F32, "master", who);
    if (st != DPG_OK) return st;
    if (n_views > 0 && !views) return fail(DPG_ERR_INVALID_ARG, "%s: param_views is NULL", who);
    for (int k = 0; k < n_views; ++k) {
        st = check_flat(views[k], DPG_BF16, "a parameter view", who);
        if (st != DPG_OK) return st;
        a.views[k] = views[k];
    }
    a.ortho = static_cast<const uint16_t*>(ortho);
    a.master = master;
    a.n_views = n_views;
    a.rule = hp->scale_rule == DPG_SCALE_RMS;
    a.decay = hp->weight_decay != 0.0;
    a.lr_wd = float(hp->lr * hp->weight_decay);
    a.lr = hp->lr;
    return DPG_OK;
}

static int launch_apply(const Matrices& m, ApplyArgs& a, cudaStream_t s, const char* who) {
    if (m.apply_items.empty()) return DPG_OK;
    a.items = m.d_apply_items;
    a.scales = m.d_scales;
    a.status = m.ws ? reinterpret_cast<const int32_t*>(m.ws + m.o_status) : nullptr;
    return launch_k(k_muon_apply, unsigned(m.apply_items.size()), kChunkThreads, s, who, a);
}

}  // namespace dpg

using dpg::fail;

extern "C" {

int dpg_muon_momentum(const dpg_plan_t* plan, const void* const* grads, int32_t grads_dtype,
                      const void* const* last_micro_bf16, const int64_t* valid_tokens,
                      int32_t n_counts, const dpg_muon_hparams* hp, float* momentum, void* update,
                      int32_t update_dtype, int32_t b0, int32_t b1, void* stream) {
    dpg::clear_error();
    const dpg::Trace trace("dpg_muon_momentum");
    if (!plan) return fail(DPG_ERR_INVALID_ARG, "dpg_muon_momentum: plan is NULL");
    dpg::MomentumArgs a{};
    int grid = 0;
    const int st = dpg::momentum_args(const_cast<dpg_plan_t*>(plan)->p, grads, grads_dtype,
                                      last_micro_bf16, valid_tokens, n_counts, hp, momentum, update,
                                      update_dtype, b0, b1, a, &grid, "dpg_muon_momentum");
    if (st != DPG_OK) return st;
    return dpg::launch_momentum(a, grid, grads_dtype, last_micro_bf16 != nullptr,
                                static_cast<cudaStream_t>(stream), "dpg_muon_momentum");
}

int dpg_orthogonalize(dpg_matrices_t* mats, const void* update, int32_t update_dtype,
                      const dpg_muon_hparams* hp, void* ortho_bf16, void* stream) {
    dpg::clear_error();
    const dpg::Trace trace("dpg_orthogonalize");
    if (!mats) return fail(DPG_ERR_INVALID_ARG, "dpg_orthogonalize: mats is NULL");
    dpg::OrthoSchedule sch;
    int st = dpg::ortho_steps(hp, &sch, "dpg_orthogonalize");
    if (st != DPG_OK) return st;
    if (mats->m.n_matrices == 0) return DPG_OK;
    st = dpg::check_flat(update, update_dtype, "update", "dpg_orthogonalize");
    if (st == DPG_OK) st = dpg::check_flat(ortho_bf16, DPG_BF16, "ortho_bf16", "dpg_orthogonalize");
    if (st == DPG_OK) st = dpg::upload_matrices(mats->m, sch.both_steps > 0);
    if (st != DPG_OK) return st;
    return dpg::ortho_launch(mats->m, update, update_dtype, hp, sch, ortho_bf16, stream, "dpg_orthogonalize");
}

int dpg_muon_apply(dpg_matrices_t* mats, const void* ortho_bf16, const dpg_muon_hparams* hp,
                   float* master, void* const* param_views, int32_t n_views, void* stream) {
    dpg::clear_error();
    const dpg::Trace trace("dpg_muon_apply");
    if (!mats) return fail(DPG_ERR_INVALID_ARG, "dpg_muon_apply: mats is NULL");
    dpg::ApplyArgs a{};
    int st = dpg::apply_args(mats->m, ortho_bf16, hp, master, param_views, n_views, a, "dpg_muon_apply");
    if (st != DPG_OK || mats->m.apply_items.empty()) return st;
    st = dpg::upload_for_update(mats->m);
    if (st != DPG_OK) return st;
    return dpg::launch_apply(mats->m, a, static_cast<cudaStream_t>(stream), "dpg_muon_apply");
}

int dpg_muon_step(const dpg_plan_t* plan, dpg_matrices_t* mats, const void* const* grads,
                  int32_t grads_dtype, const void* const* last_micro_bf16,
                  const int64_t* valid_tokens, int32_t n_counts, const dpg_muon_hparams* hp,
                  float* master, float* momentum, void* update, int32_t update_dtype,
                  void* const* param_views, int32_t n_views, void* stream) {
    dpg::clear_error();
    const dpg::Trace trace("dpg_muon_step");
    const char* who = "dpg_muon_step";
    if (!plan || !mats) return fail(DPG_ERR_INVALID_ARG, "%s: plan or mats is NULL", who);
    dpg::Plan& p = const_cast<dpg_plan_t*>(plan)->p;
    dpg::Matrices& m = mats->m;
    if (m.total_padded != p.total_padded || m.param_offset != p.param_offset || m.numels != p.numels)
        return fail(DPG_ERR_INVALID_ARG, "%s: mats were made from another plan", who);
    dpg::OrthoSchedule sch;
    int st = dpg::ortho_steps(hp, &sch, who);
    if (st != DPG_OK) return st;
    dpg::MomentumArgs a{};
    int grid = 0;
    st = dpg::momentum_args(p, grads, grads_dtype, last_micro_bf16, valid_tokens, n_counts, hp, momentum,
                            update, update_dtype, 0, p.n_buckets, a, &grid, who);
    if (st != DPG_OK) return st;
    dpg::ApplyArgs b{};
    st = dpg::apply_args(m, update, hp, master, param_views, n_views, b, who);
    if (st != DPG_OK || m.n_matrices == 0) return st;
    st = dpg::upload_matrices(m, sch.both_steps > 0);
    if (st != DPG_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = dpg::launch_momentum(a, grid, grads_dtype, last_micro_bf16 != nullptr, s, who);
    if (st == DPG_OK) st = dpg::ortho_launch(m, update, update_dtype, hp, sch, update, stream, who);
    if (st == DPG_OK) st = dpg::launch_apply(m, b, s, who);
    return st;
}

}  // extern "C"
