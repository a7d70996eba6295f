// C entries of the operators around the block: host-side validation and
// dispatch.
#include <math.h>

#include "mg_block.h"
#include "mg_internal.h"

namespace {

using namespace mg;

int hip_status(hipError_t h, const char* where) {
    return h == hipSuccess ? MG_OK : fail_msg(MG_ERR_HIP, "%s: %s", where, hipGetErrorString(h));
}

constexpr int64_t kMaxEpRow = (1 << 20) - 256;   // 256 rows of 4-byte elements stay below 1 GiB

size_t elem_size(int32_t dtype) { return dtype == MG_F32 ? 4 : 2; }

// A pointer to elements of `dtype` (already checked): not null, aligned to them.
int check_elems(const void* p, int32_t dtype, const char* name) {
    if (p == nullptr) return fail_msg(MG_ERR_ARG, "%s: null pointer", name);
    if (reinterpret_cast<uintptr_t>(p) % elem_size(dtype)) return fail_msg(MG_ERR_ALIGN, "%s: not aligned to its elements", name);
    return MG_OK;
}

// M rows of `width` elements of `dtype`, ld elements apart
int check_rows(const void* p, int32_t dtype, int64_t ld, int32_t width, const char* name) {
    if (int e = check_dtype(dtype)) return e;
    if (ld < width) return fail_msg(MG_ERR_SHAPE, "%s: ld=%lld is below the width %d", name, (long long)ld, width);
    return check_elems(p, dtype, name);
}

int check_width(int64_t M, int32_t K) {
    if (M < 0) return fail_msg(MG_ERR_SHAPE, "M=%lld must be >= 0", (long long)M);
    if (M > 0x7FFFFFFFll) return fail_msg(MG_ERR_UNSUPPORTED, "M=%lld exceeds 2^31 - 1 rows", (long long)M);
    if (K <= 0) return fail_msg(MG_ERR_SHAPE, "K=%d must be positive", K);
    if (K > kMaxK) return fail_msg(MG_ERR_UNSUPPORTED, "K=%d exceeds %d", K, kMaxK);
    return MG_OK;
}

int take_norm(const mg_norm* n, const char* name, NormArgs* out) {
    *out = NormArgs{};
    if (n == nullptr) return fail_msg(MG_ERR_ARG, "%s: null", name);
    if (n->kind != MG_NORM_LAYER && n->kind != MG_NORM_RMS)
        return fail_msg(MG_ERR_ARG, "%s: kind %d is not MG_NORM_LAYER/MG_NORM_RMS", name, n->kind);
    if (!(n->eps >= 0.0 && isfinite(n->eps))) return fail_msg(MG_ERR_ARG, "%s: eps=%g must be >= 0", name, n->eps);
    if (n->weight || n->bias) {
        if (int e = check_dtype(n->dtype)) return e;
        if (n->weight)
            if (int e = check_elems(n->weight, n->dtype, "norm weight")) return e;
        if (n->bias)
            if (int e = check_elems(n->bias, n->dtype, "norm bias")) return e;
    }
    *out = NormArgs{n->weight, n->bias, n->weight || n->bias ? n->dtype : MG_F32, n->kind, (float)n->eps};
    return MG_OK;
}

// m may be null; with `gate`, only its gate is taken, else scale and shift
int take_mod(const mg_mod* m, int64_t M, int32_t width, bool gate, ModArgs* out) {
    *out = ModArgs{};
    out->group = 0x7FFFFFFFu;         // every row uses modulation row 0
    out->rows = 1;
    out->dtype = MG_F32;
    if (m == nullptr) return MG_OK;
    const void* scale = gate ? nullptr : m->scale;
    const void* shift = gate ? nullptr : m->shift;
    const void* g = gate ? m->gate : nullptr;
    if (m->rows <= 0) return fail_msg(MG_ERR_SHAPE, "modulation: rows=%d must be positive", m->rows);
    if (scale || shift || g) {
        if (int e = check_dtype(m->dtype)) return e;
        if (m->ld < width && m->rows > 1)
            return fail_msg(MG_ERR_SHAPE, "modulation: ld=%lld is below the width %d", (long long)m->ld, width);
        if (scale)
            if (int e = check_elems(scale, m->dtype, "modulation scale")) return e;
        if (shift)
            if (int e = check_elems(shift, m->dtype, "modulation shift")) return e;
        if (g)
            if (int e = check_elems(g, m->dtype, "modulation gate")) return e;
        out->dtype = m->dtype;
    }
    if (m->index) {
        if (reinterpret_cast<uintptr_t>(m->index) & 3u) return fail_msg(MG_ERR_ALIGN, "modulation index: not aligned");
    } else {
        if (m->group <= 0) return fail_msg(MG_ERR_SHAPE, "modulation: group=%lld must be positive", (long long)m->group);
        if (M > 0 && (M - 1) / m->group >= m->rows)
            return fail_msg(MG_ERR_SHAPE, "modulation: %lld rows of groups of %lld need more than %d modulation rows",
                            (long long)M, (long long)m->group, m->rows);
        out->group = m->group < 0x7FFFFFFFll ? (uint32_t)m->group : 0x7FFFFFFFu;
    }
    out->scale = scale;
    out->shift = shift;
    out->gate = g;
    out->index = m->index;
    out->ld = m->ld;
    out->rows = m->rows;
    return MG_OK;
}

// The GEMM epilogue reads whole 16-byte pieces.
int take_epilogue(const mg_epilogue* e, int64_t M, int32_t N, EpArgs* out) {
    *out = EpArgs{};
    if (int c = take_mod(e ? e->mod : nullptr, M, N, true, &out->mod)) return c;
    if (e == nullptr) return MG_OK;
    if (e->reserved != 0) return fail_msg(MG_ERR_ARG, "mg_epilogue.reserved must be 0");
    if (e->act != MG_ACT_NONE && e->act != MG_ACT_GELU_TANH && e->act != MG_ACT_SILU)
        return fail_msg(MG_ERR_ARG, "act %d is not MG_ACT_NONE/MG_ACT_GELU_TANH/MG_ACT_SILU", e->act);
    if (e->bias) {
        if (int c = check_dtype(e->bias_dtype)) return c;
        MG_CHECK_PTR(e->bias, "epilogue bias");
    }
    if (e->residual) {
        if (int c = check_rows(e->residual, e->residual_dtype, e->ldr, N, "epilogue residual")) return c;
        MG_CHECK_PTR(e->residual, "epilogue residual");
        if (e->ldr % 8) return fail_msg(MG_ERR_ALIGN, "epilogue residual: ldr=%lld is not a multiple of 8", (long long)e->ldr);
    }
    if (out->mod.gate) {
        MG_CHECK_PTR(out->mod.gate, "epilogue gate");
        if (out->mod.ld % 8 && out->mod.rows > 1)
            return fail_msg(MG_ERR_ALIGN, "epilogue gate: ld=%lld is not a multiple of 8", (long long)out->mod.ld);
    }
    out->bias = e->bias;
    out->bias_dtype = e->bias ? e->bias_dtype : MG_F32;
    out->residual = e->residual;
    out->residual_dtype = e->residual ? e->residual_dtype : MG_F32;
    out->ldr = e->ldr;
    out->act = e->act;
    out->gated = out->mod.gate != nullptr || out->mod.index != nullptr;
    return MG_OK;
}

int check_gemm_ep(const mg_plan* p, const mg_act* a, int64_t M, const mg_epilogue* e, const void* Y, int32_t y_dtype,
                  EpArgs* out) {
    if (int c = check_plan(p, true)) return c;
    if (int c = check_dtype(y_dtype)) return c;
    if (M < 0) return fail_msg(MG_ERR_SHAPE, "M=%lld must be >= 0", (long long)M);
    if (int c = take_epilogue(e, M, p->d.N, out)) return c;
    if (M == 0) return MG_OK;
    if (int c = check_act(p, a)) return c;
    if (int c = check_gemm_size(p, M)) return c;
    MG_CHECK_PTR(Y, "Y");
    // a tile's 256 rows of Y and of the residual are addressed with 32-bit offsets
    if ((int64_t)p->d.N > kMaxEpRow || out->ldr > kMaxEpRow)
        return fail_msg(MG_ERR_UNSUPPORTED, "N=%d or ldr=%lld exceeds %lld", p->d.N, (long long)out->ldr,
                        (long long)kMaxEpRow);
    return MG_OK;
}

hipError_t run_gemm_ep(const mg_plan* p, const mg_act* a, int64_t M, const EpArgs& e, void* Y, int32_t y_dtype,
                       hipStream_t stream) {
    const int bytes = (y_dtype == MG_F32 ? 4 : 2) + (e.residual ? (e.residual_dtype == MG_F32 ? 4 : 2) : 0);
    const int tile = few_tile(M, p->d.N, p->d.K, p->d.k, bytes);
    if (tile >= 0)
        return launch_dual_gemm_few(a->Aq, a->As, a->XO, p->Wq, p->Ws, p->WO, M, p->d.N, p->d.K, p->d.k, e, Y, y_dtype,
                                    tile, stream);
    return launch_dual_gemm_ep(a->Aq, a->As, a->XO, p->Wq, p->Ws, p->WO, M, p->d.N, p->d.K, p->d.k, e, Y, y_dtype,
                               stream);
}

}  // namespace

extern "C" {

int mg_norm_mod(const mg_norm* norm, const mg_mod* mod, const void* X, int32_t dtype, int64_t ldx, int64_t M,
                int32_t K, void* H, int32_t h_dtype, int64_t ldh, hipStream_t stream) {
    RowArgs r{};
    if (int e = check_width(M, K)) return e;
    if (int e = take_norm(norm, "norm", &r.norm)) return e;
    if (int e = take_mod(mod, M, K, false, &r.mod)) return e;
    if (int e = take_mod(nullptr, M, K, true, &r.gate)) return e;
    if (int e = check_dtype(dtype)) return e;
    if (int e = check_dtype(h_dtype)) return e;
    if (M == 0) return MG_OK;
    if (int e = check_rows(X, dtype, ldx, K, "X")) return e;
    if (int e = check_rows(H, h_dtype, ldh, K, "H")) return e;
    r.X = X; r.H = H; r.ldx = ldx; r.ldh = ldh; r.M = M; r.K = K;
    r.x_dtype = dtype; r.h_dtype = h_dtype; r.has_norm = 1;
    return hip_status(launch_rows(r, stream), "mg_norm_mod");
}

int mg_residual_norm(const mg_residual* a, int64_t M, int32_t K, hipStream_t stream) {
    RowArgs r{};
    if (a == nullptr) return fail_msg(MG_ERR_ARG, "null mg_residual");
    if (a->reserved != 0) return fail_msg(MG_ERR_ARG, "mg_residual.reserved must be 0");
    if (int e = check_width(M, K)) return e;
    if (int e = take_mod(a->gate, M, K, true, &r.gate)) return e;
    if (int e = take_mod(a->norm ? a->mod : nullptr, M, K, false, &r.mod)) return e;
    if (a->post)
        if (int e = take_norm(a->post, "post norm", &r.post)) return e;
    if (a->norm)
        if (int e = take_norm(a->norm, "norm", &r.norm)) return e;
    if (!a->norm && a->H) return fail_msg(MG_ERR_ARG, "H without a norm");
    if (!a->norm && a->mod) return fail_msg(MG_ERR_ARG, "modulation without a norm");
    if (int e = check_dtype(a->dtype)) return e;
    if (int e = check_dtype(a->y_dtype)) return e;
    if (a->norm)
        if (int e = check_dtype(a->h_dtype)) return e;
    if (M == 0) return MG_OK;
    if (int e = check_rows(a->X, a->dtype, a->ldx, K, "X")) return e;
    if (int e = check_rows(a->Y, a->y_dtype, a->ldy, K, "Y")) return e;
    if (int e = check_rows(a->O, a->dtype, a->ldo, K, "O")) return e;
    if (a->norm)
        if (int e = check_rows(a->H, a->h_dtype, a->ldh, K, "H")) return e;
    r.X = a->X; r.Y = a->Y; r.O = a->O; r.H = a->H;
    r.ldx = a->ldx; r.ldy = a->ldy; r.ldo = a->ldo; r.ldh = a->ldh;
    r.M = M; r.K = K;
    r.x_dtype = a->dtype; r.y_dtype = a->y_dtype; r.h_dtype = a->norm ? a->h_dtype : MG_BF16;
    r.has_post = a->post != nullptr;
    r.has_norm = a->norm != nullptr;
    return hip_status(launch_rows(r, stream), "mg_residual_norm");
}

int mg_norm_quantize_act(const mg_plan* p, const mg_norm* norm, const mg_mod* mod, const void* X, int32_t dtype,
                         int64_t ldx, int64_t M, const mg_act* a, hipStream_t stream) {
    NormQuantArgs q{};
    if (int e = check_plan(p, false)) return e;
    const int32_t K = p->d.K;
    if (int e = check_width(M, K)) return e;
    if (int e = take_norm(norm, "norm", &q.r.norm)) return e;
    if (int e = take_mod(mod, M, K, false, &q.r.mod)) return e;
    if (int e = check_dtype(dtype)) return e;
    if (M == 0) return MG_OK;
    if (int e = check_rows(X, dtype, ldx, K, "X")) return e;
    if (int e = check_act(p, a)) return e;
    q.r.X = X; q.r.ldx = ldx; q.r.M = M; q.r.K = K; q.r.x_dtype = dtype; q.r.has_norm = 1;
    q.r.gate.group = 0x7FFFFFFFu;
    q.s = p->s; q.rcp = p->rcp; q.pos = p->pos; q.O = p->O; q.k = p->d.k;
    q.Aq = a->Aq; q.As = a->As; q.XO = reinterpret_cast<uint8_t*>(a->XO);
    return hip_status(launch_norm_quant(q, stream), "mg_norm_quantize_act");
}

int mg_dual_gemm_ep(const mg_plan* p, const mg_act* a, int64_t M, const mg_epilogue* e, void* Y, int32_t y_dtype,
                    hipStream_t stream) {
    EpArgs ep;
    if (int c = check_gemm_ep(p, a, M, e, Y, y_dtype, &ep)) return c;
    if (M == 0) return MG_OK;
    return hip_status(run_gemm_ep(p, a, M, ep, Y, y_dtype, stream), "mg_dual_gemm_ep");
}

int mg_forward_ep(const mg_plan* p, const void* X, int32_t dtype, int64_t M, const mg_act* a, const mg_epilogue* e,
                  void* Y, int32_t y_dtype, hipStream_t stream) {
    EpArgs ep;
    // every check of both steps before anything is launched
    if (int c = check_gemm_ep(p, a, M, e, Y, y_dtype, &ep)) return c;
    if (int c = check_dtype(dtype)) return c;
    if (M == 0) return MG_OK;
    MG_CHECK_PTR(X, "X");
    if (int c = mg_quantize_act(p, X, dtype, M, a, stream)) return c;
    return hip_status(run_gemm_ep(p, a, M, ep, Y, y_dtype, stream), "mg_forward_ep");
}

}  // extern "C"
