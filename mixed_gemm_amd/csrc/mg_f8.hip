// C entries of the 8-bit block-scaled layers: host-side validation and dispatch.
#include "f8_gemm.h"
#include "mg_f8.h"

namespace {

using namespace mg;

constexpr int64_t kMaxOperand = 0xC0000000ll;    // 32-bit buffer offsets, the upper quarter reads as zero
constexpr int64_t kMaxGrid = 1 << 24;            // workgroups of 256 threads of one launch
constexpr int32_t kMaxCols = 1 << 30;

int hip_status(hipError_t h, const char* where) {
    return h == hipSuccess ? MG_OK : fail_msg(MG_ERR_HIP, "%s: %s", where, hipGetErrorString(h));
}

int check_size(int64_t rows, int32_t cols, const char* name) {
    if (rows < 0) return fail_msg(MG_ERR_SHAPE, "%s: rows=%lld must be >= 0", name, (long long)rows);
    if (rows > 0x7FFFFFFFll) return fail_msg(MG_ERR_UNSUPPORTED, "%s: rows=%lld exceeds 2^31 - 1", name, (long long)rows);
    if (cols <= 0 || cols % 32 != 0) return fail_msg(MG_ERR_SHAPE, "%s: cols=%d must be a positive multiple of 32", name, cols);
    if (cols > kMaxCols) return fail_msg(MG_ERR_UNSUPPORTED, "%s: cols=%d exceeds %d", name, cols, kMaxCols);
    return MG_OK;
}

// x's description and, unless it has no rows, its buffers
int take(const mg_f8* x, const char* name, F8Args* out) {
    *out = F8Args{};
    if (x == nullptr) return fail_msg(MG_ERR_ARG, "%s: null", name);
    if (int e = check_size(x->rows, x->cols, name)) return e;
    if (x->format != MG_E4M3 && x->format != MG_E5M2)
        return fail_msg(MG_ERR_ARG, "%s: format %d is not MG_E4M3/MG_E5M2", name, x->format);
    if (x->rows > 0) {
        MG_CHECK_PTR(x->q, name);
        MG_CHECK_PTR(x->s, name);
    }
    *out = F8Args{x->q, x->s, x->rows, x->cols, x->format};
    return MG_OK;
}

int need_shape(const F8Args& x, int64_t rows, int64_t cols, const char* name) {
    if (x.rows != rows || x.cols != cols)
        return fail_msg(MG_ERR_SHAPE, "%s: [%lld][%d], expected [%lld][%lld]", name, (long long)x.rows, x.cols,
                        (long long)rows, (long long)cols);
    return MG_OK;
}

int need_e4m3(const F8Args& x, const char* name) {
    return x.fmt == MG_E4M3 ? MG_OK : fail_msg(MG_ERR_DTYPE, "%s must be MG_E4M3", name);
}

// M rows of `cols` elements, ld apart
int check_matrix(const void* p, int32_t dtype, int64_t ld, int64_t rows, int32_t cols, const char* name) {
    if (int e = check_dtype(dtype)) return e;
    if (ld < cols && rows > 1) return fail_msg(MG_ERR_SHAPE, "%s: ld=%lld is below the width %d", name, (long long)ld, cols);
    if (p == nullptr) return fail_msg(MG_ERR_ARG, "%s: null pointer", name);
    if (reinterpret_cast<uintptr_t>(p) % (dtype == MG_F32 ? 4 : 2))
        return fail_msg(MG_ERR_ALIGN, "%s: not aligned to its elements", name);
    return MG_OK;
}

int check_grid(int64_t rows, int64_t cols, const char* name) {
    if ((rows + 31) / 32 * f8_windows(cols) >= kMaxGrid)
        return fail_msg(MG_ERR_UNSUPPORTED, "%s: [%lld][%lld] is too large for one call", name, (long long)rows, (long long)cols);
    return MG_OK;
}

int check_operand(const F8Args& x, const char* name) {
    if (f8_q_bytes(x.rows, x.cols) >= kMaxOperand || 4 * f8_s_words(x.rows, x.cols) >= kMaxOperand)
        return fail_msg(MG_ERR_UNSUPPORTED, "%s: [%lld][%d] exceeds 3 GiB", name, (long long)x.rows, x.cols);
    return MG_OK;
}

int check_act_fn(int32_t act) {
    if (act != MG_ACT_NONE && act != MG_ACT_GELU_TANH && act != MG_ACT_SILU)
        return fail_msg(MG_ERR_ARG, "act %d is not MG_ACT_NONE/MG_ACT_GELU_TANH/MG_ACT_SILU", act);
    return MG_OK;
}

// two operands of a product
int check_pair(const F8Args& a, const F8Args& w, const char* an, const char* wn) {
    if (a.cols != w.cols)
        return fail_msg(MG_ERR_SHAPE, "%s has %d columns, %s has %d", an, a.cols, wn, w.cols);
    if (int e = need_e4m3(w, wn)) return e;
    if (w.rows <= 0 || w.rows % 32 != 0 || w.rows > kMaxEpRow)
        return fail_msg(w.rows > kMaxEpRow ? MG_ERR_UNSUPPORTED : MG_ERR_SHAPE,
                        "%s: rows=%lld must be a positive multiple of 32 and at most %lld", wn, (long long)w.rows,
                        (long long)kMaxEpRow);
    if (int e = check_operand(a, an)) return e;
    return check_operand(w, wn);
}

int check_save(int32_t save) {
    return save == 0 || save == 1 ? MG_OK : fail_msg(MG_ERR_ARG, "save %d is not 0 or 1", save);
}

// mg_f8_gemm's arguments; the kernels' and a's format
int check_gemm(const mg_f8* a, const mg_f8* w, const mg_epilogue* e, void* Y, int32_t y_dtype, F8GemmArgs* g, int* fmt) {
    F8Args x, b;
    EpArgs ep;
    *g = F8GemmArgs{};
    if (int c = take(a, "a", &x)) return c;
    if (int c = take(w, "w", &b)) return c;
    if (int c = check_pair(x, b, "a", "w")) return c;
    if (int c = check_dtype(y_dtype)) return c;
    if (int c = take_epilogue(e, x.rows, (int32_t)b.rows, &ep)) return c;
    if (x.fmt != MG_E4M3 && ep.act != MG_ACT_NONE)
        return fail_msg(MG_ERR_UNSUPPORTED, "an activation needs an MG_E4M3 a");
    if (ep.ldr > kMaxEpRow) return fail_msg(MG_ERR_UNSUPPORTED, "ldr=%lld exceeds %lld", (long long)ep.ldr, (long long)kMaxEpRow);
    *fmt = x.fmt;
    if (x.rows == 0) return MG_OK;
    MG_CHECK_PTR(Y, "Y");
    *g = F8GemmArgs{x.q, x.s, b.q, b.s, Y, nullptr, x.rows, (int32_t)b.rows, x.cols, 0, ep};
    return MG_OK;
}

// The gated block's first product: x, w13, h and gu (may be null, sv->q then is)
int check_gated(const mg_f8* x, const mg_f8* w13, int32_t act, const mg_f8* h, const mg_f8* gu, F8Args* a, F8Args* w,
                F8Args* o, F8Args* sv) {
    *sv = F8Args{};
    if (int e = take(x, "x", a)) return e;
    if (int e = take(w13, "w13", w)) return e;
    if (int e = take(h, "h", o)) return e;
    if (int e = check_pair(*a, *w, "x", "w13")) return e;
    if (int e = need_e4m3(*a, "x")) return e;
    if (int e = need_e4m3(*o, "h")) return e;
    if (o->cols > kMaxK) return fail_msg(MG_ERR_UNSUPPORTED, "h: cols=%d exceeds %d", o->cols, kMaxK);
    const int64_t F2 = 2 * (int64_t)f8_pad(o->cols);
    if (int e = need_shape(*o, a->rows, o->cols, "h")) return e;
    if (int e = need_shape(*w, F2, w->cols, "w13")) return e;
    if (gu) {
        if (int e = take(gu, "gu", sv)) return e;
        if (int e = need_e4m3(*sv, "gu")) return e;
        if (int e = need_shape(*sv, a->rows, F2, "gu")) return e;
        if (int e = check_operand(*sv, "gu")) return e;
    }
    if (int e = check_act_fn(act)) return e;
    return check_operand(*o, "h");
}

bool fused_up(const F8Args& a, const F8Args& o, const F8Args& sv) {
    return gated_fused(a.rows, o.cols, a.cols, sv.q ? kGatedSave : kGatedForward);
}

int run_gated(const F8Args& a, const F8Args& w, int32_t act, const F8Args& o, const F8Args& sv, void* scratch,
              hipStream_t stream, const char* where) {
    if (fused_up(a, o, sv)) return hip_status(launch_gated_fused(a, w, act, o, sv, stream), where);
    const F8GemmArgs g{a.q, a.s, w.q, w.s, scratch, nullptr, a.rows, (int32_t)w.rows, a.cols, 0, no_epilogue()};
    if (int e = hip_status(launch_f8_gemm(g, a.fmt, MG_F32, stream), where)) return e;
    return hip_status(launch_gated_act(static_cast<const float*>(scratch), a.rows, o.cols, act, o, sv, stream), where);
}

}  // namespace

extern "C" {

int mg_f8_bytes(int64_t rows, int32_t cols, size_t out[2]) {
    if (out == nullptr) return fail_msg(MG_ERR_ARG, "out: null pointer");
    if (int e = check_size(rows, cols, "mg_f8_bytes")) return e;
    out[0] = (size_t)f8_q_bytes(rows, cols);
    out[1] = 4 * (size_t)f8_s_words(rows, cols);
    return MG_OK;
}

int mg_f8_quantize(const void* X, int32_t dtype, int64_t ldx, const mg_f8* x, hipStream_t stream) {
    F8Args a;
    if (int e = take(x, "x", &a)) return e;
    if (int e = check_dtype(dtype)) return e;
    if (a.rows == 0) return MG_OK;
    if (int e = check_matrix(X, dtype, ldx, a.rows, a.cols, "X")) return e;
    if (int e = check_grid(a.rows, a.cols, "x")) return e;
    return hip_status(launch_f8_quantize(X, dtype, ldx, a, stream), "mg_f8_quantize");
}

int mg_f8_dequantize(const mg_f8* x, void* X, int32_t dtype, int64_t ldx, hipStream_t stream) {
    F8Args a;
    if (int e = take(x, "x", &a)) return e;
    if (int e = check_dtype(dtype)) return e;
    if (a.rows == 0) return MG_OK;
    if (int e = check_matrix(X, dtype, ldx, a.rows, a.cols, "X")) return e;
    if (int e = check_grid(a.rows, a.cols, "x")) return e;
    return hip_status(launch_f8_dequantize(a, X, dtype, ldx, stream), "mg_f8_dequantize");
}

int mg_f8_transpose(const mg_f8* x, const mg_f8* xt, hipStream_t stream) {
    F8Args a, t;
    if (int e = take(x, "x", &a)) return e;
    if (a.rows == 0) return MG_OK;
    if (int e = take(xt, "xt", &t)) return e;
    if (int e = need_shape(t, a.cols, (a.rows + 31) / 32 * 32, "xt")) return e;
    if (t.fmt != a.fmt) return fail_msg(MG_ERR_DTYPE, "xt must have x's format");
    if (int e = check_grid(t.rows, t.cols, "xt")) return e;
    return hip_status(launch_f8_transpose(a, t, stream), "mg_f8_transpose");
}

int mg_f8_prepare_back(const void* dY, int32_t dtype, int64_t ldy, const mg_f8* dy, const mg_f8* dyt, const mg_f8* a,
                       const mg_f8* at, const mg_f8* b, const mg_f8* bt, hipStream_t stream) {
    F8Args x, xt{}, m[2] = {}, t[2] = {};
    const mg_f8* const from[2] = {a, b};
    const mg_f8* const to[2] = {at, bt};
    const char* const names[2][2] = {{"a", "at"}, {"b", "bt"}};
    if (int e = take(dy, "dy", &x)) return e;
    if (int e = check_dtype(dtype)) return e;
    const int64_t up = (x.rows + 31) / 32 * 32;
    for (int i = 0; i < 2; ++i) {
        if ((from[i] == nullptr) != (to[i] == nullptr)) return fail_msg(MG_ERR_ARG, "%s goes with %s", names[i][0], names[i][1]);
        if (from[i] == nullptr) continue;
        if (int e = take(from[i], names[i][0], &m[i])) return e;
        if (int e = need_e4m3(m[i], names[i][0])) return e;
        if (int e = need_shape(m[i], x.rows, m[i].cols, names[i][0])) return e;
        if (x.rows == 0) continue;
        if (int e = take(to[i], names[i][1], &t[i])) return e;
        if (int e = need_e4m3(t[i], names[i][1])) return e;
        if (int e = need_shape(t[i], m[i].cols, up, names[i][1])) return e;
    }
    if (x.rows == 0) return MG_OK;
    if (dyt) {
        if (int e = take(dyt, "dyt", &xt)) return e;
        if (int e = need_shape(xt, x.cols, up, "dyt")) return e;
        if (xt.fmt != x.fmt) return fail_msg(MG_ERR_DTYPE, "dyt must have dy's format");
    }
    if (int e = check_matrix(dY, dtype, ldy, x.rows, x.cols, "dY")) return e;
    if (2 * f8_prep_blocks(x, t[0], t[1]) >= kMaxGrid)             // of 512 threads
        return fail_msg(MG_ERR_UNSUPPORTED, "dy: [%lld][%d] is too large for one call", (long long)x.rows, x.cols);
    return hip_status(launch_f8_prep(dY, dtype, ldy, x, xt, m[0], t[0], m[1], t[1], stream), "mg_f8_prepare_back");
}

int mg_f8_pack_w(const void* W, int32_t dtype, int64_t ldw, const mg_f8* w, const mg_f8* wt, hipStream_t stream) {
    F8Args a, t{};
    if (int e = take(w, "w", &a)) return e;
    if (int e = need_e4m3(a, "w")) return e;
    if (a.rows <= 0 || a.rows % 32) return fail_msg(MG_ERR_SHAPE, "w: rows=%lld must be a positive multiple of 32", (long long)a.rows);
    if (wt) {
        if (int e = take(wt, "wt", &t)) return e;
        if (int e = need_e4m3(t, "wt")) return e;
        if (int e = need_shape(t, a.cols, a.rows, "wt")) return e;
    }
    if (int e = check_matrix(W, dtype, ldw, a.rows, a.cols, "W")) return e;
    if (int e = check_operand(a, "w")) return e;
    return hip_status(launch_f8_pack(W, nullptr, dtype, ldw, (int32_t)a.rows, a.cols, a, t, stream), "mg_f8_pack_w");
}

int mg_f8_gemm(const mg_f8* a, const mg_f8* w, const mg_epilogue* e, void* Y, int32_t y_dtype, hipStream_t stream) {
    F8GemmArgs g;
    int fmt;
    if (int c = check_gemm(a, w, e, Y, y_dtype, &g, &fmt)) return c;
    if (g.M == 0) return MG_OK;
    return hip_status(launch_f8_gemm(g, fmt, y_dtype, stream), "mg_f8_gemm");
}

int mg_f8_forward(const void* X, int32_t dtype, int64_t ldx, const mg_f8* act, int32_t save, const mg_f8* w,
                  const mg_epilogue* e, void* Y, int32_t y_dtype, hipStream_t stream) {
    F8GemmArgs g;
    F8Args x;
    int fmt;
    // every check of both steps before anything is launched
    if (int c = check_gemm(act, w, e, Y, y_dtype, &g, &fmt)) return c;
    if (int c = take(act, "act", &x)) return c;
    if (int c = need_e4m3(x, "act")) return c;
    if (int c = check_save(save)) return c;
    if (int c = check_dtype(dtype)) return c;
    if (g.M == 0) return MG_OK;
    if (int c = check_matrix(X, dtype, ldx, x.rows, x.cols, "X")) return c;
    if (int c = check_grid(x.rows, x.cols, "act")) return c;
    if (!save && f8_direct_pays(g.M, g.K, g.N)) {
        const F8DirectArgs d{X, ldx, g.Wq, g.Ws, Y, (int32_t)g.M, g.N, g.K, 0, 0, g.ep, 0, 0};
        return hip_status(launch_f8_direct(d, dtype, y_dtype, false, stream), "mg_f8_forward");
    }
    if (int c = hip_status(launch_f8_quantize(X, dtype, ldx, x, stream), "mg_f8_forward")) return c;
    return hip_status(launch_f8_gemm(g, fmt, y_dtype, stream), "mg_f8_forward");
}

int mg_gated_pack_w(const void* Wg, const void* Wu, int32_t dtype, int64_t ldw, int32_t F, const mg_f8* w13,
                    const mg_f8* w13t, hipStream_t stream) {
    F8Args a, t{};
    if (F <= 0 || F % 32) return fail_msg(MG_ERR_SHAPE, "F=%d must be a positive multiple of 32", F);
    if (F > kMaxK) return fail_msg(MG_ERR_UNSUPPORTED, "F=%d exceeds %d", F, kMaxK);
    const int32_t Fp = f8_pad(F);
    if (int e = take(w13, "w13", &a)) return e;
    if (int e = need_e4m3(a, "w13")) return e;
    if (int e = need_shape(a, 2 * (int64_t)Fp, a.cols, "w13")) return e;
    if (w13t) {
        if (int e = take(w13t, "w13t", &t)) return e;
        if (int e = need_e4m3(t, "w13t")) return e;
        if (int e = need_shape(t, a.cols, 2 * (int64_t)Fp, "w13t")) return e;
    }
    if (int e = check_matrix(Wg, dtype, ldw, F, a.cols, "Wg")) return e;
    if (int e = check_matrix(Wu, dtype, ldw, F, a.cols, "Wu")) return e;
    if (int e = check_operand(a, "w13")) return e;
    return hip_status(launch_f8_pack(Wg, Wu, dtype, ldw, F, a.cols, a, t, stream), "mg_gated_pack_w");
}

int mg_gated_scratch_bytes(int64_t M, int32_t F, int32_t C, size_t out[2]) {
    if (out == nullptr) return fail_msg(MG_ERR_ARG, "out: null pointer");
    if (int e = check_size(M, F, "F")) return e;
    if (int e = check_size(0, C, "C")) return e;
    if (F > kMaxK) return fail_msg(MG_ERR_UNSUPPORTED, "F=%d exceeds %d", F, kMaxK);
    const bool fused = gated_fused(M, F, C, kGatedForward) && gated_fused(M, F, C, kGatedSave);
    out[0] = fused ? 0 : (size_t)M * 8 * f8_pad(F);
    out[1] = gated_fused(M, F, C, kGatedBack) ? 0 : (size_t)M * 4 * F;
    return MG_OK;
}

int mg_gated_gemm(const mg_f8* x, const mg_f8* w13, int32_t act, const mg_f8* h, const mg_f8* gu, void* scratch,
                  hipStream_t stream) {
    F8Args a, w, o, s;
    if (int e = check_gated(x, w13, act, h, gu, &a, &w, &o, &s)) return e;
    if (a.rows == 0) return MG_OK;
    if (!fused_up(a, o, s)) MG_CHECK_PTR(scratch, "scratch");
    return run_gated(a, w, act, o, s, scratch, stream, "mg_gated_gemm");
}

int mg_gated_forward(const void* X, int32_t dtype, int64_t ldx, const mg_f8* x, const mg_f8* w13, int32_t act,
                     const mg_f8* h, const mg_f8* gu, void* scratch, const mg_f8* wd, const mg_epilogue* e, void* Y,
                     int32_t y_dtype, hipStream_t stream) {
    F8Args a, w, o, s;
    F8GemmArgs g;
    int fmt;
    if (int c = check_gated(x, w13, act, h, gu, &a, &w, &o, &s)) return c;
    if (int c = check_gemm(h, wd, e, Y, y_dtype, &g, &fmt)) return c;
    if (int c = check_dtype(dtype)) return c;
    if (a.rows == 0) return MG_OK;
    if (int c = check_matrix(X, dtype, ldx, a.rows, a.cols, "X")) return c;
    if (int c = check_grid(a.rows, a.cols, "x")) return c;
    if (!fused_up(a, o, s)) MG_CHECK_PTR(scratch, "scratch");
    const char* where = "mg_gated_forward";
    if (gu == nullptr && f8_direct_pays_gated(a.rows, a.cols, o.cols, g.N)) {
        const int32_t M = (int32_t)a.rows, F = o.cols;
        const F8DirectArgs up{X, ldx, w.q, w.s, scratch, M, (int32_t)w.rows, a.cols, F, act, no_epilogue(), 0, 0};
        if (int c = hip_status(launch_f8_direct(up, dtype, MG_F32, true, stream), where)) return c;
        const F8DirectArgs down{scratch, F, g.Wq, g.Ws, Y, M, g.N, F, 0, 0, g.ep, 0, 0};
        return hip_status(launch_f8_direct(down, MG_F32, y_dtype, false, stream), where);
    }
    if (int c = hip_status(launch_f8_quantize(X, dtype, ldx, a, stream), where)) return c;
    if (int c = run_gated(a, w, act, o, s, scratch, stream, where)) return c;
    return hip_status(launch_f8_gemm(g, fmt, y_dtype, stream), where);
}

int mg_gated_gemm_back(const mg_f8* dy, const mg_f8* wdt, const mg_f8* gu, int32_t act, const mg_f8* dgu,
                       const mg_f8* dgut, void* scratch, hipStream_t stream) {
    F8Args a, w, s, o, t{};
    if (int e = take(dy, "dy", &a)) return e;
    if (int e = take(wdt, "wdt", &w)) return e;
    if (int e = take(gu, "gu", &s)) return e;
    if (int e = take(dgu, "dgu", &o)) return e;
    if (int e = check_pair(a, w, "dy", "wdt")) return e;
    if (int e = need_e4m3(s, "gu")) return e;
    if (w.rows > kMaxK) return fail_msg(MG_ERR_UNSUPPORTED, "wdt: rows=%lld exceeds %d", (long long)w.rows, kMaxK);
    const int32_t F = (int32_t)w.rows, Fp = f8_pad(F);
    if (int e = need_shape(s, a.rows, 2 * (int64_t)Fp, "gu")) return e;
    if (int e = need_shape(o, a.rows, 2 * (int64_t)Fp, "dgu")) return e;
    if (o.fmt != a.fmt) return fail_msg(MG_ERR_DTYPE, "dgu must have dy's format");
    if (int e = check_act_fn(act)) return e;
    if (int e = check_operand(s, "gu")) return e;
    if (a.rows == 0) return MG_OK;
    if (dgut) {
        if (int e = take(dgut, "dgut", &t)) return e;
        if (int e = need_shape(t, 2 * (int64_t)Fp, (a.rows + 31) / 32 * 32, "dgut")) return e;
        if (t.fmt != o.fmt) return fail_msg(MG_ERR_DTYPE, "dgut must have dy's format");
        if (int e = check_grid(t.rows, t.cols, "dgut")) return e;
    }
    const char* where = "mg_gated_gemm_back";
    if (gated_fused(a.rows, F, a.cols, kGatedBack)) {
        if (int e = hip_status(launch_gated_back_fused(a, w, s, act, o, stream), where)) return e;
        return dgut ? hip_status(launch_f8_transpose(o, t, stream), where) : MG_OK;
    }
    MG_CHECK_PTR(scratch, "scratch");
    const F8GemmArgs g{a.q, a.s, w.q, w.s, scratch, nullptr, a.rows, F, a.cols, 0, no_epilogue()};
    if (int e = hip_status(launch_f8_gemm(g, a.fmt, MG_F32, stream), where)) return e;
    return hip_status(launch_gated_back(static_cast<const float*>(scratch), a.rows, F, act, s, o, t, stream), where);
}

int mg_gated_gemm_dw(const mg_f8* dgut, const mg_f8* xt, int32_t F, void* dWg, void* dWu, int32_t y_dtype,
                     hipStream_t stream) {
    F8Args a, w;
    if (F <= 0 || F % 32) return fail_msg(MG_ERR_SHAPE, "F=%d must be a positive multiple of 32", F);
    if (F > kMaxK) return fail_msg(MG_ERR_UNSUPPORTED, "F=%d exceeds %d", F, kMaxK);
    if (int e = take(dgut, "dgut", &a)) return e;
    if (int e = take(xt, "xt", &w)) return e;
    if (int e = check_pair(a, w, "dgut", "xt")) return e;
    if (int e = need_shape(a, 2 * (int64_t)f8_pad(F), a.cols, "dgut")) return e;
    if (int e = check_dtype(y_dtype)) return e;
    MG_CHECK_PTR(dWg, "dWg");
    MG_CHECK_PTR(dWu, "dWu");
    const F8GemmArgs g{a.q, a.s, w.q, w.s, dWg, dWu, a.rows, (int32_t)w.rows, a.cols, F, no_epilogue()};
    return hip_status(launch_f8_gemm(g, a.fmt, y_dtype, stream), "mg_gated_gemm_dw");
}

}  // extern "C"
