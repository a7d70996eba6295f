// What the 8-bit products share: their arguments, the matrix instruction and
// the choice between the kernels.
#pragma once
#include "mg_f8.h"

namespace mg {

// Y [M][N] = ep(A W^T), A [M][K] codes Aq and scales As, W [N][K].
struct F8GemmArgs {
    const uint8_t* Aq;
    const uint32_t* As;
    const uint8_t* Wq;
    const uint32_t* Ws;
    void* Y;
    void* Y2;             // not null: Y and Y2 [F][N] take runs of 128 of the M rows in turn
    int64_t M;
    int32_t N, K;
    int32_t F;
    EpArgs ep;
    // the gated block's epilogues
    uint8_t* Oq;          // h, or the gradients of gate and up sums
    uint32_t* Os;
    uint8_t* Gq;          // the gate and up sums
    uint32_t* Gs;
};

// The product straight from activations X [M][K] for few rows (up to
// f8_direct_rows(K)): Y = ep(Q(X) W^T), or (gated) the hidden activation act(g)
// u in fp32, Y [M][F], with W [2 Fp][K].
struct F8DirectArgs {
    const void* X;
    int64_t ldx;
    const uint8_t* Wq;
    const uint32_t* Ws;
    void* Y;
    int32_t M, N, K;
    int32_t F, act;
    EpArgs ep;
    int32_t tiles, vec;   // set by the launcher
};
int f8_direct_rows(int32_t K);
// whether a layer, or the gated block, is faster so than with its rows quantized first
bool f8_direct_pays(int64_t M, int32_t K, int32_t N);
bool f8_direct_pays_gated(int64_t M, int32_t K, int32_t F, int32_t N);
hipError_t launch_f8_direct(F8DirectArgs a, int32_t x_dtype, int32_t y_dtype, bool gated, hipStream_t st);

// an epilogue that changes nothing
inline EpArgs no_epilogue() {
    EpArgs e{};
    e.mod.group = 0x7FFFFFFFu;
    e.mod.rows = 1;
    return e;
}

// The product by the kernel that its sizes ask for (fmt: A's).
hipError_t launch_f8_gemm(const F8GemmArgs& a, int fmt, int32_t y_dtype, hipStream_t st);
// The kernel that a product takes, its expected time and that of 256 x 256 tiles (us).
struct F8Choice {
    int tile;
    double time, time256;
};
F8Choice f8_choice(int64_t M, int32_t N, int32_t K, bool f32);
// Whether a product of the gated block (M rows, F hidden channels, C contracted
// columns) runs with the gate in its epilogue; else the fp32 sums pass through
// scratch.
enum { kGatedForward = 0, kGatedSave = 1, kGatedBack = 2 };
bool gated_fused(int64_t M, int32_t F, int32_t C, int what);
hipError_t launch_gated_fused(const F8Args& x, const F8Args& w, int32_t act, const F8Args& h, const F8Args& gu, hipStream_t st);
hipError_t launch_gated_back_fused(const F8Args& dy, const F8Args& wdt, const F8Args& gu, int32_t act, const F8Args& dgu,
                                   hipStream_t st);

hipError_t launch_f8_gemm_256(const F8GemmArgs& a, int fmt, int32_t y_dtype, hipStream_t st);
hipError_t launch_f8_gemm_192(const F8GemmArgs& a, int fmt, hipStream_t st);   // into bf16, without Y2
hipError_t launch_f8_gemm_128(const F8GemmArgs& a, int fmt, int32_t y_dtype, hipStream_t st);
hipError_t launch_f8_gemm_few(const F8GemmArgs& a, int fmt, int32_t y_dtype, int tile, hipStream_t st);

#if defined(__HIPCC__)

typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

// 32 output columns (E4M3 rows of W, whose two slices are w0, w1) by 32 rows of
// A (format FA, slices a0, a1) by 64 of K, scale codes in byte 0 of sw, sa.
// Lane l holds row l % 32 of both and 16 codes of each slice; which half of the
// instruction's K they count as is the same for both.  Register 4 q + c of lane
// l gets A's row l % 32 and W's row 8 q + 4 (l / 32) + c.
template <int FA, typename V>
__device__ __forceinline__ v16f f8_mfma(const V& w0, const V& w1, const V& a0, const V& a1, uint32_t sw, uint32_t sa, v16f c) {
    const v8i wv = {(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]};
    const v8i av = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3], (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, c, 0, FA == MG_E5M2 ? 1 : 0, 0, (int)sw, 0, (int)sa);
}

// The same sums with fp32 precision.  The 8-bit matrix instructions (all of
// them) cut each of eight products off at 2^-13 of the largest before they add
// them; the bf16 ones do not, and a code times its scale is a bf16 value.  So
// results that keep fp32's precision (MG_F32, and sums that are rounded to 8
// bits again: five in a thousand codes of them would come out a step off) are
// formed by bf16 instructions, at half the 8-bit rate, from operands that are
// still read and staged as codes.
//
// The 16 codes of a lane's piece times 2^(c - 127) (s) as two operands of the
// 32x32x16 bf16 instruction.
template <int FMT, typename V>
__device__ __forceinline__ void f8_widen(const V& p, float s, v8bf (&o)[2]) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        v2bf lo, hi;
        if constexpr (FMT == MG_E5M2) {
            lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(p[w], s, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(p[w], s, true);
        } else {
            lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p[w], s, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p[w], s, true);
        }
        o[w >> 1][4 * (w & 1)] = lo[0]; o[w >> 1][4 * (w & 1) + 1] = lo[1];
        o[w >> 1][4 * (w & 1) + 2] = hi[0]; o[w >> 1][4 * (w & 1) + 3] = hi[1];
    }
}
__device__ __forceinline__ v16f f8_mfma_wide(const v8bf (&w)[2], const v8bf (&a)[2], v16f c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[0], a[0], c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[1], a[1], c, 0, 0, 0);
}

#endif

}  // namespace mg
