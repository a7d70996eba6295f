// Kernel-side descriptions and launchers of the operators around the block:
// norm + modulation, gated residual + norm, norm + quantize, and the dual
// GEMM's epilogue.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mixed_gemm.h"

namespace mg {

// mg_mod as the kernels take it (all pointers null: no modulation).
struct ModArgs {
    const void* scale;
    const void* shift;
    const void* gate;
    const int32_t* index;
    int64_t ld;
    uint32_t group;       // clamped to the row count: r / group in 32 bits
    int32_t rows;
    int32_t dtype;
};

// mg_norm as the kernels take it.
struct NormArgs {
    const void* weight;
    const void* bias;
    int32_t dtype;
    int32_t kind;
    float eps;
};

// One pass over rows: O = X + gate post(Y), H = norm_mod(O) (any part absent).
struct RowArgs {
    const void* X;
    const void* Y;        // null: no residual step (H from X)
    void* O;
    void* H;
    int64_t ldx, ldy, ldo, ldh;
    int64_t M;
    int32_t K;
    int32_t x_dtype, y_dtype, h_dtype;
    int32_t has_post, has_norm;
    int32_t apart;        // O and H share no memory with X and Y (set by launch_rows)
    NormArgs post, norm;
    ModArgs gate, mod;
};
hipError_t launch_rows(const RowArgs& a, hipStream_t st);

// Norm + modulation of X rounded to bf16, quantized as the input of a layer.
struct NormQuantArgs {
    RowArgs r;            // X, norm, mod (H, Y, O unused)
    const float* s;
    const float* rcp;
    const int32_t* pos;
    const int32_t* O;
    uint8_t* Aq;
    uint8_t* As;
    uint8_t* XO;
    int32_t k;
};
hipError_t launch_norm_quant(const NormQuantArgs& a, hipStream_t st);

// mg_epilogue as the kernels take it.
struct EpArgs {
    const void* bias;
    const void* residual;
    ModArgs mod;          // gate only
    int64_t ldr;
    int32_t bias_dtype, residual_dtype;
    int32_t act;
    int32_t gated;        // mod.gate or padding rows to look at
};
hipError_t launch_dual_gemm_ep(const uint8_t* Aq, const uint8_t* As, const uint16_t* XO, const uint8_t* Wq,
                               const uint8_t* Ws, const uint16_t* WO, int64_t M, int32_t N, int32_t K, int32_t k,
                               const EpArgs& e, void* Y, int32_t y_dtype, hipStream_t st);
// The same for few rows, with K split over a workgroup's waves, and the tile
// it would take (-1: the 256x256 tiles of launch_dual_gemm_ep are expected to
// be faster).
int few_tile(int64_t M, int32_t N, int32_t K, int32_t k, int bytes);
hipError_t launch_dual_gemm_few(const uint8_t* Aq, const uint8_t* As, const uint16_t* XO, const uint8_t* Wq,
                                const uint8_t* Ws, const uint16_t* WO, int64_t M, int32_t N, int32_t K, int32_t k,
                                const EpArgs& e, void* Y, int32_t y_dtype, int tile, hipStream_t st);

// Modulation row of token row r, or -1 for a padding token.
__device__ __forceinline__ int mod_row(const ModArgs& m, int64_t r) {
    if (m.index == nullptr) return (int)((uint32_t)r / m.group);
    const int i = m.index[r];
    return (uint32_t)i < (uint32_t)m.rows ? i : -1;
}

// Element `at` of an f32 or bf16 array, as f32.
__device__ __forceinline__ float load_elem(const void* p, int64_t at, int32_t dtype) {
    if (dtype == MG_F32) return static_cast<const float*>(p)[at];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16);
}

}  // namespace mg
