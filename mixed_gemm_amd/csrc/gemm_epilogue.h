// The dual GEMM's epilogue with bias, activation, gate and residual (EpOut
// outputs of the tiled kernel).
#pragma once
#include <type_traits>

#include "mg_block.h"
#include "mg_device.h"

namespace mg {

// act(v) of one fp32 sum
__device__ __forceinline__ float ep_act(float v, int act) {
    if (act == MG_ACT_GELU_TANH) return gelu_f32(v);
    if (act == MG_ACT_SILU) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
    return v;
}

// One output value: column col of row `row` (modulation row mi) from its fp32 sum.
template <typename YT>
__device__ __forceinline__ void ep_store1(const EpArgs& e, YT* Y, int64_t row, int N, int col, int mi, float v) {
    if (e.bias) v += load_elem(e.bias, col, e.bias_dtype);
    v = ep_act(v, e.act);
    const float r = e.residual ? load_elem(e.residual, row * e.ldr + col, e.residual_dtype) : 0.0f;
    if (e.mod.gate && mi >= 0) v *= load_elem(e.mod.gate, mi * e.mod.ld + col, e.mod.dtype);
    v = mi >= 0 ? r + v : r;
    if constexpr (std::is_same_v<YT, float>) Y[row * N + col] = v;
    else Y[row * N + col] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// The wave's part of a tile: acc[i][j] register 4 q + c of lane (l32, h) is
// the sum of row m0 + 32 i + l32 and column n0 + 32 j + 8 q + 4 h + c.
template <typename YT, int JB, typename ACC>
__device__ __forceinline__ void ep_store(const EpArgs& e, void* Y, ACC& acc, int64_t m0, int n0, int64_t M, int N,
                                         int l32, int h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = m0 + 32 * i + l32;
        if (row >= M) continue;
        const int mi = mod_row(e.mod, row);
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = n0 + 32 * j + 8 * q + 4 * h;
                if (col < N) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        ep_store1<YT>(e, static_cast<YT*>(Y), row, N, col + c, mi, acc[i][j][4 * q + c]);
                }
            }
    }
}

}  // namespace mg
