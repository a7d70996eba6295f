// The dual GEMM's epilogue with bias, activation, gate and residual, on one
// wave's part of an output tile held in its accumulators:
//     Y = r + g act(v + b)
// v the fp32 sum, b and g one value per column (g per modulation row), r one
// per element.
//
// The accumulators hold Y^T pieces: register 4 q + c of acc[i][j] in lane
// (l32, h) is row 32 i + l32, column 32 j + 8 q + 4 h + c of the part (128
// rows, 32 JB columns).  Both forms pass through the wave's own 8 JB / 2 KB of
// LDS, so that memory is read and written in whole row pieces:
//  - bias and activation only, bf16 out: applied on the accumulators, rounded,
//    then staged as bf16, 64 rows at a time;
//  - otherwise the fp32 sums are staged, 32 rows at a time, and everything else
//    happens on the way out, where a lane has 8 consecutive columns of a row:
//    b and g are then 8 registers each for the whole tile and r is one 16- or
//    32-byte piece per row, loaded one pass ahead.
// Bound: the pieces' way to and from memory after the tile's last product,
// which the one workgroup of a CU does not hide.  32760 tokens: 5120 -> 13824
// with bias and GELU 1150-1210 us against 1060-1130 us for the product with
// nothing behind it; 13824 -> 5120 with gate and f32 residual and output (1.34
// GB, 264 us at a copy's rate) 1180-1210 us against 1015-1045 us.  Storing from
// the accumulators instead, in pieces of 4 columns, took 2.2 ms; staging the
// first form in fp32 too is 3 % slower.
#pragma once
#include <type_traits>

#include "mg_block.h"
#include "mg_device.h"

namespace mg {

typedef uint32_t ep_u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t ep_u32x2 __attribute__((ext_vector_type(2)));
typedef float ep_f32x4 __attribute__((ext_vector_type(4)));
typedef float ep_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 ep_bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kEpNowhere = 0xC0000000u;   // a buffer offset past every range: reads 0, stores nothing

__device__ __forceinline__ uint32_t ep_pack(float lo, float hi) {
    const ep_f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, ep_bf16x2));
}

// act(v) of one fp32 sum
template <int ACT>
__device__ __forceinline__ float ep_act(float v) {
    if constexpr (ACT == MG_ACT_GELU_TANH) return gelu_f32(v);
    if constexpr (ACT == MG_ACT_SILU)
        return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
    return v;
}

// f(integral_constant<int, act>)
template <typename F>
__host__ __device__ __forceinline__ void ep_by_act(int act, F&& f) {
    if (act == MG_ACT_GELU_TANH) f(std::integral_constant<int, MG_ACT_GELU_TANH>{});
    else if (act == MG_ACT_SILU) f(std::integral_constant<int, MG_ACT_SILU>{});
    else f(std::integral_constant<int, MG_ACT_NONE>{});
}

// N (4 or 8) consecutive elements of type dtype at byte `off` of a buffer, as f32.
template <int N>
__device__ __forceinline__ void ep_load(__amdgpu_buffer_rsrc_t r, uint32_t off, bool f32, float (&v)[N]) {
    if (f32) {
#pragma unroll
        for (int p = 0; p < N / 4; ++p) {
            const ep_u32x4 w = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16u * p, 0, 0));
#pragma unroll
            for (int c = 0; c < 4; ++c) v[4 * p + c] = __uint_as_float(w[c]);
        }
    } else if constexpr (N == 8) {
        const ep_u32x4 w = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = __uint_as_float(c & 1 ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
    } else {
        const ep_u32x2 w = __builtin_bit_cast(ep_u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = __uint_as_float(c & 1 ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
    }
}

// 4 or 8 consecutive elements from a place aligned to them on.
__device__ __forceinline__ void ep_load4(const void* p, int64_t at, bool f32, float (&v)[4]) {
    if (f32) {
        const ep_f32x4 a = *reinterpret_cast<const ep_f32x4*>(static_cast<const float*>(p) + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = a[c];
    } else {
        const ep_u32x2 w = *reinterpret_cast<const ep_u32x2*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = __uint_as_float(c & 1 ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
    }
}

__device__ __forceinline__ void ep_load8(const void* p, int64_t at, bool f32, float (&v)[8]) {
    if (f32) {
        const ep_f32x4* x = reinterpret_cast<const ep_f32x4*>(static_cast<const float*>(p) + at);
        const ep_f32x4 a = x[0], b = x[1];
#pragma unroll
        for (int c = 0; c < 4; ++c) { v[c] = a[c]; v[4 + c] = b[c]; }
    } else {
        const ep_u32x4 w = *reinterpret_cast<const ep_u32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = __uint_as_float(c & 1 ? w[c >> 1] & 0xFFFF0000u : w[c >> 1] << 16);
    }
}

// Bias and activation into bf16.  (m0, n0): the part's first row and column;
// rY covers the tile's rows of Y from row m0 - mt0 on (byte range rows * 2 N).
template <int ACT, int JB, typename ACC>
__device__ __forceinline__ void ep_bias_act_bf16(const EpArgs& e, __amdgpu_buffer_rsrc_t rY, ACC& acc, uint32_t mt0,
                                                 int n0, int N, uint8_t* wbuf, uint32_t lane) {
    constexpr uint32_t CH = 4 * JB, RBY = 64 * JB;                // 16-byte chunks and bytes per staged row
    const uint32_t l32 = lane & 31u, h = lane >> 5, rl = lane / CH, cl = lane & (CH - 1);
    const bool bf32 = e.bias_dtype == MG_F32;
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(e.bias, e.bias ? (uint64_t)N * (bf32 ? 4 : 2) : 0);
    float b[JB][4][4];
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            ep_load<4>(rB, (uint32_t)(n0 + 32 * j + 8 * q + 4 * (int)h) * (bf32 ? 4u : 2u), bf32, b[j][q]);
    const int gcol = n0 + (int)cl * 8;
    const uint32_t rowY = 2u * (uint32_t)N;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int ii = 0; ii < 2; ++ii) {
            const int i = 2 * p + ii;
#pragma unroll
            for (int j = 0; j < JB; ++j) asm volatile("" : "+a"(acc[i][j]));    // read here, not earlier
            const uint32_t r = (uint32_t)(32 * ii) + l32;
            const uint32_t rb = r * RBY + h * 8, rs = r & (CH - 1);
#pragma unroll
            for (int j = 0; j < JB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = ep_act<ACT>(acc[i][j][4 * q + c] + b[j][q][c]);
                    *reinterpret_cast<ep_u32x2*>(wbuf + rb + ((((uint32_t)(4 * j + q)) ^ rs) << 4)) =
                        ep_u32x2{ep_pack(v[0], v[1]), ep_pack(v[2], v[3])};
                }
        }
#pragma unroll
        for (int s0 = 0; s0 < (int)CH; s0 += 4) {
            ep_u32x4 v[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t rr = (uint32_t)(64 / CH * (s0 + s)) + rl;
                v[s] = *reinterpret_cast<const ep_u32x4*>(wbuf + rr * RBY + ((cl ^ (rr & (CH - 1))) << 4));
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t rr = (uint32_t)(64 / CH * (s0 + s)) + rl;
                const uint32_t off = gcol < N ? (mt0 + 64u * p + rr) * rowY + 2u * (uint32_t)gcol : kEpNowhere;
                __builtin_amdgcn_raw_buffer_store_b128(v[s], rY, off, 0, 2);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Everything, into bf16 or f32 (YT uint16_t or float), with an f32 residual
// (RF32) or a bf16 one or none.
template <typename YT, int ACT, bool RF32, int JB, typename ACC>
__device__ __forceinline__ void ep_full(const EpArgs& e, __amdgpu_buffer_rsrc_t rY, ACC& acc, int64_t tile_m0,
                                        uint32_t mt0, int n0, int64_t M, int N, uint8_t* wbuf, uint32_t lane) {
    constexpr bool YF = std::is_same_v<YT, float>;
    constexpr uint32_t CH = 8 * JB, RBY = 128 * JB;               // chunks and bytes per staged fp32 row
    constexpr uint32_t LR = CH / 2, RS = 64 / LR, ST = 32 / RS;   // lanes per row, rows per step, steps per pass
    const uint32_t l32 = lane & 31u, h = lane >> 5, rl = lane / LR, cl = lane & (LR - 1);
    const int gcol = n0 + (int)cl * 8;
    const bool col_ok = gcol < N;
    const bool bf32 = e.bias_dtype == MG_F32, gf32 = e.mod.dtype == MG_F32;
    const int64_t left = M - tile_m0;
    const uint32_t nrow = (uint32_t)(left < 256 ? left : 256);
    float b[8] = {}, g[8] = {1, 1, 1, 1, 1, 1, 1, 1};
    if (e.bias)
        ep_load<8>(make_rsrc(e.bias, (uint64_t)N * (bf32 ? 4 : 2)), (uint32_t)gcol * (bf32 ? 4u : 2u), bf32, b);
    // one modulation row for the whole tile, or one per row
    const uint32_t gs = gf32 ? 4u : 2u;
    const int i0 = (int)((uint32_t)tile_m0 / e.mod.group);
    const bool one = e.mod.index == nullptr && (int)(((uint32_t)tile_m0 + nrow - 1u) / e.mod.group) == i0;
    auto gate_rsrc = [&](int64_t i) {
        return make_rsrc(static_cast<const uint8_t*>(e.mod.gate) + i * e.mod.ld * gs, e.mod.gate ? (uint64_t)N * gs : 0);
    };
    if (one && e.mod.gate) ep_load<8>(gate_rsrc(i0), (uint32_t)gcol * gs, gf32, g);
    // the tile's rows of the residual; out of range (no residual, rows past M) reads 0
    const uint32_t rs = RF32 ? 4u : 2u, rowR = (uint32_t)e.ldr * rs;
    const __amdgpu_buffer_rsrc_t rR = make_rsrc(static_cast<const uint8_t*>(e.residual) + tile_m0 * (int64_t)rowR,
                                                e.residual ? (uint64_t)(nrow - 1u) * rowR + (uint64_t)N * rs : 0);
    ep_u32x4 res[ST][RF32 ? 2 : 1];               // the residual of each step, loaded one pass ahead
    const uint32_t offR = col_ok ? (mt0 + rl) * rowR + (uint32_t)gcol * rs : kEpNowhere;
    auto load_res = [&](int p, int s) {
        const uint32_t off = offR + (32u * p + RS * s) * rowR;      // kEpNowhere plus a tile stays out of range
        res[s][0] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(rR, off, 0, 2));
        if constexpr (RF32) res[s][1] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(rR, off + 16u, 0, 2));
    };
    if (e.residual) {
#pragma unroll
        for (int s = 0; s < (int)ST; ++s) load_res(0, s);
    }
    const uint32_t rowY = (YF ? 4u : 2u) * (uint32_t)N;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        int mis[ST] = {};              // modulation rows of the pass's rows, where they differ
        if (!one) {
#pragma unroll
            for (int s = 0; s < (int)ST; ++s) {
                const uint32_t mt = mt0 + 32u * p + RS * s + rl;
                mis[s] = mt < nrow ? mod_row(e.mod, tile_m0 + mt) : -1;
            }
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) asm volatile("" : "+a"(acc[p][j]));
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<ep_f32x4*>(wbuf + l32 * RBY + (((uint32_t)(8 * j + 2 * q) + h) ^ (l32 & (CH - 1))) * 16u) =
                    ep_f32x4{acc[p][j][4 * q], acc[p][j][4 * q + 1], acc[p][j][4 * q + 2], acc[p][j][4 * q + 3]};
#pragma unroll
        for (int s = 0; s < (int)ST; ++s) {
            const uint32_t rr = RS * s + rl, mt = mt0 + 32u * p + rr;
            float v[8];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const ep_f32x4 w = *reinterpret_cast<const ep_f32x4*>(wbuf + rr * RBY + ((2u * cl + c) ^ (rr & (CH - 1))) * 16u);
#pragma unroll
                for (int d = 0; d < 4; ++d) v[4 * c + d] = w[d] + b[4 * c + d];
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = ep_act<ACT>(v[c]);
            float r[8] = {};
            if (e.residual) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const ep_u32x4* x = res[s];
                    if constexpr (RF32) r[c] = __uint_as_float(x[c >> 2][c & 3]);
                    else r[c] = __uint_as_float(c & 1 ? x[0][c >> 1] & 0xFFFF0000u : x[0][c >> 1] << 16);
                }
                if (p < 3) load_res(p + 1, s);
            }
            if (one) {
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = __builtin_fmaf(g[c], v[c], r[c]);
            } else {
                const int mi = mis[s];
                float gr[8] = {1, 1, 1, 1, 1, 1, 1, 1};
                if (e.mod.gate && col_ok && mi >= 0) ep_load8(e.mod.gate, (int64_t)mi * e.mod.ld + gcol, gf32, gr);
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = mi < 0 ? r[c] : __builtin_fmaf(gr[c], v[c], r[c]);
            }
            const uint32_t off = col_ok ? mt * rowY + (YF ? 4u : 2u) * (uint32_t)gcol : kEpNowhere;
            if constexpr (YF) {
                ep_u32x4 w[2];
#pragma unroll
                for (int c = 0; c < 8; ++c) w[c >> 2][c & 3] = __float_as_uint(v[c]);
                __builtin_amdgcn_raw_buffer_store_b128(w[0], rY, off, 0, 2);
                __builtin_amdgcn_raw_buffer_store_b128(w[1], rY, off + 16u, 0, 2);
            } else {
                const ep_u32x4 w = {ep_pack(v[0], v[1]), ep_pack(v[2], v[3]), ep_pack(v[4], v[5]), ep_pack(v[6], v[7])};
                __builtin_amdgcn_raw_buffer_store_b128(w, rY, off, 0, 2);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace mg
