// The 8-bit product for a few rows straight from 16- or 32-bit activations: one
// launch in place of the quantize step and the product, whose latencies would
// add up.
//
// Every workgroup quantizes all M rows into LDS (a scale's 128 channels to 16
// lanes, as the quantize step does it, with the same codes) while its first
// weights are on their way, then multiplies them like k_f8_few.hip: NG groups
// of 32 columns per workgroup, the blocks of 128 channels dealt to its waves,
// weights from memory straight into registers, the waves' sums joined in their
// order.
//
// The gated block's first product writes h = act(g) u in fp32: a workgroup has
// the gate and the up rows of the same 32 hidden channels; the second product
// quantizes h on its way in.
//
// Bound: the weights' way from memory.  One row, 5120 -> 13824 (71 MB of codes) 12.2
// us, 5.8 TB/s, part of it out of the last-level cache; the quantize step and the
// few-row kernel take 15.  The gated block of one token (212 MB) 43.2 us, 4.9 TB/s:
// at that size most of the codes come from HBM, and a copy moves 5.1.
#include "gemm_epilogue.h"
#include "f8_gemm.h"

namespace mg {

namespace {

constexpr int kDirRow = 144;                       // bytes of a row's 128 codes in LDS (16 of pad: rows on other banks)

enum { kDirBf16 = 0, kDirF32 = 1, kDirGated = 2 };

template <typename XT, int OUT, int NG, int NW, int D>
__global__ void __launch_bounds__(64 * NW) f8_direct(F8DirectArgs g) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];     // codes, scale codes; then the waves' sums
    constexpr bool WIDE = OUT != kDirBf16;
    constexpr int ROW = 32 * NG + 4;
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = g.K, N = g.N, M = g.M;
    const EpArgs& e = g.ep;
    // column tiles of an XCD (workgroups go round-robin) follow each other
    const int bx = ((int)blockIdx.x & 7) * ((int)gridDim.x >> 3) + ((int)blockIdx.x >> 3);
    if (bx >= g.tiles) return;
    const uint32_t ns = (uint32_t)f8_slices(K);
    const int units = (int)ns / 4;
    const uint32_t nwin = (uint32_t)f8_windows(K);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.Wq, (uint64_t)f8_q_bytes(N, K));
    const __amdgpu_buffer_rsrc_t rBs = make_rsrc(g.Ws, 4 * (uint64_t)f8_s_words(N, K));
    // W's row groups: NG in a row, or the gate and up rows of the tile's 32 channels
    uint32_t offB[NG], offBs[NG];
#pragma unroll
    for (int c = 0; c < NG; ++c) {
        const int grp = OUT == kDirGated ? 8 * (bx >> 2) + 4 * c + (bx & 3) : bx * NG + c;
        const int n = 32 * grp + l32;
        offB[c] = n < N ? (uint32_t)grp * ns * kFragBlock + 16u * (uint32_t)lane : kEpNowhere;
        offBs[c] = n < N ? 4u * (uint32_t)f8_s_at(n, 0, nwin) : kEpNowhere;
    }
    ep_u32x4 w[D][NG][4];
    uint32_t sw[D][NG];
    auto load_w = [&](int u, int d) {
        const bool ok = u < units;
        const uint32_t so = ok ? (uint32_t)(u >> 2) * 1024u + (uint32_t)(u & 3) : 0u;
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            sw[d][c] = __builtin_amdgcn_raw_buffer_load_b8(rBs, ok ? offBs[c] : kEpNowhere, so, 0);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                w[d][c][s] = __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                              rB, ok ? offB[c] : kEpNowhere,
                                                              ok ? (4u * (uint32_t)u + (uint32_t)s) * kFragBlock : 0u, 0));
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load_w(wave + d * NW, d);

    // ---- the rows' codes: (block u, row m) at (u M + m) kDirRow, scale codes behind them
    uint32_t* sc = reinterpret_cast<uint32_t*>(lds + (size_t)units * M * kDirRow);
    {
        const XT* X = static_cast<const XT*>(g.X);
        const int c8 = tid & 15, pairs = units * M;
        const bool vec = g.vec != 0;
        for (int p0 = 0; p0 < pairs; p0 += 4 * NW) {
            const int p = p0 + (tid >> 4);
            const int u = p / M, m = p - u * M, col = 128 * u + 8 * c8;
            const bool on = p < pairs && col < K;
            float v[8];
            if (on) {
                const XT* x = X + (int64_t)m * g.ldx + col;
                if (vec) f8_load8<XT, true>(x, v);
                else f8_load8<XT, false>(x, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.0f;
            }
            uint32_t lo, hi;
            const uint32_t c = f8_encode8<MG_E4M3>(v, on, lo, hi);
            if (p < pairs) {
                uint8_t* q = lds + (size_t)p * kDirRow + (c8 >> 2) * 32 + 4 * (c8 & 3);
                *reinterpret_cast<uint32_t*>(q) = lo;
                *reinterpret_cast<uint32_t*>(q + 16) = hi;
                if (c8 == 0) sc[p] = c;
            }
        }
    }
    __syncthreads();

    v16f acc[NG];
#pragma unroll
    for (int c = 0; c < NG; ++c) acc[c] = v16f{};
    const int mrow = l32 < M ? l32 : M - 1;                           // the other lanes' results are not stored
    auto multiply = [&](int u, int d) {
        const int uc = u < units ? u : units - 1;                     // beyond: the weights are 0
        const uint8_t* q = lds + (size_t)(uc * M + mrow) * kDirRow + 16 * h;
        const uint32_t sa = sc[uc * M + mrow];
        ep_u32x4 a[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) a[s] = *reinterpret_cast<const ep_u32x4*>(q + 32 * s);
        if constexpr (WIDE) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                v8bf aw[2];
                f8_widen<MG_E4M3>(a[s], f8_value(sa), aw);
#pragma unroll
                for (int c = 0; c < NG; ++c) {
                    v8bf ww[2];
                    f8_widen<MG_E4M3>(w[d][c][s], f8_value(sw[d][c]), ww);
                    acc[c] = f8_mfma_wide(ww, aw, acc[c]);
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 4; s += 2)
#pragma unroll
                for (int c = 0; c < NG; ++c)
                    acc[c] = f8_mfma<MG_E4M3>(w[d][c][s], w[d][c][s + 1], a[s], a[s + 1], sw[d][c], sa, acc[c]);
        }
    };
    int u0 = wave;
    for (; u0 + D * NW < units; u0 += D * NW) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            multiply(u0 + d * NW, d);
            load_w(u0 + (d + D) * NW, d);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) multiply(u0 + d * NW, d);

    // ---- join and epilogue
    __syncthreads();                                                  // the codes are read
    float* part = reinterpret_cast<float*>(lds);
    if (l32 < M) {
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<ep_f32x4*>(part + (size_t)(wave * M + l32) * ROW + 32 * c + 8 * q + 4 * h) =
                    ep_f32x4{acc[c][4 * q], acc[c][4 * q + 1], acc[c][4 * q + 2], acc[c][4 * q + 3]};
    }
    __syncthreads();
    constexpr int PR = OUT == kDirGated ? 8 : 8 * NG;                 // pieces of 4 columns per row
    for (int p = tid; p < M * PR; p += 64 * NW) {
        const int m = p / PR, pc = 4 * (p - m * PR);
        auto sum = [&](int col, float (&v)[4]) {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = 0.0f;
#pragma unroll
            for (int x = 0; x < NW; ++x) {
                const ep_f32x4 s = *reinterpret_cast<const ep_f32x4*>(part + (size_t)(x * M + m) * ROW + col);
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] += s[c];
            }
        };
        float v[4];
        sum(pc, v);
        if constexpr (OUT == kDirGated) {
            float u[4];
            sum(32 + pc, u);
            ep_by_act(g.act, [&](auto A) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float a, d;
                    act_slope<decltype(A)::value>(v[c], a, d);
                    v[c] = a * u[c];
                }
            });
            *reinterpret_cast<ep_f32x4*>(static_cast<float*>(g.Y) + (int64_t)m * g.F + 32 * bx + pc) = ep_f32x4{v[0], v[1], v[2], v[3]};
        } else {
            const int col = 32 * NG * bx + pc;
            if (col >= N) continue;
            float b[4] = {}, r[4] = {}, gt[4] = {1.0f, 1.0f, 1.0f, 1.0f};
            const int mi = mod_row(e.mod, m);
            if (e.bias) ep_load4(e.bias, col, e.bias_dtype == MG_F32, b);
            if (e.residual) ep_load4(e.residual, m * e.ldr + col, e.residual_dtype == MG_F32, r);
            if (e.mod.gate && mi >= 0) ep_load4(e.mod.gate, (int64_t)mi * e.mod.ld + col, e.mod.dtype == MG_F32, gt);
            ep_by_act(e.act, [&](auto A) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = ep_act<decltype(A)::value>(v[c] + b[c]);
            });
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = mi < 0 ? r[c] : __builtin_fmaf(gt[c], v[c], r[c]);
            if constexpr (OUT == kDirF32)
                *reinterpret_cast<ep_f32x4*>(static_cast<float*>(g.Y) + (int64_t)m * N + col) = ep_f32x4{v[0], v[1], v[2], v[3]};
            else
                *reinterpret_cast<ep_u32x2*>(static_cast<uint16_t*>(g.Y) + (int64_t)m * N + col) =
                    ep_u32x2{ep_pack(v[0], v[1]), ep_pack(v[2], v[3])};
        }
    }
}

constexpr int kDirLds = 64 * 1024;                 // two workgroups a CU
constexpr int kDirRows = 16;
static_assert(8 * kDirRows * 68 * 4 <= kDirLds, "the waves' sums fit");

int lds_bytes(int M, int K, int NG, int NW) {
    const int codes = (int)(f8_slices(K) / 4) * M * (kDirRow + 4), sums = NW * M * (32 * NG + 4) * 4;
    return codes > sums ? codes : sums;
}

template <typename XT, int OUT, int NG, int NW, int D>
hipError_t run(F8DirectArgs a, hipStream_t st) {
    a.tiles = OUT == kDirGated ? a.F / 32 : (a.N + 32 * NG - 1) / (32 * NG);
    hipLaunchKernelGGL((f8_direct<XT, OUT, NG, NW, D>), dim3((unsigned)((a.tiles + 7) / 8 * 8)), dim3(64 * NW),
                       lds_bytes(a.M, a.K, NG, NW), st, a);
    return hipGetLastError();
}

// 8 waves a workgroup with two blocks of weights each in flight, one when they are
// the gate's and the up product's: one row 5120 -> 13824 12.2 us; 4 waves, or 1, 3 or
// 4 blocks, 12.7-14.4; the gated block 43.2, the others 44.2-46.5.
template <typename XT>
hipError_t by_out(const F8DirectArgs& a, int32_t y_dtype, bool gated, hipStream_t st) {
    if (gated) return run<XT, kDirGated, 2, 8, 1>(a, st);
    return y_dtype == MG_F32 ? run<XT, kDirF32, 1, 8, 2>(a, st) : run<XT, kDirBf16, 1, 8, 2>(a, st);
}

}  // namespace

int f8_direct_rows(int32_t K) {
    const int fit = kDirLds / ((int)(f8_slices(K) / 4) * (kDirRow + 4));
    return fit < kDirRows ? fit : kDirRows;
}

// Column tiles of the last product for each CU, at least 1.
static double tiles_per_cu(int32_t N) {
    const double t = (N + 31) / 32 / (double)device_cu_count();
    return t > 1.0 ? t : 1.0;
}

// Every workgroup quantizes all rows, so the two launches win once that is more
// than a launch's latency, and the sooner the more workgroups a CU runs.  Up to
// three rows of 2048 channels or more stay: their weights' way is the time, and
// the direct kernel streams them faster.  Direct against two launches, in a graph,
// weights from memory: 5120 -> 13824 1 row 15.1 us, 17.1; 3 rows 16.9, 17.4; 4 rows
// 17.9, 17.5; 5 rows 18.8, 17.5; 5120 -> 55296 1 row 52, 58; 5 rows 60, 56; 13824 -> 5120
// 2 rows 19.1, 20.3; 3 rows 21.1, 20.3; 5120 -> 5120 4 rows 10.1, 10.7; 8 rows 12.6, 10.8; 2048
// -> 8192 14 rows 9.0, 9.2; 1024 -> 1056 16 rows 5.2, 6.2; 1024 -> 13824 12 rows 7.9, 8.0;
// 16 rows 8.5, 8.1; 1024 -> 55296 1 row 16.0, 14.7; 16 rows 24.4, 15.8; 1024 -> 131072 16
// rows 49.6, 29.9.  Of 133 such calls (K 1024 to 13824, N 1056 to 131072) the rule
// takes the slower one, by 4 to 7 %, at 5120 -> 8192 5 rows, 13824 -> 8192 and -> 27648 2
// rows, 5120 -> 27648 3 rows, and by less elsewhere.
bool f8_direct_pays(int64_t M, int32_t K, int32_t N) {
    const int64_t units = f8_slices(K) / 4;
    if (M > f8_direct_rows(K) || M * units > 224) return false;
    return (M <= 3 && units >= 16) || (double)(M * units + 32) * tiles_per_cu(N) <= 264.0;
}

// The gated block saves two launches and quantizes twice.  Direct against its
// steps apart: 5120 -> 13824 -> 5120 1 row 47.0, 49.9; 3 rows 48.8, 50.6; 4 rows 51.0, 50.6; 1024
// -> 4096 -> 1024 9 rows 17.1, 17.3; 13 rows 19.5, 17.4; 5120 -> 5120 -> 5120 5 rows 27.2, 26.6; 7 rows
// 30.0, 26.9; 5120 -> 1024 -> 5120 11 rows 22.3, 18.7; 2048 -> 2048 -> 55296 3 rows 31.3, 34.3; 16 rows
// 50.0, 36.0.  Of 71 such blocks the rule takes the slower form, by 9 %, at 5120
// -> 1024 -> 5120 8 rows, and by 2 % at most elsewhere.
bool f8_direct_pays_gated(int64_t M, int32_t K, int32_t F, int32_t N) {
    const int64_t units = f8_slices(K) / 4 + f8_slices(F) / 4;
    if (M > f8_direct_rows(K) || M > f8_direct_rows(F) || M * units > 600) return false;
    return M <= 3 || (double)(M * units) * tiles_per_cu(N) <= 470.0;
}

hipError_t launch_f8_direct(F8DirectArgs a, int32_t x_dtype, int32_t y_dtype, bool gated, hipStream_t st) {
    const int64_t size = x_dtype == MG_F32 ? 4 : 2;
    a.vec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && (a.M == 1 || a.ldx * size % 16 == 0);
    return x_dtype == MG_F32 ? by_out<float>(a, y_dtype, gated, st) : by_out<uint16_t>(a, y_dtype, gated, st);
}

}  // namespace mg
