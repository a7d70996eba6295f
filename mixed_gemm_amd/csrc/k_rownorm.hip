// Row operators around the block: the norm ahead of it with its modulation,
// the gated residual after it (with the norm after the block), and the norm
// fused with the quantize step of the projection behind it.
//
// A workgroup takes whole rows and keeps them in registers: a thread holds V
// vectors of 8 consecutive channels (vector v at channel 8 (v T + thread), T
// threads), so X and Y are read once and everything else is arithmetic on
// registers.  The mean and the sum of squared deviations are formed without
// cancellation: each wave sums its own channels, takes deviations from its
// own mean, and the waves' (sum, squares) pairs are joined by the parallel
// variance formula (T. Chan, G. Golub, R. LeVeque, 1983), so one exchange
// through LDS serves both.
#include <type_traits>

#include "mg_block.h"
#include "mg_device.h"
#include "mg_internal.h"

namespace mg {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) Piece16 { u32x4 v; };   // 16 bytes at any element's alignment

constexpr int kMaxWaves = 16;

// Sum over the wave's 64 lanes, in every lane: DPP adds inside rows of 16,
// then across the rows into lane 63.
__device__ __forceinline__ float wave_sum(float v) {
    auto dpp = [](float x, auto ctrl, auto rows) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value,
                                                          decltype(rows)::value, 0xF, true));
    };
#define MG_DPP_ADD(ctrl, rows) v += dpp(v, std::integral_constant<int, ctrl>{}, std::integral_constant<int, rows>{})
    MG_DPP_ADD(0xB1, 0xF);     // lane ^ 1
    MG_DPP_ADD(0x4E, 0xF);     // lane ^ 2
    MG_DPP_ADD(0x141, 0xF);    // mirror in 8
    MG_DPP_ADD(0x140, 0xF);    // mirror in 16
    MG_DPP_ADD(0x142, 0xA);    // row 0 -> 1, 2 -> 3
    MG_DPP_ADD(0x143, 0xC);    // rows 0-1 -> 2, 3
#undef MG_DPP_ADD
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// 8 consecutive elements from p on, of which `left` exist (the rest read as 0).
__device__ __forceinline__ void load8(const uint16_t* p, int left, float (&v)[8]) {
    if (left >= 8) {
        const u32x4 w = reinterpret_cast<const Piece16*>(p)->v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? bf16_to_f32(p[i]) : 0.0f;
    }
}
__device__ __forceinline__ void load8(const float* p, int left, float (&v)[8]) {
    if (left >= 8) {
        const u32x4 a = reinterpret_cast<const Piece16*>(p)->v, b = reinterpret_cast<const Piece16*>(p + 4)->v;
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = __uint_as_float(a[i]); v[4 + i] = __uint_as_float(b[i]); }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void load8(const void* p, int64_t at, int32_t dtype, int left, float (&v)[8]) {
    if (dtype == MG_F32) load8(static_cast<const float*>(p) + at, left, v);
    else load8(static_cast<const uint16_t*>(p) + at, left, v);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// two floats rounded to bf16 (nearest even, NaN kept), the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ void store8(void* p, int64_t at, int32_t dtype, int left, const float (&v)[8]) {
    if (left <= 0) return;
    if (dtype == MG_F32) {
        float* q = static_cast<float*>(p) + at;
        if (left >= 8) {
            u32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) { a[i] = __float_as_uint(v[i]); b[i] = __float_as_uint(v[4 + i]); }
            reinterpret_cast<Piece16*>(q)->v = a;
            reinterpret_cast<Piece16*>(q + 4)->v = b;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) q[i] = v[i];
        }
    } else {
        uint16_t* q = static_cast<uint16_t*>(p) + at;
        const u32x4 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        if (left >= 8) {
            reinterpret_cast<Piece16*>(q)->v = w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Elements of wave w's channels below K.
__device__ __forceinline__ int wave_count(int w, int V, int T, int K) {
    int n = 0;
    for (int v = 0; v < V; ++v) {
        const int left = K - 8 * (v * T + 64 * w);
        n += left < 0 ? 0 : left < 512 ? left : 512;
    }
    return n;
}

template <int V>
struct RowThread {
    int W, T, wave, K;
    int col[V];                     // first channel of vector v
    int n;                          // channels of this wave
    float rn;
    bool whole;                     // every lane of the wave has all its channels

    __device__ __forceinline__ RowThread(int K_) : K(K_) {
        T = blockDim.x;
        W = T >> 6;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
#pragma unroll
        for (int v = 0; v < V; ++v) col[v] = 8 * (v * T + (int)threadIdx.x);
        n = wave_count(wave, V, T, K);
        rn = n ? 1.0f / (float)n : 0.0f;
        whole = n == 512 * V;
    }
    __device__ __forceinline__ int left(int v) const { return K - col[v]; }
};

// mean (0 for rms) and 1 / sqrt(var + eps) of the row x.  The waves exchange
// (sum, squared deviations from the wave's mean) through one slot each of two
// sets used in turn, so that one barrier suffices: a wave writes a set again
// only after the barrier of the other, which every reader of the set has
// passed.
template <int V>
__device__ __forceinline__ void row_stats(const float (&x)[V][8], const RowThread<V>& t, const NormArgs& nm, f32x2 (*pair)[kMaxWaves],
                                          int& turn, float& mean, float& rstd) {
    float s = 0.0f, m = 0.0f, q = 0.0f;
    if (nm.kind == MG_NORM_LAYER) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[v][i];
        s = wave_sum(s);
        m = s * t.rn;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = t.whole || i < t.left(v) ? x[v][i] - m : 0.0f;
            q = __builtin_fmaf(d, d, q);
        }
    q = wave_sum(q);
    f32x2* set = pair[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) set[t.wave] = f32x2{s, q};
    __syncthreads();
    float S = 0.0f, Q = 0.0f;
    for (int w = 0; w < t.W; ++w) S += set[w][0];
    mean = S / (float)t.K;
    for (int w = 0; w < t.W; ++w) {
        const float nw = (float)wave_count(w, V, t.T, t.K);
        const float d = nw > 0.0f ? set[w][0] / nw - mean : 0.0f;
        Q += set[w][1] + nw * d * d;
    }
    rstd = 1.0f / __fsqrt_rn(Q / (float)t.K + nm.eps);
}

// v = ((x - mean) rstd) w + b of 8 channels
__device__ __forceinline__ void norm8(float (&x)[8], int64_t col, int left, const NormArgs& n, float mean, float rstd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (x[i] - mean) * rstd;
    float c[8];
    if (n.weight) {
        load8(n.weight, col, n.dtype, left, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= c[i];
    }
    if (n.bias) {
        load8(n.bias, col, n.dtype, left, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += c[i];
    }
}

// x (1 + scale_i) + shift_i, or 0 on a padding row
__device__ __forceinline__ void mod8(float (&x)[8], int64_t col, int left, const ModArgs& m, int row) {
    float c[8];
    if (row < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        return;
    }
    if (m.scale) {
        load8(m.scale, row * m.ld + col, m.dtype, left, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= 1.0f + c[i];
    }
    if (m.shift) {
        load8(m.shift, row * m.ld + col, m.dtype, left, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += c[i];
    }
}

template <int V>
__global__ void __launch_bounds__(64 * kMaxWaves) row_kernel(RowArgs a) {
    __shared__ f32x2 pair[2][kMaxWaves];
    int turn = 0;
    const RowThread<V> t(a.K);
    for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
        const int gi = mod_row(a.gate, r), mi = mod_row(a.mod, r);
        float x[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) load8(a.X, r * a.ldx + t.col[v], a.x_dtype, t.left(v), x[v]);
        if (a.Y) {
            float y[V][8];
#pragma unroll
            for (int v = 0; v < V; ++v) load8(a.Y, r * a.ldy + t.col[v], a.y_dtype, t.left(v), y[v]);
            if (a.has_post) {
                float mean, rstd;
                row_stats<V>(y, t, a.post, pair, turn, mean, rstd);
#pragma unroll
                for (int v = 0; v < V; ++v) norm8(y[v], t.col[v], t.left(v), a.post, mean, rstd);
            }
            if (gi >= 0) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float c[8] = {1, 1, 1, 1, 1, 1, 1, 1};
                    if (a.gate.gate) load8(a.gate.gate, gi * a.gate.ld + t.col[v], a.gate.dtype, t.left(v), c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[v][i] = t.whole || i < t.left(v) ? __builtin_fmaf(c[i], y[v][i], x[v][i]) : 0.0f;
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) store8(a.O, r * a.ldo + t.col[v], a.x_dtype, t.left(v), x[v]);
        }
        if (a.has_norm) {
            float mean, rstd;
            row_stats<V>(x, t, a.norm, pair, turn, mean, rstd);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                norm8(x[v], t.col[v], t.left(v), a.norm, mean, rstd);
                mod8(x[v], t.col[v], t.left(v), a.mod, mi);
                store8(a.H, r * a.ldh + t.col[v], a.h_dtype, t.left(v), x[v]);
            }
        }
    }
}

template <int V>
__global__ void __launch_bounds__(64 * kMaxWaves) norm_quant_kernel(NormQuantArgs g) {
    __shared__ f32x2 pair[2][kMaxWaves];
    int turn = 0;
    const RowArgs& a = g.r;
    const int K = a.K;
    const RowThread<V> t(K);
    const int64_t ns4 = frag_slices(K / 2), nso = frag_slices(2 * (int64_t)g.k);
    const int64_t Mp = (a.M + kScRows - 1) / kScRows * kScRows, M32 = (a.M + 31) / 32 * 32;
    for (int64_t r = blockIdx.x; r < Mp; r += gridDim.x) {
        const bool live = r < a.M, piece = r < M32;
        float x[V][8] = {};
        if (live) {
            const int mi = mod_row(a.mod, r);
#pragma unroll
            for (int v = 0; v < V; ++v) load8(a.X, r * a.ldx + t.col[v], a.x_dtype, t.left(v), x[v]);
            float mean, rstd;
            row_stats<V>(x, t, a.norm, pair, turn, mean, rstd);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                norm8(x[v], t.col[v], t.left(v), a.norm, mean, rstd);
                mod8(x[v], t.col[v], t.left(v), a.mod, mi);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int j0 = t.col[v];
            if (j0 >= (K + 511) / 512 * 512) continue;        // whole waves
            float q[8], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                q[i] = 0.0f;
                if (j0 < K) {                                 // K % 32 == 0: whole vectors
                    q[i] = __fdiv_rn(bf16_to_f32(pack_bf16(x[v][i], 0.0f) & 0xFFFFu), g.s[j0 + i]);
                    const int p = g.pos[j0 + i];
                    if (p >= 0) {
                        if (piece)
                            *reinterpret_cast<uint16_t*>(g.XO + frag_offset(r, 2 * (int64_t)p, nso)) =
                                (uint16_t)f32_to_bf16_rne(q[i]);
                        q[i] = 0.0f;
                    }
                }
                amax = fmaxf(amax, __builtin_fabsf(q[i]));
            }
            const uint32_t c = e8m0_from_amax_bits(quad_max_bits(__float_as_uint(amax)));
            const float scale = e8m0_to_f32(c);
            uint32_t word = 0;
            MG_CVT_FP4X2(word, q[0], q[1], scale, 0);
            MG_CVT_FP4X2(word, q[2], q[3], scale, 1);
            MG_CVT_FP4X2(word, q[4], q[5], scale, 2);
            MG_CVT_FP4X2(word, q[6], q[7], scale, 3);
            if (piece && j0 < 64 * ns4) *reinterpret_cast<uint32_t*>(g.Aq + frag_offset(r, j0 / 2, ns4)) = word;
            if ((threadIdx.x & 3) == 0) g.As[sc_offset(r, j0 / 32, sc_nwin(K))] = (uint8_t)c;
        }
        if (piece && (int)threadIdx.x < 16 * (int)nso - g.k)
            *reinterpret_cast<uint16_t*>(g.XO + frag_offset(r, 2 * (int64_t)(g.k + threadIdx.x), nso)) = 0;
    }
}

// Waves and vectors per thread for rows of K channels: 512 channels a wave and
// vector, up to 8 waves, then more vectors, then more waves.
struct Shape { int W, V; };
Shape shape_of(int32_t K) {
    const int nw = (K + 511) / 512;
    int V = (nw + 7) / 8;
    V = V <= 4 ? V : 8;
    return Shape{(nw + V - 1) / V, V};
}

template <typename F>
hipError_t by_v(int V, F&& f) {
    switch (V) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 3: return f(std::integral_constant<int, 3>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

}  // namespace

hipError_t launch_rows(const RowArgs& a, hipStream_t st) {
    const Shape sh = shape_of(a.K);
    const int64_t blocks = a.M < 65536 ? a.M : 65536;
    return by_v(sh.V, [&](auto v) {
        hipLaunchKernelGGL((row_kernel<decltype(v)::value>), dim3((unsigned)blocks), dim3(64 * sh.W), 0, st, a);
        return hipGetLastError();
    });
}

hipError_t launch_norm_quant(const NormQuantArgs& a, hipStream_t st) {
    const Shape sh = shape_of(a.r.K);
    const int64_t Mp = (a.r.M + kScRows - 1) / kScRows * kScRows;
    const int64_t blocks = Mp < 65536 ? Mp : 65536;
    return by_v(sh.V, [&](auto v) {
        hipLaunchKernelGGL((norm_quant_kernel<decltype(v)::value>), dim3((unsigned)blocks), dim3(64 * sh.W), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace mg
