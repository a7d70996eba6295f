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
//
// Rows may start at any element and have any width from 8 on: loads are
// unaligned 16-byte loads, and a thread at the row's end holds the row's last
// 8 channels, so that no load needs a branch; those of them that the thread
// before holds too count as 0 in the sums, and are stored by both with the same
// value, or by the thread before alone where outputs and inputs share memory.
#include <type_traits>

#include "mg_block.h"
#include "mg_device.h"
#include "mg_internal.h"

namespace mg {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) Piece16 { u32x4 v; };   // 16 bytes at any element's alignment

constexpr int kMaxWaves = 16;

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, true));
}
// Sum over each row of 16 lanes, in every lane of the row.
__device__ __forceinline__ float row16_sum(float v) {
    v = dpp_add<0xB1, 0xF>(v);         // lane ^ 1
    v = dpp_add<0x4E, 0xF>(v);         // lane ^ 2
    v = dpp_add<0x141, 0xF>(v);        // mirror in 8
    return dpp_add<0x140, 0xF>(v);     // mirror in 16
}
// Sum over the wave, wave-uniform.
__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    v = dpp_add<0x142, 0xA>(v);        // row 0 -> 1, 2 -> 3
    v = dpp_add<0x143, 0xC>(v);        // rows 0-1 -> 2, 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// 8 consecutive elements as they lie in memory: T float or uint16_t (bf16).
template <typename T>
struct Raw8 {
    u32x4 d[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, Raw8<T>& r) {
    constexpr int N = sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < N; ++i) r.d[i] = reinterpret_cast<const Piece16*>(p + 8 / N * i)->v;
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(r.d[i >> 2][i & 3]);
        else v[i] = __uint_as_float(i & 1 ? r.d[0][i >> 1] & 0xFFFF0000u : r.d[0][i >> 1] << 16);
    }
}

// The same of a type known at run time (null pointer: nothing).  Loading and
// using are apart, so that the loads of several arrays are in flight together.
struct RawAny {
    u32x4 d[2];
};
__device__ __forceinline__ void load_any(const void* p, int64_t at, int32_t dtype, RawAny& r) {
    if (p == nullptr) return;
    if (dtype == MG_F32) {
        const Piece16* q = reinterpret_cast<const Piece16*>(static_cast<const float*>(p) + at);
        r.d[0] = q[0].v;
        r.d[1] = q[1].v;
    } else {
        r.d[0] = reinterpret_cast<const Piece16*>(static_cast<const uint16_t*>(p) + at)->v;
    }
}
__device__ __forceinline__ void unpack(const RawAny& r, int32_t dtype, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float(dtype == MG_F32 ? r.d[i >> 2][i & 3]
                                               : i & 1 ? r.d[0][i >> 1] & 0xFFFF0000u : r.d[0][i >> 1] << 16);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// two floats rounded to bf16 (nearest even, NaN kept), the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ u32x4 pack8_bf16(const float (&v)[8]) {
    return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

// A thread's place in rows of K >= 8 channels: V vectors, W waves.  ODD: K need
// not be a multiple of 8.
template <int V, bool ODD = true>
struct RowThread {
    int W, T, wave, K, shift;       // shift: channels missing in the row's last vector
    int col[V];                     // first channel of vector v
    int at[V];                      // channel of its first element (past K - 8: K - 8, the row's last 8)
    uint32_t full, cut;             // bit v: the wave's vector lies inside the row; holds its last, partial vector
    float rn, rK;                   // 1 / channels of this wave, 1 / K
    float nl, rnl;                  // channels of wave (lane % 16), 1 / them (0 past the last wave)

    __device__ __forceinline__ RowThread(int K_) : K(K_) {
        T = blockDim.x;
        W = T >> 6;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        shift = (8 - (K & 7)) & 7;
        full = cut = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            col[v] = 8 * (v * T + (int)threadIdx.x);
            at[v] = col[v] < K - 8 ? col[v] : K - 8;
            const int l = K - 8 * (v * T + 64 * wave);
            full |= (l >= 512 ? 1u : 0u) << v;
            cut |= (shift && l > 0 && l < 512 ? 1u : 0u) << v;
        }
        auto count = [&](int w) {
            int c = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int l = K - 8 * (v * T + 64 * w);
                c += l < 0 ? 0 : l < 512 ? l : 512;
            }
            return c;
        };
        const int c = count(wave), cl = (int)(threadIdx.x & 15) < W ? count((int)threadIdx.x & 15) : 0;
        rn = c ? 1.0f / (float)c : 0.0f;
        nl = (float)cl;
        rnl = cl ? 1.0f / (float)cl : 0.0f;
        rK = 1.0f / (float)K;
    }
    // Of a vector's 8 elements the first skip(v) are not its own: 0 inside the
    // row, 8 or more past it.  In the row's last, partial vector they are the
    // vector before's: not counted in the sums, and stored with its values.
    __device__ __forceinline__ int skip(int v) const { return col[v] - at[v]; }
    __device__ __forceinline__ bool whole() const { return full == (1u << V) - 1u; }
    // 0 past the row (the wave of the partial vector masks its sums instead)
    __device__ __forceinline__ void own(int v, float (&x)[8]) const {
        if (full >> v & 1u || (ODD && (cut >> v & 1u))) return;
        const bool in = skip(v) == 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = in ? x[i] : 0.0f;
    }
    // 8 values of a [K] array of either type
    __device__ __forceinline__ void load8(const void* p, int64_t row, int32_t dtype, int v, float (&x)[8]) const {
        RawAny r;
        load_any(p, row + at[v], dtype, r);
        unpack(r, dtype, x);
    }
    __device__ __forceinline__ void store8(void* p, int64_t row, int32_t dtype, int v, const float (&x)[8], bool apart) const {
        const bool f32 = dtype == MG_F32;
        float* const pf = static_cast<float*>(p) + row + at[v];
        uint16_t* const pb = static_cast<uint16_t*>(p) + row + at[v];
        auto piece = [&]() {
            if (f32) {
                u32x4 a, b;
#pragma unroll
                for (int i = 0; i < 4; ++i) { a[i] = __float_as_uint(x[i]); b[i] = __float_as_uint(x[4 + i]); }
                reinterpret_cast<Piece16*>(pf)->v = a;
                reinterpret_cast<Piece16*>(pf + 4)->v = b;
            } else {
                reinterpret_cast<Piece16*>(pb)->v = pack8_bf16(x);
            }
        };
        if (full >> v & 1u) {
            piece();
            return;
        }
        // a partial vector as a whole one: its elements one by one took 120 us for
        // 9973 x 5121 (residual, bf16), this 108 us
        if (skip(v) < (ODD && apart ? 8 : 1)) piece();
        if (ODD && !apart && (cut >> v & 1u) && skip(v) == shift) {
            const u32x4 w = pack8_bf16(x);
#pragma unroll
            for (int i = 1; i < 8; ++i)
                if (i >= shift) {
                    if (f32) pf[i] = x[i];
                    else pb[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                }
        }
    }
};

// The waves' (sum, squared deviations from the wave's mean) of a row, two sets
// used in turn so that one barrier suffices: a wave writes a set again only
// after the barrier of the other, which every reader of the set has passed.
typedef f32x2 Pairs[2][kMaxWaves];

// 1 / sqrt(v), v >= 0 (the hardware's, one unit in the last place; subnormal v
// scaled into its range)
__device__ __forceinline__ float rsqrt_f32(float v) {
    const bool tiny = v < 0x1p-100f;
    const float r = __builtin_amdgcn_rsqf(tiny ? v * 0x1p100f : v);
    return tiny ? r * 0x1p50f : r;
}

// sum / K: the product with RN(1 / K) corrected by its remainder (P. Markstein,
// 1990), the quotient correctly rounded.  The product alone is up to 1.5 units
// of the mean off, which 1 / sqrt(eps) = 1000 made 0.03 of a constant row of 100.
__device__ __forceinline__ float mean_of(float sum, int K, float rK) {
    asm volatile("" : "+s"(K));      // converted here, not held in a vector register across the rows
    const float m = sum * rK;
    return __builtin_fmaf(__builtin_fmaf(-m, (float)K, sum), rK, m);
}

// mean (0 for rms) and 1 / sqrt(var + eps) of the row x: the parallel variance
// formula over the waves, whose pairs the 16 lanes of a row take one each.
template <int V, bool ODD>
__device__ __forceinline__ void row_stats(const float (&x)[V][8], const RowThread<V, ODD>& t, int kind, float eps, Pairs& pairs,
                                          int& turn, float& mean, float& rstd) {
    float s = 0.0f, m = 0.0f, q = 0.0f;
    const bool layer = kind == MG_NORM_LAYER;
    const bool part = ODD && t.cut != 0;                // the wave holds the partial vector
    if (layer) {
        if (!part) {                                    // (channels past the row hold 0)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[v][i];
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += i >= t.skip(v) ? x[v][i] : 0.0f;
        }
        s = wave_sum(s);
        m = s * t.rn;
    }
    if (t.whole()) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = x[v][i] - m;
                q = __builtin_fmaf(d, d, q);
            }
    } else if (!part) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float mv = t.skip(v) == 0 ? m : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = x[v][i] - mv;
                q = __builtin_fmaf(d, d, q);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i >= t.skip(v) ? x[v][i] - m : 0.0f;
                q = __builtin_fmaf(d, d, q);
            }
    }
    q = wave_sum(q);
    f32x2* set = pairs[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) set[t.wave] = f32x2{s, q};
    __syncthreads();
    const int l = (int)threadIdx.x & 15;
    const f32x2 p = l < t.W ? set[l] : f32x2{0.0f, 0.0f};
    mean = layer ? mean_of(row16_sum(p[0]), t.K, t.rK) : 0.0f;
    const float d = __builtin_fmaf(p[0], t.rnl, -mean);
    const float Q = row16_sum(__builtin_fmaf(t.nl * d, d, p[1]));
    rstd = rsqrt_f32(__builtin_fmaf(Q, t.rK, eps));
}

// A norm with its modulation folded to n a + c, n = (x - mean) rstd: a = w (1 +
// scale_i), c = b (1 + scale_i) + shift_i of 8 channels (an infinite 1 + scale
// meets a bias as inf - inf where n w + b, formed first, would have kept a sign).
struct FoldRaw {
    RawAny scale, shift, weight, bias;
};
template <typename T>
__device__ __forceinline__ void fold_load(const T& t, const NormArgs& n, const ModArgs& m, int row, int v, FoldRaw& f) {
    load_any(m.scale, row * m.ld + t.at[v], m.dtype, f.scale);
    load_any(m.shift, row * m.ld + t.at[v], m.dtype, f.shift);
    load_any(n.bias, t.at[v], n.dtype, f.bias);
    load_any(n.weight, t.at[v], n.dtype, f.weight);
}
__device__ __forceinline__ void fold_make(const NormArgs& n, const ModArgs& m, const FoldRaw& f, float (&a)[8], float (&c)[8]) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { a[i] = 1.0f; c[i] = 0.0f; }
    if (m.scale) {
        unpack(f.scale, m.dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = 1.0f + w[i];
    }
    if (m.shift) unpack(f.shift, m.dtype, c);
    if (n.bias) {
        unpack(f.bias, n.dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = __builtin_fmaf(w[i], a[i], c[i]);
    }
    if (n.weight) {
        unpack(f.weight, n.dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= w[i];
    }
}
template <typename T>
__device__ __forceinline__ void fold8(const T& t, const NormArgs& n, const ModArgs& m, int row, int v,
                                      float (&a)[8], float (&c)[8]) {
    FoldRaw f;
    fold_load(t, n, m, row, v, f);
    fold_make(n, m, f, a, c);
}
// of all vectors, two at a time
template <int V, bool ODD>
__device__ __forceinline__ void fold_all(const RowThread<V, ODD>& t, const NormArgs& n, const ModArgs& m, int row,
                                         float (&a)[V][8], float (&c)[V][8]) {
    constexpr int G = V <= 2 ? 1 : 2;
#pragma unroll
    for (int v = 0; v < V; v += G) {
        FoldRaw f[G];
#pragma unroll
        for (int k = 0; k < G; ++k) fold_load(t, n, m, row, v + k, f[k]);
#pragma unroll
        for (int k = 0; k < G; ++k) fold_make(n, m, f[k], a[v + k], c[v + k]);
    }
}
// n of one channel.  x - mean is formed first, exact where x is near the mean:
// as x rstd - mean rstd it would carry the rounding of a product that the
// distance to the mean can be any small part of.
__device__ __forceinline__ float normed(float x, float mean, float rstd) { return (x - mean) * rstd; }
// n a + c
__device__ __forceinline__ void apply8(float (&x)[8], float mean, float rstd, const float (&a)[8], const float (&c)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_fmaf(normed(x[i], mean, rstd), a[i], c[i]);
}
// 8 values of an optional array (1 without one)
template <typename T>
__device__ __forceinline__ void load_or_1(const T& t, const void* p, int64_t row, int32_t dtype, int v, float (&g)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.0f;
    if (p) t.load8(p, row, dtype, v, g);
}

// Arguments that a row rarely needs, read from the kernel-argument segment
// (which starts with a RowArgs) where they are used, through a pointer the
// compiler cannot see through: held in scalar registers across the rows they
// would be spilled there.
typedef const __attribute__((address_space(4))) RowArgs* RowKernargs;
__device__ __forceinline__ RowKernargs row_kernargs() {
    RowKernargs p = (RowKernargs)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return p;
}
__device__ __forceinline__ NormArgs norm_of(const __attribute__((address_space(4))) NormArgs& n) {
    return NormArgs{n.weight, n.bias, n.dtype, n.kind, n.eps};
}
__device__ __forceinline__ ModArgs mod_of(const __attribute__((address_space(4))) ModArgs& m) {
    return ModArgs{m.scale, m.shift, m.gate, m.index, m.ld, m.group, m.rows, m.dtype};
}
struct FoldArgs {
    NormArgs norm;
    ModArgs mod;
};
__device__ __forceinline__ FoldArgs fold_args() {
    const RowKernargs p = row_kernargs();
    return FoldArgs{norm_of(p->norm), mod_of(p->mod)};
}

// The norm after the block (weight pw; the rare bias is read where it is used).
template <typename T>
__device__ __forceinline__ void post8(const T& t, float (&y)[8], const float (&pw)[8], int v, float mean, float rstd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = normed(y[i], mean, rstd) * pw[i];
    const RowKernargs p = row_kernargs();
    if (p->post.bias) {
        float c[8];
        t.load8(p->post.bias, 0, p->post.dtype, v, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += c[i];
    }
}

// The rows of a workgroup, r0 + i step for i < count: consecutive where token
// rows of a sample share a modulation row, else spread over the workgroups.
struct RowSpan {
    int64_t chunk, step;        // rows per workgroup; 1, or the number of workgroups
};

template <int V, typename XT, typename YT>
struct RowShape {
    static constexpr bool res = !std::is_void_v<YT>, ahead = V <= 4, keep = res ? V <= 2 : V <= 4;
    static constexpr bool lds = res && V == 4;          // the folded coefficients in LDS, the gate in registers
    static constexpr int lds_thread = lds ? V * 64 : 0; // bytes of a thread
    using Y = std::conditional_t<res, YT, uint16_t>;
    static constexpr int waves = V > 4 ? 4 : V == 4 ? 2 : V == 2 ? (res ? 2 : 4) : (res ? 4 : 5);    // per SIMD
};

// While a row is worked on, the next one's loads are in flight.  Up to 16384
// channels the folded coefficients and the gate are kept until the modulation
// row changes, in registers, or the coefficients of more than 8192 channels
// with a residual in LDS, each thread its own; wider rows read them per row,
// as rows of more than 8192 do the weights of the norm after the block.  (Any
// load of a row's body returns only after the next row's, so reading them per
// row costs the time that the loads ahead are to hide.)  XT, YT: types of X
// and Y (YT void: no residual step).
//
// Bound: memory, each row read and written once.  Norm with modulation of
// 32760 x 5120, f32 in, bf16 out (1006 MB): 172 us, 5.8 TB/s (a 1 GiB copy:
// 5.1); bf16 in 123 us, 5.4.  Gated residual with the next norm of
// 75600 x 5120, f32 stream, bf16 block output (4.65 GB): 872 us, 5.3; bf16
// stream 545 us, 5.7.  10000 x 13824, f32 stream, 322 us, 5.2.  9973 x 2049 bf16
// with a norm after the block and padding rows (164 MB) 51 us, 3.2: rows at odd
// addresses and two exchanges a row.  One row: 3.8-4.2 us, the
// launch and one trip to memory.  Reading a row twice (statistics, then the
// result) would cost half as much again; two rows ahead instead of one
// measured no gain, since the waves on a CU already fill its path to memory.
template <int V, typename XT, typename YT>
__global__ void __launch_bounds__(V <= 4 ? 512 : 1024) __attribute__((amdgpu_waves_per_eu(RowShape<V, XT, YT>::waves)))
row_kernel(RowArgs a, RowSpan span) {
    using S = RowShape<V, XT, YT>;
    constexpr bool RES = S::res, KEEP = S::keep, LDS = S::lds, GATE = RES && (KEEP || LDS);
    using Y = typename S::Y;
    __shared__ Pairs pairs;
    extern __shared__ __attribute__((aligned(16))) uint8_t coefs[];      // a and c, 32 bytes each, per vector and thread
    int turn = 0;
    const RowThread<V> t(a.K);
    f32x4* const mine = reinterpret_cast<f32x4*>(coefs) + threadIdx.x;    // + T per 16 bytes: no bank conflicts, no barrier
    float na[KEEP ? V : 1][8], nc[KEEP ? V : 1][8], ga[GATE ? V : 1][8], pw[KEEP && RES ? V : 1][8];
    int mi_of = -1, gi_of = -1;       // modulation rows that the kept coefficients belong to
    Raw8<XT> rx[V];
    Raw8<Y> ry[RES ? V : 1];
    int mrow = -1, grow = -1;         // modulation rows of the row ahead
    const bool norm = !RES || a.has_norm, post = RES && a.has_post;
    int64_t left = span.step == 1 ? a.M - blockIdx.x * span.chunk : (a.M - 1 - blockIdx.x) / span.step + 1;    // rows to do
    if (span.step == 1 && left > span.chunk) left = span.chunk;
    uint32_t r = (uint32_t)(span.step == 1 ? blockIdx.x * span.chunk : blockIdx.x);      // the row ahead (M < 2^31)
    const XT* px = static_cast<const XT*>(a.X) + r * a.ldx;        // its rows of X and Y
    const Y* py = static_cast<const Y*>(a.Y) + (RES ? r * a.ldy : 0);
    int64_t oo = r * a.ldo, oh = r * a.ldh;                        // this row's of O and H
    const int64_t sx = span.step * a.ldx, sy = span.step * a.ldy, so = span.step * a.ldo, sh = span.step * a.ldh;
    auto load_row = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            load_raw(px + t.at[v], rx[v]);
            if constexpr (RES) load_raw(py + t.at[v], ry[v]);
        }
        if (norm) mrow = mod_row(a.mod, r);
        if constexpr (RES) grow = mod_row(a.gate, r);
    };
    if constexpr (KEEP && RES) {
        if (post) {
#pragma unroll
            for (int v = 0; v < V; ++v) load_or_1(t, a.post.weight, 0, a.post.dtype, v, pw[v]);
        }
    }
    load_row();
    while (true) {
        const int mi = __builtin_amdgcn_readfirstlane(mrow), gi = __builtin_amdgcn_readfirstlane(grow);
        if constexpr (KEEP || LDS) {
            const bool ng = RES && gi >= 0 && gi != gi_of;
            if (ng || (mi >= 0 && mi != mi_of)) {
                RawAny rg[V];
                ModArgs gm{};
                if (ng) {
                    gm = mod_of(row_kernargs()->gate);
#pragma unroll
                    for (int v = 0; v < V; ++v) load_any(gm.gate, gi * gm.ld + t.at[v], gm.dtype, rg[v]);
                    gi_of = gi;
                }
                if (mi >= 0 && mi != mi_of) {
                    const FoldArgs f = fold_args();
                    if constexpr (KEEP) fold_all(t, f.norm, f.mod, mi, na, nc);
                    if constexpr (LDS) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            fold8(t, f.norm, f.mod, mi, v, na[0], nc[0]);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                mine[(4 * v + i) * t.T] = f32x4{na[0][4 * i], na[0][4 * i + 1], na[0][4 * i + 2], na[0][4 * i + 3]};
                                mine[(4 * v + 2 + i) * t.T] = f32x4{nc[0][4 * i], nc[0][4 * i + 1], nc[0][4 * i + 2], nc[0][4 * i + 3]};
                            }
                        }
                    }
                    mi_of = mi;
                }
                if (ng) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) ga[GATE ? v : 0][i] = 1.0f;
                        if (gm.gate) unpack(rg[v], gm.dtype, ga[GATE ? v : 0]);
                    }
                }
            }
        }
        float x[V][8], y[RES ? V : 1][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unpack(rx[v], x[v]);
            t.own(v, x[v]);
            if constexpr (RES) {
                unpack(ry[v], y[v]);
                t.own(v, y[v]);
            }
        }
        const bool more = --left > 0;
        // past the last row it is loaded once more, without a branch
        px += more ? sx : 0;
        if constexpr (RES) py += more ? sy : 0;
        r += more ? (uint32_t)span.step : 0u;
        if constexpr (S::ahead) load_row();
        if constexpr (RES) {
            float mean = 0.0f, rstd = 1.0f;
            if (post) row_stats(y, t, a.post.kind, a.post.eps, pairs, turn, mean, rstd);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (gi >= 0) {
                    if (post) {
                        if constexpr (!KEEP) {
                            const NormArgs n = norm_of(row_kernargs()->post);
                            load_or_1(t, n.weight, 0, n.dtype, v, pw[0]);
                        }
                        post8(t, y[v], pw[KEEP ? v : 0], v, mean, rstd);
                    }
                    if constexpr (!GATE) {
                        const ModArgs m = mod_of(row_kernargs()->gate);
                        load_or_1(t, m.gate, gi * m.ld, m.dtype, v, ga[0]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[v][i] = __builtin_fmaf(ga[GATE ? v : 0][i], y[v][i], x[v][i]);
                    t.own(v, x[v]);
                }
                t.store8(a.O, oo, sizeof(XT) == 4 ? MG_F32 : MG_BF16, v, x[v], a.apart);
            }
            oo += so;
        }
        if (norm) {
            float mean, rstd;
            row_stats(x, t, a.norm.kind, a.norm.eps, pairs, turn, mean, rstd);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (mi >= 0) {
                    if constexpr (LDS) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            na[0][i] = mine[(4 * v + i / 4) * t.T][i % 4];
                            nc[0][i] = mine[(4 * v + 2 + i / 4) * t.T][i % 4];
                        }
                    } else if constexpr (!KEEP) {
                        const FoldArgs f = fold_args();
                        fold8(t, f.norm, f.mod, mi, v, na[0], nc[0]);
                    }
                    apply8(x[v], mean, rstd, na[KEEP ? v : 0], nc[KEEP ? v : 0]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[v][i] = 0.0f;
                }
                t.store8(a.H, oh, a.h_dtype, v, x[v], a.apart);
            }
            oh += sh;
        }
        if (!more) break;
        if constexpr (!S::ahead) load_row();
    }
}

// Rows of 8 to 256 channels, heads as a norm of queries and keys has them: 16
// or 32 lanes take a row, a wave 4 or 2 (a wave each leaves most lanes idle:
// residual bf16 of 75600 rows, 65 wide 46 us against 12, 129 wide 47 us against
// 20, 256 wide 46 us against 32, in the last-level cache).  No barrier, one row
// ahead in flight.  The sums are row_kernel's of one wave, so the bits are.
// Bound: memory where rows fill the lanes (75600 x 256, residual bf16, 32 us, 4.8
// TB/s; x 100 15-16 us, 3.8, from the cache 12.2; norm of f32 into bf16 11.5 us,
// 3.9), else the instructions of a row.
struct NarrowThread {
    int at[1];                      // channel of the lane's first element
    __device__ __forceinline__ void load8(const void* p, int64_t row, int32_t dtype, int v, float (&x)[8]) const {
        RawAny r;
        load_any(p, row + at[v], dtype, r);
        unpack(r, dtype, x);
    }
};
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    v = row16_sum(v);
    if constexpr (LANES == 32) v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));   // lane ^ 16
    return v;
}
template <int LANES, typename XT, typename YT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) row_narrow_kernel(RowArgs a) {
    constexpr int ROWS = 256 / LANES;               // of a workgroup
    constexpr bool RES = !std::is_void_v<YT>;
    using Y = std::conditional_t<RES, YT, uint16_t>;
    const int K = a.K, col = 8 * ((int)threadIdx.x & (LANES - 1));
    NarrowThread t;
    t.at[0] = col < K - 8 ? col : K - 8;
    const int skip = col - t.at[0];                 // leading elements that are not the lane's own (8 and more: past the row)
    const float nK = (float)K, rK = 1.0f / nK;
    const bool norm = !RES || a.has_norm, post = RES && a.has_post;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
    if (r >= a.M) return;
    float na[8], nc[8], ga[8], pw[8];
    int mi_of = -1, gi_of = -1, mrow = -1, grow = -1;
    Raw8<XT> rx;
    Raw8<Y> ry;
    auto load_row = [&](int64_t row) {
        load_raw(static_cast<const XT*>(a.X) + row * a.ldx + t.at[0], rx);
        if constexpr (RES) load_raw(static_cast<const Y*>(a.Y) + row * a.ldy + t.at[0], ry);
        if (norm) mrow = mod_row(a.mod, row);
        if constexpr (RES) grow = mod_row(a.gate, row);
    };
    auto stats = [&](const float (&x)[8], int kind, float eps, float& mean, float& rstd) {
        float s = 0.0f, q = 0.0f;
        mean = 0.0f;
        if (kind == MG_NORM_LAYER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s += i >= skip ? x[i] : 0.0f;
            s = lanes_sum<LANES>(s);
            mean = mean_of(s, K, rK);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = i >= skip ? x[i] - mean : 0.0f;
            q = __builtin_fmaf(d, d, q);
        }
        const float d = __builtin_fmaf(s, rK, -mean);
        rstd = rsqrt_f32(__builtin_fmaf(__builtin_fmaf(nK * d, d, lanes_sum<LANES>(q)), rK, eps));
    };
    auto store8 = [&](void* p, int64_t row, bool f32, const float (&x)[8]) {
        float* const pf = static_cast<float*>(p) + row + t.at[0];
        uint16_t* const pb = static_cast<uint16_t*>(p) + row + t.at[0];
        const u32x4 w = pack8_bf16(x);
        if (skip < (a.apart ? 8 : 1)) {
            if (f32) {
                u32x4 u, v;
#pragma unroll
                for (int i = 0; i < 4; ++i) { u[i] = __float_as_uint(x[i]); v[i] = __float_as_uint(x[4 + i]); }
                reinterpret_cast<Piece16*>(pf)->v = u;
                reinterpret_cast<Piece16*>(pf + 4)->v = v;
            } else {
                reinterpret_cast<Piece16*>(pb)->v = w;
            }
        } else if (skip < 8) {
#pragma unroll
            for (int i = 1; i < 8; ++i)
                if (i >= skip) {
                    if (f32) pf[i] = x[i];
                    else pb[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                }
        }
    };
    if (post) load_or_1(t, a.post.weight, 0, a.post.dtype, 0, pw);
    load_row(r);
    for (; r < a.M; r += step) {
        const int mi = mrow, gi = grow;
        if (RES && gi >= 0 && gi != gi_of) {
            load_or_1(t, a.gate.gate, gi * a.gate.ld, a.gate.dtype, 0, ga);
            gi_of = gi;
        }
        if (mi >= 0 && mi != mi_of) {
            fold8(t, a.norm, a.mod, mi, 0, na, nc);
            mi_of = mi;
        }
        float x[8], y[8], mean, rstd;
        unpack(rx, x);
        if constexpr (RES) unpack(ry, y);
        load_row(r + step < a.M ? r + step : r);
        if constexpr (RES) {
            if (post) stats(y, a.post.kind, a.post.eps, mean, rstd);
            if (gi >= 0) {
                if (post) post8(t, y, pw, 0, mean, rstd);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __builtin_fmaf(ga[i], y[i], x[i]);
            }
            store8(a.O, r * a.ldo, sizeof(XT) == 4, x);
        }
        if (norm) {
            stats(x, a.norm.kind, a.norm.eps, mean, rstd);
            if (mi >= 0) {
                apply8(x, mean, rstd, na, nc);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.0f;
            }
            store8(a.H, r * a.ldh, a.h_dtype == MG_F32, x);
        }
    }
}

// Rows of fewer than 8 channels: a thread takes a row.
__global__ void __launch_bounds__(256) row_small_kernel(RowArgs a) {
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (r >= a.M) return;
    const int K = a.K;
    auto stats = [&](const float (&x)[7], const NormArgs& n, float& mean, float& rstd) {
        float s = 0.0f, q = 0.0f;
        for (int j = 0; j < K; ++j) s += x[j];
        mean = n.kind == MG_NORM_LAYER ? s / (float)K : 0.0f;
        for (int j = 0; j < K; ++j) q = __builtin_fmaf(x[j] - mean, x[j] - mean, q);
        rstd = rsqrt_f32(q / (float)K + n.eps);
    };
    auto norm1 = [&](float x, int j, const NormArgs& n, float mean, float rstd) {
        x = normed(x, mean, rstd);
        if (n.weight) x *= load_elem(n.weight, j, n.dtype);
        return n.bias ? x + load_elem(n.bias, j, n.dtype) : x;
    };
    auto put = [&](void* p, int64_t at, int32_t dtype, float v) {
        if (dtype == MG_F32) static_cast<float*>(p)[at] = v;
        else static_cast<uint16_t*>(p)[at] = (uint16_t)pack_bf16(v, 0.0f);
    };
    float x[7], y[7], mean, rstd;
    for (int j = 0; j < K; ++j) x[j] = load_elem(a.X, r * a.ldx + j, a.x_dtype);
    if (a.Y) {
        const int gi = mod_row(a.gate, r);
        for (int j = 0; j < K; ++j) y[j] = load_elem(a.Y, r * a.ldy + j, a.y_dtype);
        if (a.has_post) stats(y, a.post, mean, rstd);
        for (int j = 0; j < K; ++j) {
            if (gi >= 0) {
                const float b = a.has_post ? norm1(y[j], j, a.post, mean, rstd) : y[j];
                x[j] = __builtin_fmaf(a.gate.gate ? load_elem(a.gate.gate, gi * a.gate.ld + j, a.gate.dtype) : 1.0f, b, x[j]);
            }
            put(a.O, r * a.ldo + j, a.x_dtype, x[j]);
        }
    }
    if (a.has_norm) {
        const int mi = mod_row(a.mod, r);
        stats(x, a.norm, mean, rstd);
        for (int j = 0; j < K; ++j) {
            float h = 0.0f;
            if (mi >= 0) {
                h = norm1(x[j], j, a.norm, mean, rstd);
                if (a.mod.scale) h *= 1.0f + load_elem(a.mod.scale, mi * a.mod.ld + j, a.mod.dtype);
                if (a.mod.shift) h += load_elem(a.mod.shift, mi * a.mod.ld + j, a.mod.dtype);
            }
            put(a.H, r * a.ldh + j, a.h_dtype, h);
        }
    }
}

// ---- norm, modulation and the quantize step of the projection behind them

// A thread's 8 channels' smoothing scales, their reciprocals with 0 on outlier
// channels (whose bulk quotient is then +-0 and whose codes `keep` clears), and
// the bound of the fast quotient (0 where a scale is out of its range).
struct QuantLane {
    float s[8], rz[8];
    uint32_t keep, lim;
};
struct QuantRaw {                       // 32-byte pieces of the plan's vectors, loaded ahead of their use
    float4 s0, s1, r0, r1;
    int4 p0, p1;
};
__device__ __forceinline__ void quant_load(const NormQuantArgs& g, int j0, bool in, QuantRaw& q) {
    const int j = in ? j0 : 0;
    const float4* ps = reinterpret_cast<const float4*>(g.s + j);
    const float4* pr = reinterpret_cast<const float4*>(g.rcp + j);
    const int4* pp = reinterpret_cast<const int4*>(g.pos + j);
    q = QuantRaw{ps[0], ps[1], pr[0], pr[1], pp[0], pp[1]};
}
__device__ __forceinline__ void quant_make(const QuantRaw& w, bool in, QuantLane& q) {
    bool ok = true;
    q.keep = 0xFFFFFFFFu;
    const float4 s0 = w.s0, s1 = w.s1, r0 = w.r0, r1 = w.r1;
    const int4 p0 = w.p0, p1 = w.p1;
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w}, r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
    const int p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q.s[i] = in ? s[i] : 1.0f;
        const bool out = in && p[i] >= 0;
        q.rz[i] = in && !out ? r[i] : 0.0f;
        q.keep &= out ? ~(0xFu << (4 * i)) : 0xFFFFFFFFu;
        ok &= div_fast_ok_s(q.s[i]);
    }
    q.lim = ok ? kF32Pow126 : 0u;
}

__device__ __forceinline__ void quant_lane(const NormQuantArgs& g, int j0, bool in, QuantLane& q) {
    QuantRaw w;
    quant_load(g, j0, in, w);
    quant_make(w, in, q);
}

// E2M1 codes (packed, first value in the low nibble) and E8M0 code of 8 bf16
// values w of a row, 4 lanes forming a block of 32: the activation quantizer's
// arithmetic with its conditions for the fast division (k_quant.hip states
// them), and the correctly rounded division for the wave where a lane fails.
__device__ __forceinline__ uint32_t quant8(const float (&s)[8], const float (&rz)[8], uint32_t keep, uint32_t lim, u32x4 w,
                                           uint32_t& code) {
    float q[8], a0 = 0.0f, aq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t wi = w[i >> 1];
        const float x = __uint_as_float((i & 1) ? (wi & 0xFFFF0000u) : (wi << 16));
        const float q0 = x * rz[i];
        const float t = __builtin_fmaf(q0, s[i], -x);
        q[i] = __builtin_fmaf(-t, rz[i], q0);
        a0 = fmaxf(a0, __builtin_fabsf(q0));
        aq = fmaxf(aq, __builtin_fabsf(q[i]));
    }
    uint32_t qb = quad_max_bits(__float_as_uint(aq));
    const uint64_t bad = __builtin_amdgcn_uicmp(__float_as_uint(a0), lim, kCmpUGE) |
                         __builtin_amdgcn_uicmp(qb - 1u, kF32PowM74 - 1u, kCmpULT);
    if (bad) {
        aq = 0.0f;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {             // rare: kept small
            const uint32_t wi = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
            float lo = 0.0f, hi = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k == i) {
                    lo = keep >> (8 * k) & 1u ? __fdiv_rn(__uint_as_float(wi << 16), s[2 * k]) : 0.0f;
                    hi = keep >> (8 * k + 4) & 1u ? __fdiv_rn(__uint_as_float(wi & 0xFFFF0000u), s[2 * k + 1]) : 0.0f;
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                q[2 * k] = k == i ? lo : q[2 * k];
                q[2 * k + 1] = k == i ? hi : q[2 * k + 1];
            }
            aq = fmaxf(aq, fmaxf(__builtin_fabsf(lo), __builtin_fabsf(hi)));
        }
        qb = quad_max_bits(__float_as_uint(aq));
    }
    const int32_t sb = __builtin_elementwise_max((int32_t)(qb & 0x7F800000u) - (2 << 23), 0x00200000);
    const float scale = __int_as_float(sb);
    code = (uint32_t)sb >> 23;
    uint32_t word = 0;
    MG_CVT_FP4X2(word, q[0], q[1], scale, 0);
    MG_CVT_FP4X2(word, q[2], q[3], scale, 1);
    MG_CVT_FP4X2(word, q[4], q[5], scale, 2);
    MG_CVT_FP4X2(word, q[6], q[7], scale, 3);
    return word & keep;
}

// Outlier columns are formed apart from the bulk, a lane per column of XO: its
// channel's value is read again (the row has just been loaded), normed,
// rounded and divided like every other's, so 64 of them cost one wave some 40
// instructions and are stored as whole pieces.  Columns k ... 16 nso - 1 are
// pads holding 0.
struct OutlierLane {
    int j, at;                      // channel (-1: a pad column), byte offset of the column in a row's part of XO (-1: none)
    float s, a, c;
};
__device__ __forceinline__ OutlierLane outlier_lane(const NormQuantArgs& g, int col, int cols) {
    OutlierLane o;
    o.j = col < g.k ? g.O[col] : -1;
    o.at = col < cols ? (col >> 4) * kFragBlock + ((col >> 3) & 1) * 512 + 2 * (col & 7) : -1;
    o.s = o.j >= 0 ? g.s[o.j] : 1.0f;
    o.a = 0.0f;
    o.c = 0.0f;
    return o;
}
// a and c of its channel, as fold8 forms them
__device__ __forceinline__ void outlier_fold(OutlierLane& o, const FoldArgs& f, int row) {
    const int j = o.j < 0 ? 0 : o.j;
    float a = 1.0f, c = 0.0f;
    if (f.mod.scale) a = 1.0f + load_elem(f.mod.scale, row * f.mod.ld + j, f.mod.dtype);
    if (f.mod.shift) c = load_elem(f.mod.shift, row * f.mod.ld + j, f.mod.dtype);
    if (f.norm.bias) c = __builtin_fmaf(load_elem(f.norm.bias, j, f.norm.dtype), a, c);
    if (f.norm.weight) a *= load_elem(f.norm.weight, j, f.norm.dtype);
    o.a = a;
    o.c = c;
}
__device__ __forceinline__ void outlier_put(const OutlierLane& o, float x, float mean, float rstd, bool pad, uint8_t* xo) {
    if (o.at < 0) return;
    const float h = __builtin_fmaf(normed(x, mean, rstd), o.a, o.c);
    const float q = __fdiv_rn(bf16_to_f32(pack_bf16(h, 0.0f) & 0xFFFFu), o.s);
    *reinterpret_cast<uint16_t*>(xo + o.at) = o.j < 0 || pad ? 0 : (uint16_t)f32_to_bf16_rne(q);
}
template <typename XT>
__device__ __forceinline__ float outlier_x(const XT* row, const OutlierLane& o) {
    return o.j < 0 ? 0.0f : load_elem(row, o.j, sizeof(XT) == 4 ? MG_F32 : MG_BF16);
}

// A unit's rows r0 ... r0 + R - 1 from their staged codes (`live` of them; zeros
// for pad rows) to Aq and As, and the pad rows of XO, by T threads: 16-byte
// pieces, rows fastest, R of them contiguous in memory.
template <int FIXED>
__device__ __forceinline__ void flush_unit(const NormQuantArgs& g, int64_t r0, int live, int64_t M32, int64_t ns4, int64_t nso,
                                           int nwin, const uint8_t* stA, int rowA, const uint8_t* stS, int rowS, int T,
                                           int R_ = FIXED) {
    const int R = FIXED ? FIXED : R_, sh = FIXED ? 3 : 31 - __builtin_clz(R), tid = threadIdx.x;
    const int rows = M32 - r0 < R ? (M32 > r0 ? (int)(M32 - r0) : 0) : R;
    const u32x4 zero = {0, 0, 0, 0};
    uint8_t* const aq = g.Aq + (r0 >> 5) * ns4 * kFragBlock + ((r0 & 31) << 4);
#pragma unroll 2
    for (int i = tid; i < (int)ns4 * 2 * R; i += T) {
        const int rr = i & (R - 1), line = i >> sh;
        if (rr < rows)
            *reinterpret_cast<u32x4*>(aq + (line >> 1) * kFragBlock + (line & 1) * 512 + rr * 16) =
                rr < live ? *reinterpret_cast<const u32x4*>(stA + rr * rowA + line * 16) : zero;
    }
    uint8_t* const as = g.As + (r0 / kScRows) * nwin * kScWinBytes + (r0 % kScRows) * kScBlocks;
#pragma unroll 1
    for (int i = tid; i < nwin * R; i += T) {
        const int rr = i & (R - 1), win = i >> sh;
        *reinterpret_cast<u32x4*>(as + (int64_t)win * kScWinBytes + rr * kScBlocks) =
            rr < live ? *reinterpret_cast<const u32x4*>(stS + rr * rowS + win * 16) : zero;
    }
    if (live < rows) {
        uint8_t* const xo = g.XO + (r0 >> 5) * nso * kFragBlock + ((r0 & 31) << 4);
#pragma unroll 1
        for (int i = tid; i < (int)nso * 2 * R; i += T) {
            const int rr = i & (R - 1), line = i >> sh;
            if (rr >= live && rr < rows)
                *reinterpret_cast<u32x4*>(xo + (line >> 1) * kFragBlock + (line & 1) * 512 + rr * 16) = zero;
        }
    }
}

// Norm, modulation, rounding to bf16 and the quantize step.  A workgroup takes
// units of R consecutive rows (8 where there are enough: whole 128-byte lines
// of the operand's fragment blocks and scale windows).  Each row's codes are
// staged in LDS and a unit's rows leave together.  Rows are row_kernel's, with
// the same sums, so the codes are those of its bf16 output quantized.
// Bound: for the few rows it runs, latency: the row, the statistics, the
// coefficients' loads, the division and the blocks' maxima one after the other:
// one row of 5120 7.7 us, 256 rows 8.9 us.  From more rows on the form below
// is faster (32760 x 5120 f32: 352 us here); its 10 windows a row are the most
// that registers hold, so wider rows stay here (8000 x 13824 bf16 113 us, 2.5
// TB/s).
template <int V, typename XT>
__global__ void __launch_bounds__(V <= 4 ? 512 : 1024) __attribute__((amdgpu_waves_per_eu(V > 4 ? 4 : V == 4 ? 2 : V == 2 ? 3 : 4)))
norm_quant_kernel(NormQuantArgs g, int R) {
    constexpr bool KEEP = V <= 4;
    __shared__ Pairs pairs;
    extern __shared__ __attribute__((aligned(16))) uint8_t stage[];   // R rows: codes (256 bytes a window, 16 pad), scales (16)
    int turn = 0;
    const RowArgs& a = g.r;
    const int K = a.K, nwin = (int)sc_nwin(K), lane = (int)threadIdx.x & 63;
    const RowThread<V, false> t(K);
    const XT* X = static_cast<const XT*>(a.X);
    const int64_t ns4 = frag_slices(K / 2), nso = frag_slices(2 * (int64_t)g.k);
    const int64_t M = a.M, M32 = (M + 31) / 32 * 32, Mp = (M + kScRows - 1) / kScRows * kScRows;
    const int rowA = nwin * 256 + 16, rowS = nwin * 16, cols = 16 * (int)nso;
    uint8_t* const stS = stage + (size_t)R * rowA;
    float na[KEEP ? V : 1][8], nc[KEEP ? V : 1][8];
    QuantLane ql[KEEP ? V : 1];
    int mi_of = -1, mrow = -1;
    Raw8<XT> rx[V];
    auto load_row = [&](int64_t r) {
        r = r < M ? r : M - 1;
#pragma unroll
        for (int v = 0; v < V; ++v) load_raw(X + r * a.ldx + t.at[v], rx[v]);
        mrow = mod_row(a.mod, r);
    };
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t r0 = (int64_t)blockIdx.x * R;
    if (r0 >= M) {                                                    // pad rows only
        for (; r0 < Mp; r0 += step) flush_unit<0>(g, r0, 0, M32, ns4, nso, nwin, stage, rowA, stS, rowS, t.T, R);
        return;
    }
    if constexpr (KEEP) {
        load_row(r0);
#pragma unroll
        for (int v = 0; v < V; ++v) quant_lane(g, t.col[v], t.col[v] < K, ql[v]);
    }
    OutlierLane ol = outlier_lane(g, 64 * t.wave + lane, cols);       // this wave's first 64 columns
    for (; r0 < Mp; r0 += step) {
        const int live = r0 >= M ? 0 : M - r0 < R ? (int)(M - r0) : R;
        for (int rr = 0; rr < live; ++rr) {
            const int64_t r = r0 + rr;
            if constexpr (!KEEP) load_row(r);
            const int mi = __builtin_amdgcn_readfirstlane(mrow);
            if (mi >= 0 && mi != mi_of) {
                const FoldArgs f = fold_args();
                if constexpr (KEEP) fold_all(t, f.norm, f.mod, mi, na, nc);
                outlier_fold(ol, f, mi);
                mi_of = mi;
            }
            float x[V][8];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                unpack(rx[v], x[v]);
                t.own(v, x[v]);
            }
            const float xo0 = outlier_x(X + r * a.ldx, ol);
            if constexpr (KEEP) load_row(rr + 1 < live ? r + 1 : r0 + step);
            float mean, rstd;
            row_stats(x, t, a.norm.kind, a.norm.eps, pairs, turn, mean, rstd);
            uint8_t* const xo = g.XO + (r >> 5) * nso * kFragBlock + ((r & 31) << 4);
            outlier_put(ol, xo0, mean, rstd, mi < 0, xo);
#pragma unroll 1
            for (int c = 64 * (t.wave + t.W); c < cols; c += 64 * t.W) {
                OutlierLane o = outlier_lane(g, c + lane, cols);
                if (mi >= 0) outlier_fold(o, fold_args(), mi);
                outlier_put(o, outlier_x(X + r * a.ldx, o), mean, rstd, mi < 0, xo);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int win = v * t.W + t.wave;
                if (win >= nwin) continue;                            // whole waves
                if constexpr (!KEEP) {
                    const FoldArgs f = fold_args();
                    fold8(t, f.norm, f.mod, mi < 0 ? 0 : mi, v, na[0], nc[0]);
                    quant_lane(g, t.col[v], t.col[v] < K, ql[0]);
                }
                apply8(x[v], mean, rstd, na[KEEP ? v : 0], nc[KEEP ? v : 0]);
                u32x4 w = pack8_bf16(x[v]);
                if (mi < 0 || !(t.full >> v & 1u)) {                  // K % 32 == 0: whole blocks
                    const bool on = mi >= 0 && t.col[v] < K;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = on ? w[i] : 0u;
                }
                uint32_t code;
                const QuantLane& L = ql[KEEP ? v : 0];
                const uint32_t word = quant8(L.s, L.rz, L.keep, L.lim, w, code);
                *reinterpret_cast<uint32_t*>(stage + rr * rowA + win * 256 + 4 * lane) = word;
                if ((lane & 3) == 0) stS[rr * rowS + win * 16 + sc_pos(lane >> 2)] = (uint8_t)code;
            }
        }
        if (live) __syncthreads();                                    // the unit's codes are staged
        flush_unit<0>(g, r0, live, M32, ns4, nso, nwin, stage, rowA, stS, rowS, t.T, R);
    }
}

// The same with a row per wave, for up to 5120 channels and many rows: the
// per-channel constants (a, c, s, 1 / s: 16 bytes a channel) lie in LDS, once
// for the 8 waves of the workgroup, a row needs no barrier and one wave's
// bookkeeping instead of W waves', and its registers are refilled window by
// window with the next row.  V: windows of 512 channels, of which only the
// last can be partial.  The sums are row_kernel's (those of its W waves), so
// the bits are.
// Bound: memory and the arithmetic of the quantize step together: 32760 x 5120
// f32 (764 MB) 161-167 us, 4.6-4.7 TB/s; bf16 (428 MB, 84 us at a copy's rate)
// 123 us, 3.5, where the arithmetic is likely the longer part.  A row per W waves with
// the constants in registers took 352 us and 322 us, dividing the outlier
// channels with the others 238 us and 198 us.
template <int V>
struct WaveShape {
    static constexpr int W = V <= 8 ? V : (V + 1) / 2;             // row_kernel's waves (and one or two vectors) for V windows
    static constexpr int rowA = V * 256 + 16, rowS = V * 16;       // staged bytes of a row: codes, scales
    static constexpr int consts = V * 64 * 136;                    // a, c, s, rz, and keep and lim
    static constexpr int lds = consts + 2 * 8 * (rowA + rowS);
};
template <int V, typename XT>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2))) norm_quant_wave_kernel(NormQuantArgs g) {
    using S = WaveShape<V>;
    extern __shared__ __attribute__((aligned(16))) uint8_t stage[];
    float4* const ka = reinterpret_cast<float4*>(stage);              // [array a, c, s, rz][window][half][lane]
    uint2* const kk = reinterpret_cast<uint2*>(stage + V * 64 * 128);  // [window][lane] keep, lim
    uint8_t* const st = stage + S::consts;
    const RowArgs& a = g.r;
    const int K = a.K, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const XT* X = static_cast<const XT*>(a.X);
    const int64_t ns4 = frag_slices(K / 2), nso = frag_slices(2 * (int64_t)g.k);
    const int64_t M = a.M, M32 = (M + 31) / 32 * 32, Mp = (M + kScRows - 1) / kScRows * kScRows;
    const int cols = 16 * (int)nso;
    const bool last_in = 512 * (V - 1) + 8 * lane < K;               // the lane's channels of the last window exist
    auto slot = [&](int arr, int win, int half, int l) -> float4& { return ka[((arr * V + win) * 2 + half) * 64 + l]; };
    auto put8 = [&](int arr, int win, int l, const float (&v)[8]) {
        slot(arr, win, 0, l) = make_float4(v[0], v[1], v[2], v[3]);
        slot(arr, win, 1, l) = make_float4(v[4], v[5], v[6], v[7]);
    };
    auto get8 = [&](int arr, int win, float (&v)[8]) {
        const float4 x = slot(arr, win, 0, lane), y = slot(arr, win, 1, lane);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    };
    // a thread's place as fold8 needs it: one vector at a time
    RowThread<1, false> t(K);
    auto at_window = [&](int win, int l) {
        t.col[0] = (win * 64 + l) * 8;
        t.at[0] = t.col[0] < K - 8 ? t.col[0] : K - 8;
    };
    for (int i = tid; i < V * 64; i += 512) {
        QuantLane q;
        quant_lane(g, i * 8, i * 8 < K, q);
        put8(2, i >> 6, i & 63, q.s);
        put8(3, i >> 6, i & 63, q.rz);
        kk[i] = make_uint2(q.keep, q.lim);
    }
    OutlierLane ol = outlier_lane(g, lane, cols);
    // channels of row_kernel's wave w: windows w, w + W, ...
    auto count = [&](int w) {
        int c = 0;
#pragma unroll
        for (int v = 0; v * S::W < V; ++v) {
            const int l = K - 512 * (v * S::W + w);
            c += l < 0 ? 0 : l < 512 ? l : 512;
        }
        return c;
    };
    const int cl = (lane & 15) < S::W ? count(lane & 15) : 0;
    const float nl = (float)cl, rnl = cl ? 1.0f / (float)cl : 0.0f, rK = 1.0f / (float)K;
    const bool layer = a.norm.kind == MG_NORM_LAYER;
    const float eps = a.norm.eps;
    int loaded = -1, turn = 0;
    Raw8<XT> rx[V];
    auto load_win = [&](const XT* row, int v) {
        const int col = 512 * v + 8 * lane;
        load_raw(row + (v < V - 1 || col < K - 8 ? col : K - 8), rx[v]);
    };
    auto row_at = [&](int64_t r) { return X + (r < M ? r : M - 1) * a.ldx; };
    const int64_t step = (int64_t)gridDim.x * 8;
    int64_t r0 = (int64_t)blockIdx.x * 8;
    {
        const XT* row = row_at(r0 + wave);
#pragma unroll
        for (int v = 0; v < V; ++v) load_win(row, v);
    }
    float xo0 = outlier_x(row_at(r0 + wave), ol);
    auto mod_rows = [&](int64_t r) { return lane < 8 && r + lane < M ? mod_row(a.mod, r + lane) : -1; };
    int mis = mod_rows(r0);
    // every wave reads what all of them have put into LDS above; a first unit of
    // padding rows meets no barrier of the modulation's below
    __syncthreads();
    for (; r0 < Mp; r0 += step) {
        const int64_t r = r0 + wave;
        const int live = r0 >= M ? 0 : M - r0 < 8 ? (int)(M - r0) : 8;
        const int mi = __builtin_amdgcn_readlane(mis, wave);
        const uint64_t some = __builtin_amdgcn_ballot_w64(mis >= 0);
        const int want = some ? __builtin_amdgcn_readlane(mis, __builtin_ctzll(some)) : loaded;
        mis = mod_rows(r0 + step);
        if (want != loaded) {           // the same in every wave
            __syncthreads();
            const FoldArgs f = fold_args();
#pragma unroll 1
            for (int i = tid; i < V * 64; i += 512) {
                float na[8], nc[8];
                at_window(i >> 6, i & 63);
                fold8(t, f.norm, f.mod, want, 0, na, nc);
                put8(0, i >> 6, i & 63, na);
                put8(1, i >> 6, i & 63, nc);
            }
            outlier_fold(ol, f, want);
            __syncthreads();
            loaded = want;
        }
        uint8_t* const stA = st + turn * 8 * (S::rowA + S::rowS), * const stS = stA + 8 * S::rowA;
        if (wave < live) {
            float x[V][8];
#pragma unroll
            for (int v = 0; v < V; ++v) unpack(rx[v], x[v]);
            // sums of row_kernel's waves, step by step side by side
            float sw[S::W], qw[S::W], m[S::W];
            auto sums = [&](float (&u)[S::W]) {
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = dpp_add<0xB1, 0xF>(u[w]);
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = dpp_add<0x4E, 0xF>(u[w]);
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = dpp_add<0x141, 0xF>(u[w]);
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = dpp_add<0x140, 0xF>(u[w]);
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = dpp_add<0x142, 0xA>(u[w]);
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = dpp_add<0x143, 0xC>(u[w]);
#pragma unroll
                for (int w = 0; w < S::W; ++w) u[w] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(u[w]), 63));
            };
#pragma unroll
            for (int w = 0; w < S::W; ++w) {
                sw[w] = 0.0f;
                m[w] = 0.0f;
                if (layer) {
#pragma unroll
                    for (int v = w; v < V; v += S::W)
#pragma unroll
                        for (int i = 0; i < 8; ++i) sw[w] += v < V - 1 || last_in ? x[v][i] : 0.0f;
                }
            }
            if (layer) {
                sums(sw);
#pragma unroll
                for (int w = 0; w < S::W; ++w) {
                    const int c = count(w);
                    m[w] = sw[w] * (c ? 1.0f / (float)c : 0.0f);
                }
            }
#pragma unroll
            for (int w = 0; w < S::W; ++w) {
                qw[w] = 0.0f;
#pragma unroll
                for (int v = w; v < V; v += S::W)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float d = v < V - 1 || last_in ? x[v][i] - m[w] : 0.0f;
                        qw[w] = __builtin_fmaf(d, d, qw[w]);
                    }
            }
            sums(qw);
            float s = 0.0f, q = 0.0f;   // of wave (lane % 16)
#pragma unroll
            for (int w = 0; w < S::W; ++w) {
                s = (lane & 15) == w ? sw[w] : s;
                q = (lane & 15) == w ? qw[w] : q;
            }
            const float mean = layer ? mean_of(row16_sum(s), K, rK) : 0.0f;
            const float d = __builtin_fmaf(s, rnl, -mean);
            const float rstd = rsqrt_f32(__builtin_fmaf(row16_sum(__builtin_fmaf(nl * d, d, q)), rK, eps));
            uint8_t* const xo = g.XO + (r >> 5) * nso * kFragBlock + ((r & 31) << 4);
            const bool own = mi != loaded && mi >= 0;                 // another modulation row than the unit's
            {
                OutlierLane o = ol;
                if (own) outlier_fold(o, fold_args(), mi);
                outlier_put(o, xo0, mean, rstd, mi < 0, xo);
#pragma unroll 1
                for (int c = 64; c < cols; c += 64) {
                    o = outlier_lane(g, c + lane, cols);
                    if (mi >= 0) outlier_fold(o, fold_args(), mi);
                    outlier_put(o, outlier_x(row_at(r), o), mean, rstd, mi < 0, xo);
                }
                xo0 = outlier_x(row_at(r + step), ol);
            }
            const XT* next = row_at(r + step);
            uint8_t* const stw = stA + wave * S::rowA + 4 * lane;
            uint8_t* const sts = stS + wave * S::rowS + sc_pos(lane >> 2);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float na[8], nc[8];
                if (own) {
                    const FoldArgs f = fold_args();
                    at_window(v, lane);
                    fold8(t, f.norm, f.mod, mi, 0, na, nc);
                } else {
                    get8(0, v, na);
                    get8(1, v, nc);
                }
                apply8(x[v], mean, rstd, na, nc);
                u32x4 w = pack8_bf16(x[v]);
                load_win(next, v);
                if (v == V - 1 || mi < 0) {
                    const bool on = mi >= 0 && (v < V - 1 || last_in);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = on ? w[i] : 0u;
                }
                float s8[8], rz[8];
                get8(2, v, s8);
                get8(3, v, rz);
                const uint2 kl = kk[v * 64 + lane];
                uint32_t code;
                const uint32_t word = quant8(s8, rz, kl.x, kl.y, w, code);
                *reinterpret_cast<uint32_t*>(stw + v * 256) = word;
                if ((lane & 3) == 0) sts[v * 16] = (uint8_t)code;
            }
        }
        // one barrier a unit: the next unit stages into the other half, and is
        // past its barrier only when every wave has left this one's
        if (live) __syncthreads();
        turn ^= 1;
        flush_unit<8>(g, r0, live, M32, ns4, nso, V, stA, S::rowA, stS, S::rowS, 512);
    }
}

// Waves and vectors per thread for rows of K channels: 512 channels a wave and
// vector, up to 8 waves, then more vectors, then more waves.  At equal
// bytes one vector was as fast as any from 512 to 4096 channels, and 5120 as
// fast with 10 waves of one as with 5 of two (residual 38.7 and 38.9 us).
struct Shape { int W, V; };
Shape shape_of(int32_t K) {
    const int nw = (K + 511) / 512;
    const int need = (nw + 7) / 8, V = need <= 2 ? need : need <= 4 ? 4 : 8;
    return Shape{(nw + V - 1) / V, V};
}

template <typename F>
hipError_t by_v(int V, F&& f) {
    switch (V) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        default: return f(std::integral_constant<int, 8>{});
    }
}

// Workgroups of `threads` threads and `lds` bytes of a kernel that run on the
// device at once, looked up once per device, kernel and size.
int64_t resident(const void* kern, int threads, int lds) {
    struct Entry { const void* k; int threads, lds, dev, n; };
    static thread_local Entry cache[96] = {};
    static thread_local int used = 0;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return device_cu_count();
    for (int i = 0; i < used; ++i)
        if (cache[i].k == kern && cache[i].threads == threads && cache[i].lds == lds && cache[i].dev == dev) return cache[i].n;
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, lds) != hipSuccess || n < 1) n = 1;
    n *= device_cu_count();
    if (used < 96) cache[used++] = Entry{kern, threads, lds, dev, n};
    return n;
}

// Workgroups of W waves of a row kernel that run on a CU at once.  A workgroup
// starts only where every SIMD takes ceil(W / 4) more waves, and a SIMD takes
// 6 waves of these kernels at most (their scalar registers): a grid that
// leaves workgroups to a second round costs more than one with fewer.  Norm
// of 11973 x 5120 bf16 (W = 5, 4 waves a SIMD): 46 us with 2 workgroups a CU,
// 55 us with the 3 that 16 waves would hold.
int64_t row_groups(const void* kern, int W) {
    const int64_t per = resident(kern, 64, 0) / device_cu_count() / 4, waves = per < 6 ? (per > 1 ? per : 1) : 6;
    const int64_t n = W % 4 ? (4 * waves - (W + 3) / 4 * 4) / W + 1 : 4 * waves / W;
    return n > 1 ? n : 1;
}

template <int V, typename XT, typename YT>
hipError_t run_rows(const RowArgs& a, int W, hipStream_t st) {
    const auto kern = row_kernel<V, XT, YT>;
    int64_t n = row_groups(reinterpret_cast<const void*>(kern), W);
    // Memory is read fastest with about 18 KB of rows on their way to each CU:
    // with 30000 rows of 2048, residual bf16 89 us with 2 workgroups a CU
    // (16 KB), 97 us with 4; f32 150 us with 1 (16 KB), 168 us with 2 or 3.
    // More workgroups pay for few rows (4099 rows, bf16: 18.1 us with 2, 17.0
    // us with 4) and where a row waits longer, for a norm after the block or a
    // partial vector (9973 rows of 2048 with it: 42 us with 2, 36 us with 4;
    // 9973 rows of 2049: 57 us with 2, 47 us with 3).
    if (a.M >= 32 * (int64_t)device_cu_count() && !a.has_post && a.K % 8 == 0) {
        const int64_t row = a.K * (int64_t)(sizeof(XT) + (RowShape<V, XT, YT>::res ? sizeof(typename RowShape<V, XT, YT>::Y) : 0));
        const int64_t best = (18 * 1024 + row / 2) / row;
        if (n > best) n = best > 1 ? best : 1;
    }
    const int64_t most = n * device_cu_count();
    // consecutive rows where modulation rows may change often: a workgroup that
    // meets every group forms its coefficients once for each (4099 x 1537 of 7
    // samples: 12.6 us, spread 16.2; with one modulation row the spread rows
    // read memory about 5 % faster)
    const int64_t chunk = (a.M + most - 1) / most;
    const int64_t group = a.mod.group < a.gate.group ? a.mod.group : a.gate.group;
    const bool same = !a.mod.index && !a.gate.index && (a.M + group - 1) / group * 8 <= chunk + 8;
    const int64_t blocks = same ? (a.M < most ? a.M : most) : (a.M + chunk - 1) / chunk;
    constexpr int per = RowShape<V, XT, YT>::lds_thread;
    if constexpr (per != 0) {
        static thread_local int configured_dev = -1;
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess) return hipErrorNoDevice;
        if (configured_dev != dev) {
            const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, 512 * per);
            if (e != hipSuccess) return e;
            configured_dev = dev;
        }
    }
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(64 * W), 64 * W * per, st, a, RowSpan{chunk, same ? blocks : 1});
    return hipGetLastError();
}

template <int LANES, typename XT, typename YT>
hipError_t run_narrow(const RowArgs& a, hipStream_t st) {
    const auto kern = row_narrow_kernel<LANES, XT, YT>;
    constexpr int ROWS = 256 / LANES;
    const int64_t most = row_groups(reinterpret_cast<const void*>(kern), 4) * device_cu_count(), units = (a.M + ROWS - 1) / ROWS;
    hipLaunchKernelGGL(kern, dim3((unsigned)(units < most ? units : most)), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int V, typename XT>
hipError_t run_quant(const NormQuantArgs& a, int W, hipStream_t st) {
    const auto kern = norm_quant_kernel<V, XT>;
    const int nwin = (int)sc_nwin(a.r.K), row = nwin * 272 + 16;       // staged bytes of a row
    // 8 rows a unit where that leaves every CU a unit, fewer for few rows
    int R = 8;
    while (R > 1 && ((a.r.M + R - 1) / R < device_cu_count() || R * row > 128 * 1024)) R >>= 1;
    const int lds = R * row;
    static thread_local int configured_dev = -1;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return hipErrorNoDevice;
    if (configured_dev != dev) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
        if (e != hipSuccess) return e;
        configured_dev = dev;
    }
    const int64_t most = resident(reinterpret_cast<const void*>(kern), 64 * W, lds);
    const int64_t units = (a.r.M + kScRows - 1) / kScRows * kScRows / R;
    hipLaunchKernelGGL(kern, dim3((unsigned)(units < most ? units : most)), dim3(64 * W), lds, st, a, R);
    return hipGetLastError();
}

template <int V, typename XT>
hipError_t run_quant_wave(const NormQuantArgs& a, hipStream_t st) {
    const auto kern = norm_quant_wave_kernel<V, XT>;
    constexpr int lds = WaveShape<V>::lds;
    static thread_local int configured_dev = -1;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return hipErrorNoDevice;
    if (configured_dev != dev) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        configured_dev = dev;
    }
    const int64_t most = resident(reinterpret_cast<const void*>(kern), 512, lds);
    const int64_t units = (a.r.M + kScRows - 1) / kScRows * (kScRows / 8);
    hipLaunchKernelGGL(kern, dim3((unsigned)(units < most ? units : most)), dim3(512), lds, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rows(const RowArgs& args, hipStream_t st) {
    RowArgs a = args;
    struct Range { uintptr_t lo, hi; };
    auto range = [&](const void* p, int64_t ld, int32_t dtype) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        return Range{lo, p ? lo + (uintptr_t)((a.M - 1) * ld + a.K) * (dtype == MG_F32 ? 4 : 2) : lo};
    };
    const Range in[2] = {range(a.X, a.ldx, a.x_dtype), range(a.Y, a.ldy, a.y_dtype)};
    const Range out[2] = {range(a.O, a.ldo, a.x_dtype), range(a.H, a.ldh, a.h_dtype)};
    a.apart = 1;
    for (const Range& i : in)
        for (const Range& o : out)
            if (i.lo < o.hi && o.lo < i.hi) a.apart = 0;
    if (a.K < 8) {
        hipLaunchKernelGGL(row_small_kernel, dim3((unsigned)((a.M + 255) / 256)), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    const bool xf = a.x_dtype == MG_F32, yf = a.y_dtype == MG_F32;
    if (a.K <= 256) {
        auto run = [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            if (a.Y == nullptr) return xf ? run_narrow<L, float, void>(a, st) : run_narrow<L, uint16_t, void>(a, st);
            if (xf) return yf ? run_narrow<L, float, float>(a, st) : run_narrow<L, float, uint16_t>(a, st);
            return yf ? run_narrow<L, uint16_t, float>(a, st) : run_narrow<L, uint16_t, uint16_t>(a, st);
        };
        return a.K <= 128 ? run(std::integral_constant<int, 16>{}) : run(std::integral_constant<int, 32>{});
    }
    const Shape sh = shape_of(a.K);
    return by_v(sh.V, [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (a.Y == nullptr)
            return xf ? run_rows<V, float, void>(a, sh.W, st) : run_rows<V, uint16_t, void>(a, sh.W, st);
        if (xf) return yf ? run_rows<V, float, float>(a, sh.W, st) : run_rows<V, float, uint16_t>(a, sh.W, st);
        return yf ? run_rows<V, uint16_t, float>(a, sh.W, st) : run_rows<V, uint16_t, uint16_t>(a, sh.W, st);
    });
}

hipError_t launch_norm_quant(const NormQuantArgs& a, hipStream_t st) {
    const Shape sh = shape_of(a.r.K);
    // A row per wave once every CU has rows enough for the constants in LDS to
    // pay: measured at K = 5120, 1560 rows 13.6 us against 26.9, 384 rows 11.5
    // against 14.8, 256 rows 11.6 against 8.9; at K = 4096, 1560 rows 12.1
    // against 14.0, 768 rows 10.7 against 9.8.
    const int nw = (a.r.K + 511) / 512;
    if (a.r.M > (nw > 8 ? 1 : 4) * (int64_t)device_cu_count() && nw <= 10) {
        const bool xf = a.r.x_dtype == MG_F32;
        switch (nw) {
#define MG_WAVE(V) case V: return xf ? run_quant_wave<V, float>(a, st) : run_quant_wave<V, uint16_t>(a, st)
            MG_WAVE(1); MG_WAVE(2); MG_WAVE(3); MG_WAVE(4); MG_WAVE(5); MG_WAVE(6); MG_WAVE(7); MG_WAVE(8); MG_WAVE(9); MG_WAVE(10);
#undef MG_WAVE
        }
    }
    return by_v(sh.V, [&](auto v) {
        constexpr int V = decltype(v)::value;
        return a.r.x_dtype == MG_F32 ? run_quant<V, float>(a, sh.W, st) : run_quant<V, uint16_t>(a, sh.W, st);
    });
}

}  // namespace mg
