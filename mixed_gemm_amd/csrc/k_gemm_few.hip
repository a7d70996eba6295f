// The dual GEMM with its epilogue for few token rows, where the 4-bit weights
// are the traffic and the 256x256 tiles of the large kernel leave most of the
// chip idle: small output tiles, and K split over the waves of a workgroup.
//
// A workgroup takes TG groups of 32 tokens by NG groups of 32 columns; wave w
// takes every NW-th half-window of K (256 channels: four 64-channel slices,
// whose scale codes are one 32-bit word per row and half) and every NW-th
// slice of the outlier columns.  Operands are in fragment order, so a slice of
// 32 rows is one 16-byte load per lane of 1 KB of contiguous memory straight
// into the matrix instruction's registers: nothing passes through LDS, no
// barrier stands in the K loop, and a wave keeps 4 D slices per row group in
// flight.  Loads of rows past M or N and of slices past K leave the buffers'
// ranges and read 0.  The waves' partial sums meet in LDS and are added in the
// order of the waves, so a call's bits do not vary.
//
// Bound: the weights' way into the CUs.  One token, K = 5120 -> N = 13824 (37.6
// MB of codes and scales) takes 10.3 us and 13824 -> 5120 11.3 us where ten
// plans take turns and the weights come from memory (3.7 and 3.3 TB/s), 8.3 and
// 8.4 us with one plan, which the last-level cache holds, against 3.2 us for a
// 1568 x 1056 layer; all inside a graph.  With more tokens the
// operands' way into a CU (few_tile).  Fewer registers pay more than more
// loads in flight: 4 waves with one or two half-windows leave room for two to
// three workgroups on a CU, whose starts and joins overlap the others' K loops
// (8 waves with three half-windows: 1.2 to 1.6 times as long from 32 tokens on).
#include "gemm_epilogue.h"
#include "mg_block.h"
#include "mg_device.h"
#include "mg_internal.h"

namespace mg {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

struct FewArgs {
    const uint8_t* Aq;
    const uint8_t* As;
    const uint16_t* XO;
    const uint8_t* Wq;
    const uint8_t* Ws;
    const uint16_t* WO;
    void* Y;
    int64_t M;
    int32_t N, K, k;
    EpArgs ep;
};

template <int OPSEL>
__device__ __forceinline__ v16f few_fp4(ep_u32x4 w, ep_u32x4 a, uint32_t sw, uint32_t sa, v16f c) {
    const v8i wv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const v8i av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, c, 4, 4, OPSEL, (int)sw, OPSEL, (int)sa);
}

// 16 bytes at lane offset voff plus wave offset soff, which always lies inside
// the buffer; without `ok` the lane offset leaves it and 0 is read.
__device__ __forceinline__ ep_u32x4 few_load(__amdgpu_buffer_rsrc_t r, bool ok, uint32_t voff, uint32_t soff) {
    return __builtin_bit_cast(ep_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, ok ? voff : kEpNowhere, ok ? soff : 0u, 0));
}
__device__ __forceinline__ uint32_t few_load1(__amdgpu_buffer_rsrc_t r, bool ok, uint32_t voff, uint32_t soff) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, ok ? voff : kEpNowhere, ok ? soff : 0u, 0);
}

// TG groups of 32 tokens by NG groups of 32 columns per workgroup, NW waves
// that split K, D half-windows in flight per wave.
template <typename YT, int TG, int NG, int NW, int D>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4))) gemm_few(FewArgs g) {
    extern __shared__ __attribute__((aligned(16))) float part[];      // [NW][32][ROW]
    constexpr bool YF = std::is_same_v<YT, float>;
    constexpr int ROW = 32 * NG + 4;                                  // floats per staged row
    constexpr int PR = 8 * NG;                                        // pieces of 4 columns per token
    constexpr int RS = 64 * NW / PR;                                  // token rows the workgroup takes at once
    constexpr int PT = (32 + RS - 1) / RS;                            // pieces per thread and token group
    constexpr bool EARLY = TG == 1 && PT == 1;                        // epilogue inputs loaded ahead of the K loop
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = g.K, N = g.N;
    const int64_t M = g.M;
    const EpArgs& e = g.ep;
    // workgroups go round-robin to the 8 XCDs: each takes an equal run of the
    // tiles, token blocks fastest (those of a column block share its weights)
    const int gy = (int)((M + 32 * TG - 1) / (32 * TG));
    const int tile = ((int)blockIdx.x & 7) * ((int)gridDim.x >> 3) + ((int)blockIdx.x >> 3);
    const int bx = tile / gy, by = tile - bx * gy;
    const int n0 = bx * 32 * NG;
    if (n0 >= N) return;
    const int64_t t0 = (int64_t)by * 32 * TG;

    // ---- the epilogue's inputs: a thread's columns are the same in every row it takes
    const int prow = tid / PR, pcol = n0 + 4 * (tid % PR);
    const bool pon = prow < (RS < 32 ? RS : 32) && pcol < N;
    float bias[4] = {}, gate[PT][4], res[PT][4];
    int mi[PT];
    auto ep_inputs = [&](int t) {
#pragma unroll
        for (int p = 0; p < PT; ++p) {
            const int64_t m = t0 + 32 * t + p * RS + prow;
            const bool on = pon && p * RS + prow < 32 && m < M;
            mi[p] = on ? mod_row(e.mod, m) : -1;
#pragma unroll
            for (int c = 0; c < 4; ++c) { gate[p][c] = 1.0f; res[p][c] = 0.0f; }
            if (on && e.residual) ep_load4(e.residual, m * e.ldr + pcol, e.residual_dtype == MG_F32, res[p]);
            if (e.mod.gate && mi[p] >= 0) ep_load4(e.mod.gate, (int64_t)mi[p] * e.mod.ld + pcol, e.mod.dtype == MG_F32, gate[p]);
        }
    };
    if (e.bias && pon) ep_load4(e.bias, pcol, e.bias_dtype == MG_F32, bias);
    if constexpr (EARLY) ep_inputs(0);

    // ---- this wave's part of K
    const uint32_t ns4 = (uint32_t)frag_slices(K / 2);
    const int units = (int)(ns4 + 3) / 4;                             // half-windows
    const uint32_t nwin = (uint32_t)sc_nwin(K);
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.Aq, (uint64_t)frag_bytes(M, K / 2));
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.Wq, (uint64_t)frag_bytes(N, K / 2));
    const __amdgpu_buffer_rsrc_t rAs = make_rsrc(g.As, (uint64_t)sc_bytes(M, K));
    const __amdgpu_buffer_rsrc_t rBs = make_rsrc(g.Ws, (uint64_t)sc_bytes(N, K));
    const uint32_t l16 = 16u * (uint32_t)lane;
    uint32_t offA[TG], offAs[TG], offB[NG], offBs[NG];
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        const int64_t m = t0 + 32 * t + l32;                          // absent tokens read 0
        offA[t] = m < M ? (uint32_t)(m / 32) * ns4 * kFragBlock + l16 : kEpNowhere;
        offAs[t] = m < M ? (uint32_t)(m / kScRows) * nwin * kScWinBytes + (uint32_t)((m % kScRows) * kScBlocks + 8 * h) : kEpNowhere;
    }
#pragma unroll
    for (int c = 0; c < NG; ++c) {
        const int n = n0 + 32 * c + l32;
        offB[c] = n < N ? (uint32_t)(n / 32) * ns4 * kFragBlock + l16 : kEpNowhere;
        offBs[c] = n < N ? (uint32_t)(n / kScRows) * nwin * kScWinBytes + (uint32_t)((n % kScRows) * kScBlocks + 8 * h) : kEpNowhere;
    }

    v16f acc[TG][NG];
#pragma unroll
    for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int c = 0; c < NG; ++c) acc[t][c] = v16f{};
    ep_u32x4 w[D][NG][4], a[D][TG][4];
    uint32_t sw[D][NG], sa[D][TG];
    // slice s of half-window u, and the half-window's scale codes, into
    // register set d.  Slices past the last read 0 (no memory is touched), so
    // the loop needs no branches: a wave's surplus half-windows add 0.
    auto load_slice = [&](int u, int d, int s) {
        const uint32_t sl = 4u * (uint32_t)u + (uint32_t)s;
        const bool ok = sl < ns4;
#pragma unroll
        for (int c = 0; c < NG; ++c) w[d][c][s] = few_load(rB, ok, offB[c], sl * kFragBlock);
#pragma unroll
        for (int t = 0; t < TG; ++t) a[d][t][s] = few_load(rA, ok, offA[t], sl * kFragBlock);
    };
    auto load_scales = [&](int u, int d) {
        const uint32_t so = (uint32_t)(u >> 1) * kScWinBytes + 4u * (u & 1);
        const bool ok = u < units;
#pragma unroll
        for (int c = 0; c < NG; ++c) sw[d][c] = few_load1(rBs, ok, offBs[c], so);
#pragma unroll
        for (int t = 0; t < TG; ++t) sa[d][t] = few_load1(rAs, ok, offAs[t], so);
    };
    // ---- outlier columns: slices of 16 bf16 values, every NW-th a wave's.
    // The first is asked for ahead of the bulk and multiplied behind its loads.
    const uint32_t nso = (uint32_t)frag_slices(2 * (int64_t)g.k);
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(g.XO, (uint64_t)frag_bytes(M, 2 * (int64_t)g.k));
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(g.WO, (uint64_t)frag_bytes(N, 2 * (int64_t)g.k));
    ep_u32x4 ww[NG], x[TG];
    auto load_outlier = [&](uint32_t s) {
#pragma unroll
        for (int c = 0; c < NG; ++c)
            ww[c] = few_load(rW, n0 + 32 * c < N, l16, ((uint32_t)(n0 / 32 + c) * nso + s) * kFragBlock);
#pragma unroll
        for (int t = 0; t < TG; ++t)
            x[t] = few_load(rX, t0 + 32 * t < M, l16, (((uint32_t)(t0 / 32) + t) * nso + s) * kFragBlock);
    };
    auto use_outlier = [&]() {
#pragma unroll
        for (int t = 0; t < TG; ++t)
#pragma unroll
            for (int c = 0; c < NG; ++c)
                acc[t][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, ww[c]),
                                                                    __builtin_bit_cast(v8bf, x[t]), acc[t][c], 0, 0, 0);
    };
    if ((uint32_t)wave < nso) load_outlier((uint32_t)wave);
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load_scales(wave + d * NW, d);
#pragma unroll
        for (int s = 0; s < 4; ++s) load_slice(wave + d * NW, d, s);
    }
    if ((uint32_t)wave < nso) use_outlier();
    for (uint32_t s = (uint32_t)wave + NW; s < nso; s += NW) {
        load_outlier(s);
        use_outlier();
    }
    // D half-windows of the wave, refilling each slice's registers (REFILL) as
    // soon as it is multiplied
    int u0 = wave;
    auto round = [&](auto REFILL) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int next = u0 + (d + D) * NW;
            // the next scale codes are asked for ahead of the next slices, so
            // that waiting for them does not wait for those
            uint32_t cw[NG], ca[TG];
#pragma unroll
            for (int c = 0; c < NG; ++c) cw[c] = sw[d][c];
#pragma unroll
            for (int t = 0; t < TG; ++t) ca[t] = sa[d][t];
            if constexpr (decltype(REFILL)::value) load_scales(next, d);
            auto slice = [&](auto S) {
                constexpr int s = decltype(S)::value;
#pragma unroll
                for (int t = 0; t < TG; ++t)
#pragma unroll
                    for (int c = 0; c < NG; ++c)
                        acc[t][c] = few_fp4<s>(w[d][c][s], a[d][t][s], cw[c], ca[t], acc[t][c]);
                if constexpr (decltype(REFILL)::value) {
                    load_slice(next, d, s);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            slice(std::integral_constant<int, 0>{});
            slice(std::integral_constant<int, 1>{});
            slice(std::integral_constant<int, 2>{});
            slice(std::integral_constant<int, 3>{});
        }
    };
    for (; u0 + D * NW < units; u0 += D * NW) round(std::true_type{});
    round(std::false_type{});
    // ---- join and epilogue, one token group at a time: register 4 q + i of
    // lane (l32, h) is token l32, column 8 q + 4 h + i of its 32
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        if constexpr (!EARLY) ep_inputs(t);
        if (t > 0) __syncthreads();                                   // the sums of the last group are taken
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<ep_f32x4*>(part + (size_t)(wave * 32 + l32) * ROW + 32 * c + 8 * q + 4 * h) =
                    ep_f32x4{acc[t][c][4 * q], acc[t][c][4 * q + 1], acc[t][c][4 * q + 2], acc[t][c][4 * q + 3]};
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PT; ++p) {
            const int64_t m = t0 + 32 * t + p * RS + prow;
            if (!pon || p * RS + prow >= 32 || m >= M) continue;
            float v[4] = {};
#pragma unroll
            for (int x = 0; x < NW; ++x) {
                const ep_f32x4 s = *reinterpret_cast<const ep_f32x4*>(part + (size_t)(x * 32 + p * RS + prow) * ROW + 4 * (tid % PR));
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] += s[c];
            }
            ep_by_act(e.act, [&](auto A) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = ep_act<decltype(A)::value>(v[c] + bias[c]);
            });
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = mi[p] < 0 ? res[p][c] : __builtin_fmaf(gate[p][c], v[c], res[p][c]);
            YT* y = static_cast<YT*>(g.Y) + m * N + pcol;
            if constexpr (YF) *reinterpret_cast<ep_f32x4*>(y) = ep_f32x4{v[0], v[1], v[2], v[3]};
            else *reinterpret_cast<ep_u32x2*>(y) = ep_u32x2{ep_pack(v[0], v[1]), ep_pack(v[2], v[3])};
        }
    }
}

template <typename YT, int TG, int NG, int NW, int D>
hipError_t launch_few(const FewArgs& a, hipStream_t st) {
    constexpr int lds = NW * 32 * (32 * NG + 4) * 4;
    static thread_local int configured_dev = -1;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return hipErrorNoDevice;
    if (configured_dev != dev) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gemm_few<YT, TG, NG, NW, D>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        configured_dev = dev;
    }
    const int64_t gx = (a.N + 32 * NG - 1) / (32 * NG), gy = (a.M + 32 * TG - 1) / (32 * TG);
    hipLaunchKernelGGL((gemm_few<YT, TG, NG, NW, D>), dim3((unsigned)((gx * gy + 7) / 8 * 8)), dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename YT>
hipError_t run_few(int tile, const FewArgs& a, hipStream_t st) {
    switch (tile) {
        case 0: return launch_few<YT, 1, 1, 4, 2>(a, st);
        case 1: return launch_few<YT, 1, 2, 4, 1>(a, st);
        case 2: return launch_few<YT, 2, 2, 4, 1>(a, st);
        default: return launch_few<YT, 2, 3, 4, 1>(a, st);
    }
}

}  // namespace

// The tile expected to be fastest, from a model of each one's time (us): a start,
// and for every round of workgroups that the CUs make, the operands' way from
// L2 (16 (tg + ng) bytes a channel; an outlier channel counts for 2 to 4, its
// values take 4 times the bytes), what a workgroup spends outside its
// K loop, and its output's and residual's way (`bytes` an element).  The
// 256x256 tiles make their rounds one workgroup a CU; an incomplete round
// leaves memory to the fewer outputs.  Fitted to 200 measured calls (M 24 to
// 12000, K and N 256 to 13824, k 0 to 128, bias and GELU into bf16, gate and
// residual in f32), whose choices lie 1.1 % above the best tile's time, 30 % at
// worst; without k and the output's bytes 7.6 %, 150 % at worst (11496 tokens,
// 416 -> 7552: 75 us with 256x256 tiles, 190 us with (2, 3)).  Measured against the 256x256 tiles, gate
// and residual in bf16, one plan in the last-level cache: 5120 -> 13824 at 1, 64, 256, 384 tokens 8.3, 10.7, 24.5,
// 32.0 (33.4, 33.8, 35.6, 37.6), 13824 -> 5120 at 1, 64, 256, 1024 tokens 8.4,
// 12.7, 22.9, 67.9 (72.9, 73.5, 74.8, 77.0), 1568 -> 1056 at 777 tokens 6.6
// (19.6).
int few_tile(int64_t M, int32_t N, int32_t K, int32_t k, int bytes) {
    static const struct { int tg, ng; double start, own, chan, outlier, out, rest; } tiles[] = {
        {1, 1, 3.3, 0.50, 2.00e-4, 2.4, 0.0167, 0.10},
        {1, 2, 3.5, 0.51, 1.72e-4, 4.2, 0.0197, 0.65},
        {2, 2, 3.2, 1.62, 1.87e-4, 3.9, 0.0197, 0.98},
        {2, 3, 4.0, 2.72, 1.78e-4, 4.1, 0.0143, 0.91}};
    const double cus = device_cu_count();
    const double big = (double)((M + 255) / 256) * (double)((N + 255) / 256);
    const double full = big < cus ? big / cus : 1.0;
    double best = 9.3 + __builtin_ceil(big / cus) * (K * 0.00488 + k * 0.0212 + 0.97 + full * 3.49 * bytes);
    int tile = -1;
    for (int i = 0; i < 4; ++i) {
        const auto& f = tiles[i];
        const double wgs = (double)((M + 32 * f.tg - 1) / (32 * f.tg)) * (double)((N + 32 * f.ng - 1) / (32 * f.ng));
        // up to 3 workgroups share a CU and run their rounds together; then they stagger
        const double r = wgs / cus, rounds = r <= 3.0 ? __builtin_ceil(r) : r + f.rest;
        const double t = f.start + rounds * (f.chan * (K + f.outlier * k) * (f.tg + f.ng) + f.own + f.out * f.tg * f.ng * bytes);
        if (t < best) {
            best = t;
            tile = i;
        }
    }
    return tile;
}

hipError_t launch_dual_gemm_few(const uint8_t* Aq, const uint8_t* As, const uint16_t* XO, const uint8_t* Wq,
                                const uint8_t* Ws, const uint16_t* WO, int64_t M, int32_t N, int32_t K, int32_t k,
                                const EpArgs& e, void* Y, int32_t y_dtype, int tile, hipStream_t st) {
    const FewArgs a{Aq, As, XO, Wq, Ws, WO, Y, M, N, K, k, e};
    return y_dtype == MG_F32 ? run_few<float>(tile, a, st) : run_few<uint16_t>(tile, a, st);
}

}  // namespace mg
