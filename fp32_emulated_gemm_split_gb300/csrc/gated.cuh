// gated.cuh -- device code of the gated feed-forward H = act(G) * U shared by
// the GEMM's epilogue and the backward kernel: the activations, their
// derivatives, and the epilogue that turns a thread's sums of both
// projections into H (and stores G and U for the backward pass).
#pragma once

#include "emu_device.cuh"

namespace emu {

constexpr float kSqrtHalf = 0.70710678118654752f;       // sqrt(1/2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;     // 1 / sqrt(2 pi)
constexpr float kSqrt2OverPi = 0.79788456080286536f;    // sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// s = 1 / (1 + e^-g) and c = 1 - s, each without cancellation: with
// t = e^-|g| <= 1 the larger of the two is 1 / (1 + t), the smaller t / (1 + t).
__device__ __forceinline__ void sigmoid_pair(float g, float& s, float& c) {
    const float t = expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + t), tr = t * r;
    s = g < 0.0f ? tr : r;
    c = g < 0.0f ? r : tr;
}

// act(g), every step in FP32.
//   silu       g s(g),  s(g) = 1 / (1 + e^-g)
//   gelu       g erfc(-g / sqrt 2) / 2    (= g (1 + erf(g / sqrt 2)) / 2)
//   gelu_tanh  g s(2 z),  z = sqrt(2/pi) (g + 0.044715 g^3)
//              (= g (1 + tanh z) / 2, as (1 + tanh z) / 2 = 1 / (1 + e^-2z))
//   relu       max(g, 0), NaN kept;   sigmoid  s(g)
// (the forms with erfc and s keep their accuracy for negative g, where 1 +
// erf and 1 + tanh cancel)
// (g / d is __fdividef's: 2 ulp; d = 1 + e^x reaches its limit of 2^126 only
// where the quotient is below 1e-36, and is 0 there)
template <int ACT>
__device__ __forceinline__ float gated_act(float g) {
    if constexpr (ACT == kActSilu) return __fdividef(g, 1.0f + expf(-g));
    if constexpr (ACT == kActGelu) return 0.5f * g * erfcf(-g * kSqrtHalf);
    if constexpr (ACT == kActGeluTanh)
        return __fdividef(g, 1.0f + expf(-2.0f * kSqrt2OverPi * fmaf(kGeluCubic * g * g, g, g)));
    if constexpr (ACT == kActRelu) return g < 0.0f ? 0.0f : g;
    return __fdividef(1.0f, 1.0f + expf(-g));
}

// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ float2 gated_act_grad(float g) {
    float s, c;
    if constexpr (ACT == kActSilu) {
        sigmoid_pair(g, s, c);
        return make_float2(g * s, s * fmaf(g, c, 1.0f));
    }
    if constexpr (ACT == kActGelu) {
        s = 0.5f * erfcf(-g * kSqrtHalf);
        return make_float2(g * s, fmaf(g * kInvSqrt2Pi, expf(-0.5f * g * g), s));
    }
    if constexpr (ACT == kActGeluTanh) {
        sigmoid_pair(2.0f * kSqrt2OverPi * fmaf(kGeluCubic * g * g, g, g), s, c);
        const float dz = kSqrt2OverPi * fmaf(3.0f * kGeluCubic * g, g, 1.0f);
        return make_float2(g * s, s * fmaf(2.0f * g * c, dz, 1.0f));
    }
    if constexpr (ACT == kActRelu) return make_float2(g < 0.0f ? 0.0f : g, g > 0.0f ? 1.0f : 0.0f);
    sigmoid_pair(g, s, c);
    return make_float2(s, s * c);
}

// f(activation as a compile-time constant): the choice is made once around a
// whole loop.  Made per element it put the code of all five beside every one
// of an unrolled loop's elements, and the epilogues waited for instructions
// (22 us of a 78 us kernel at 24 x 4096 x (2 x 8192)).
template <int V>
struct Const {
    static constexpr int value = V;
};
template <typename F>
__host__ __device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case kActSilu: f(Const<kActSilu>{}); break;
        case kActGelu: f(Const<kActGelu>{}); break;
        case kActGeluTanh: f(Const<kActGeluTanh>{}); break;
        case kActRelu: f(Const<kActRelu>{}); break;
        default: f(Const<kActSigmoid>{}); break;
    }
}

// Store 32 rows x 16 columns of one output (lane = row, v[0..15]) whose tile
// starts at (row0, gc0): through the warp's 2 KB staging buffer and one bulk
// tensor store where the output's rows are 16-byte aligned (64-byte swizzle;
// the map ends at column N & ~3, so a lane stores its row's last N % 4
// columns itself), turned in that buffer otherwise.
__device__ __forceinline__ void store_chunk16(const float (&v)[16], const CUtensorMap& map,
                                              bool tma, float* out, int64_t ld, int M, int N,
                                              int row0, int gc0, int lane, uint32_t stage) {
    // the buffer is free again (either way: the output before may have gone by a
    // bulk store where this one does not)
    if (lane == 0) bulk_wait_read_n<0>();
    if (!tma) {
        store_unaligned16(v, 0.0f, out, ld, M, N, row0, gc0, lane, stage);
        return;
    }
    const int row = row0 + lane;
    const int n4 = N & ~3;
    {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t a = stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4);
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};"
                         :: "r"(a), "f"(v[4 * c]), "f"(v[4 * c + 1]), "f"(v[4 * c + 2]),
                            "f"(v[4 * c + 3]) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            if (gc0 < n4) tma_store_2d(&map, gc0, row0, stage);
            bulk_commit();
        }
    }
    if (row < M) {
        float* dst = out + (int64_t)row * ld;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int c = gc0 + j;
            if (c < N && c >= n4) dst[c] = v[j];
        }
    }
}

// The gated epilogue of one tile for one warp: acc[j] (j < C / 2) are column
// col0 + j of the gate for this lane's row, acc[C / 2 + j] the same columns
// of the up projection.
template <int C>
__device__ __forceinline__ void gated_epilogue(const float (&acc)[C], const TcGemmParams& p,
                                               const CUtensorMap& mapH, const CUtensorMap& mapG,
                                               const CUtensorMap& mapU, int row0, int lane,
                                               int col0, uint32_t stage) {
    if (row0 >= p.M) return;
#pragma unroll
    for (int ch = 0; ch < C / 32; ++ch) {
        const int gc = col0 + 16 * ch;
        if (gc >= p.N) break;                            // warp-uniform
        float h[16];
        with_act(p.act, [&](auto a) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                h[j] = gated_act<decltype(a)::value>(acc[16 * ch + j]) * acc[C / 2 + 16 * ch + j];
        });
        store_chunk16(h, mapH, p.tma_store, p.C, p.ldc, p.M, p.N, row0, gc, lane, stage);
        if (p.G) {
#pragma unroll
            for (int j = 0; j < 16; ++j) h[j] = acc[16 * ch + j];
            store_chunk16(h, mapG, p.tma_gu, p.G, p.ldg, p.M, p.N, row0, gc, lane, stage);
#pragma unroll
            for (int j = 0; j < 16; ++j) h[j] = acc[C / 2 + 16 * ch + j];
            store_chunk16(h, mapU, p.tma_gu, p.U, p.ldg, p.M, p.N, row0, gc, lane, stage);
        }
    }
}

// Few rows of X (gemm_few.cu): acc[j] is element (weight row m, X row col0 + j),
// stored at C[(col0 + j) * ldc + m]: a warp writes 32 neighbouring values of
// each row of C.
template <int C>
__device__ __forceinline__ void few_epilogue(const float (&acc)[C], const TcGemmParams& p, int m,
                                              int col0) {
    if (m >= p.M) return;
    float* c = p.C + (int64_t)col0 * p.ldc + m;
    // eight rows' old values of C at a time, before their stores (a store
    // between two loads would hold the second one back)
#pragma unroll
    for (int j0 = 0; j0 < C; j0 += 8) {
        float old[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            old[j] = p.beta != 0.0f && col0 + j0 + j < p.N ? c[(int64_t)(j0 + j) * p.ldc] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = p.alpha * acc[j0 + j];
            if (col0 + j0 + j < p.N)
                c[(int64_t)(j0 + j) * p.ldc] = p.beta != 0.0f ? fmaf(p.beta, old[j], v) : v;
        }
    }
}

// Gated: the tile's sums of `rows` rows of X from row j0 are in shared memory,
// 128 values each, the gate's 64 columns from f0, then the up projection's.
// Thread t of n takes every n-th element: a warp writes 32 neighbouring values
// of H.
__device__ __forceinline__ void few_gated_epilogue(const TcGemmParams& p, const float* ex, int f0,
                                                   int j0, int rows, int t, int n) {
    with_act(p.act, [&](auto a) {
#pragma unroll 2
        for (int e = t; e < 64 * rows; e += n) {
            const int j = e >> 6, f = e & 63;
            const float g = ex[j * 128 + f], u = ex[j * 128 + 64 + f];
            if (f0 + f < p.M) {
                p.C[(int64_t)(j0 + j) * p.ldc + f0 + f] = gated_act<decltype(a)::value>(g) * u;
                if (p.G) {
                    p.G[(int64_t)(j0 + j) * p.ldg + f0 + f] = g;
                    p.U[(int64_t)(j0 + j) * p.ldg + f0 + f] = u;
                }
            }
        }
    });
}

}  // namespace emu
