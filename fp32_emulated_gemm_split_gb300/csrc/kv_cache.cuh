// kv_cache.cuh -- what the kernels over the 8-bit keys and values share
// (kv_cache.cu, kv_attention.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "emu_layers.h"

namespace emu {

constexpr int64_t kKvMaxRows = (int64_t(1) << 25) - 1;       // rows of one call

// Sizes, alignments and pointers of a cache.
bool kv_cache_ok(const emu_kv_cache_t& c);

inline int kv_log2(int64_t n) {
    int l = 0;
    while ((int64_t(1) << l) < n) ++l;
    return l;
}

__device__ __forceinline__ float kv_f32(float x) { return x; }
__device__ __forceinline__ float kv_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float kv_f32(__half x) { return __half2float(x); }
// the two 16-bit values of a word
template <typename T> __device__ __forceinline__ void kv_widen(uint32_t w, float& lo, float& hi);
template <> __device__ __forceinline__ void kv_widen<__nv_bfloat16>(uint32_t w, float& lo, float& hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
}
template <> __device__ __forceinline__ void kv_widen<__half>(uint32_t w, float& lo, float& hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
}

template <typename T> __device__ __forceinline__ T kv_from(float x);
template <> __device__ __forceinline__ float kv_from<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 kv_from<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half kv_from<__half>(float x) { return __float2half_rn(x); }

// 8 neighbouring values; wide: they start on 16 bytes.
template <typename T>
__device__ __forceinline__ void kv_load8(const T* at, bool wide, float* x) {
    if (wide) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + 4);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(at);
            kv_widen<T>(a.x, x[0], x[1]);
            kv_widen<T>(a.y, x[2], x[3]);
            kv_widen<T>(a.z, x[4], x[5]);
            kv_widen<T>(a.w, x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = kv_f32(at[i]);
    }
}

template <typename T>
__device__ __forceinline__ void kv_store8(T* at, bool wide, const float (&x)[8]) {
    if (wide) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(at + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            T y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = kv_from<T>(x[i]);
            uint4 w;
            memcpy(&w, y, 16);
            *reinterpret_cast<uint4*>(at) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i] = kv_from<T>(x[i]);
    }
}

// Two e4m3 codes as FP16 values: exact (e4m3 has 4 significant bits and
// exponents -6..8, its subnormal values reach 2^-9), NaN stays NaN.
__device__ __forceinline__ uint32_t kv_half2(uint16_t codes) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(codes));
    return d;
}

// Four values, |x| <= 448 or NaN, rounded to codes (the first in the low byte).
__device__ __forceinline__ uint32_t kv_codes(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Four codes times `ratio`, rounded again.
__device__ __forceinline__ uint32_t kv_rescale(uint32_t w, float ratio) {
    float x[4];
    kv_widen<__half>(kv_half2((uint16_t)w), x[0], x[1]);
    kv_widen<__half>(kv_half2((uint16_t)(w >> 16)), x[2], x[3]);
    return kv_codes(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
}

}  // namespace emu
