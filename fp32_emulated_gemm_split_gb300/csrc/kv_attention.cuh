// kv_attention.cuh -- what the two kernels of the attention over 8-bit keys and
// values share: kv_attention.cu's for few rows of a sequence, kv_prompt.cu's for many.
#pragma once

#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"
#include "kv_cache.cuh"

namespace emu {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKvSlotRows = 256;                     // rows of a segment at most

struct Work;
struct AttnParams {
    const void* q;
    void* out;
    int64_t q_t, q_h, out_t, out_h;
    int T, heads, group, D, page_log, B, width, window;
    const uint8_t *k, *v;
    const float *ks, *vs;
    int64_t pages;
    const int32_t *table, *starts, *lengths;
    float scale;
    int wide, wide_out;                              // rows of q, of out on 16 bytes
    int depth, side;                                 // stages of a warp's ring, bytes of a stage's keys (or values)
    int copy_tokens;                                 // tokens of one tensor copy
    float* partial;                                  // [2 ctas][slot_rows][D + 4]
    float4* moved;                                   // sums of o in memory, kv_prompt.cu: [SMs][2 groups][D / 4][128 rows]
    int slot_rows;
    Work* shared;                             // [ctas]: the segment that a CTA begins and others end (or units 0)
    int* err;
};

// A sequence of the batch: its rows (none where `starts` is not in order), and its
// length, -1 where that is out of range.
struct Seq {
    int start, n, len;
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int b) {
    Seq s;
    s.start = p.starts[b];
    const int end = p.starts[b + 1];
    s.n = s.start >= 0 && end >= s.start && end <= p.T ? end - s.start : 0;
    s.len = p.lengths[b];
    if (s.len < 0 || s.len > (int64_t)p.width << p.page_log) s.len = -1;
    return s;
}
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// (lo, hi) minus its FP16 rounding h
__device__ __forceinline__ uint32_t half2_rest(float lo, float hi, uint32_t h) {
    float a, b;
    kv_widen<__half>(h, a, b);
    return half2_bits(lo - a, hi - b);
}

// Of four codes: the bytes that are NaN (0x7F, 0xFF), all bits set.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xFFu;
}

// What a row's scores are multiplied with, before the keys' scale: `scale` and log2 e, and 2^(E - 14), the inverse of what its
// queries were. NaN where a query is infinite (top): its scores are infinities or NaN, and no softmax of those is a number.
__device__ __forceinline__ float score_factor(float top, int E, float scale) {
    return top <= 3.402823466e38f ? __uint_as_float((uint32_t)(E - 14 + 127) << 23) * (scale * kLog2e)
                                  : __uint_as_float(0x7FC00000u);
}

// A bound of log2 of a page's value scale less 14 (its exponent and one, less 14), and no less than -120, so that
// 2^(the other way) is finite, and so is the sum of 128 of them: what o is held against lies this far from the
// scores' maximum.
__device__ __forceinline__ int scale_bound(float v_scale) {
    return max((int)((__float_as_uint(v_scale) >> 23) & 0xFF) - 126 - 14, -120);
}

// A weight p s_v against o's reference is x f, x = 2^(score - m), f = s_v 2^(m - ref).  It is 2^14 at most, but where the
// row's largest scores are those of pages of a tiny scale (of zeros: 2^-126), m lies up to 120 over ref, and the f of
// another page is infinite.  From here on x is 2^(score - ref), f s_v, and sums of x count 2^(ref - m) of themselves.
constexpr float kFarScale = 1e37f, kFarValue = 7.0f;     // no f over the first with an s_v up to the second

// A CTA's way through the units, and the segment that it is at (in shared memory: both are
// looked at between segments only).
struct Work {
    int64_t all, ctas;                               // units, CTAs that share them
    int64_t at, stop;                                // the CTA's next unit, the end of its range
    int64_t base;                                    // units of the sequences before `seq`
    int64_t begin, end;                              // the segment's units
    int seq, start, len, pos0;                       // sequence, its first row, its length, position of its first row
    int head, row0, rows;                            // the segment's key head, first row of the sequence, rows
    int token0, units;                               // of the CTA's part: first token, units
    bool bad, starts, whole;                         // no length; the part has the segment's first unit, all of them
};

// What a row's sums are multiplied with: maximum m, sum of weights l, reference ref.
__device__ __forceinline__ float row_factor(bool bad, float m, float l, float ref) {
    return bad ? __uint_as_float(0x7FC00000u) : l > 0.0f || l != l ? exp2_of(ref - m) / l : 0.0f;
}
// Four values of a row from its sums.
template <typename T>
__device__ __forceinline__ void write_row(const AttnParams& p, const Work& w, int r, int d, float m, float l, float ref, float4 v) {
    const int row = w.row0 + r, i = row / p.group;
    const float f = row_factor(w.bad, m, l, ref);
    T* to = static_cast<T*>(p.out) + (w.start + i) * p.out_t + (w.head * p.group + row - i * p.group) * p.out_h + d;
    to[0] = kv_from<T>(v.x * f);
    to[1] = kv_from<T>(v.y * f);
    to[2] = kv_from<T>(v.z * f);
    to[3] = kv_from<T>(v.w * f);
}
// Part sums: v += x y.
__device__ __forceinline__ void add_to(float4& v, float x, const float4& y) {
    v.x = fmaf(y.x, x, v.x);
    v.y = fmaf(y.y, x, v.y);
    v.z = fmaf(y.z, x, v.z);
    v.w = fmaf(y.w, x, v.w);
}
// What a part counts: of its weights' sum and of its o (one that saw nothing has no weight; NaN stays).
__device__ __forceinline__ float weight_of(float m, float l, float m_all) {
    return m > -INFINITY || l != 0.0f ? exp2_of(m - m_all) : 0.0f;
}
__device__ __forceinline__ float share_of(float ref, float ref_all) {
    return ref > -INFINITY ? exp2_of(ref - ref_all) : 1.0f;
}

// Launches kv_join_kernel (kv_attention.cu) behind the kernel that wrote the parts, of a grid of `ctas`.
cudaError_t launch_join(int dtype, const AttnParams& p, unsigned ctas, unsigned rows, cudaStream_t stream);

// Many rows of a sequence (kv_prompt.cu), D up to 128.
cudaError_t launch_prompt(int dtype, const AttnParams& p, int64_t max_rows, int sms, cudaStream_t stream);

}  // namespace emu
