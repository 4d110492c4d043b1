// kv_attention.cu -- causal attention over keys and values kept in 8 bits
// (emu_kv_attention, include/emu_layers.h).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  k_j = s_k K_j, v_j = s_v V_j
//   over the tokens j that the query's position sees, K and V e4m3 codes, s_k and
//   s_v a number for each page and head
//
// A code is an FP16 value (4 significant bits, exponents -6..8), so one FP16 piece
// of K and V is exact, and FP32 queries and weights p need two pieces each, hi +
// lo (22 to 24 bits), where a product of two FP32 operands would need nine of three:
// S = q_hi K + q_lo K, O = p_hi V + p_lo V, FP32 sums.  BF16 and FP16 queries are
// exact in one piece (a row is scaled by a power of two so that its largest value
// lies in 2^14..2^15; what falls below 2^-24 there is 2^-39 of the largest), and
// their outputs take p in one piece, rounded to 11 bits where the output keeps 8 or
// 11.  The page's s_v goes into p before its rounding: p s_v is held against a
// reference of its own, the running maximum of log2(p s_v), so that p keeps its
// bits however far the pages' scales are apart.
//
// Next tokens and drafts: bound by reading the cache.  The work is cut into units
// of kUnit tokens of one sequence and key head for 16 rows (a key head's query
// heads, of one token after another); the CTAs take equal consecutive ranges of all
// units.  A range's first and last segment may be shared with neighbours: their
// sums go to a slot in memory and the last one to arrive adds them up in order, so
// the result does not depend on who is last.  Within a CTA each warp takes every
// kWarps-th tile of 16 tokens (always inside one page) through a ring of its own,
// filled by asynchronous copies: no barrier but at a segment's end.
#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"
#include "kv_cache.cuh"

namespace emu {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16;                            // tokens of a warp's step
constexpr int kUnit = kTile * kWarps;
constexpr int kRows = 16;                            // rows of a segment
constexpr int kKvCtasPerSm = 3;
constexpr float kLog2e = 1.4426950408889634f;

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
    int wide;                                        // rows of q on 16 bytes
    float* partial;                                  // [2 ctas][kRows][D + 4]
    unsigned* arrived;                               // [ctas], zero between calls
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
// Tiles start on 16 tokens; the first one that any row of the sequence sees.
__device__ __forceinline__ int first_tile_token(const AttnParams& p, const Seq& s) {
    if (!p.window) return 0;
    return max(0, s.len - s.n - p.window + 1) & ~(kTile - 1);
}
__device__ __forceinline__ int units_of(const AttnParams& p, const Seq& s) {       // of one segment
    return max(1, (s.len - first_tile_token(p, s) + kUnit - 1) / kUnit);
}
__device__ __forceinline__ int64_t all_units(const AttnParams& p, const Seq& s) {  // of the sequence
    const int64_t rows = (int64_t)s.n * p.group;
    return (rows + kRows - 1) / kRows * p.heads * units_of(p, s);
}

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Codes in shared memory: rows of NG x 64 bytes, their 16-byte pieces c at c ^
// f(row), so that a quarter warp's reads of K (two rows, four pieces each) and a
// half warp's of V (four rows two apart, two pieces each) meet all banks.
template <int NG>
__device__ __forceinline__ uint32_t piece_at(int row, int c) {
    const int f = NG % 2 == 0 ? (row & 1) << 2 ^ (row >> 1 & 3) << 1 : (row >> 1 & 1) << 1;
    return row * (NG * 64) + ((c ^ f) << 4);
}

template <int NG>
struct Ring {
    static constexpr int side = kTile * NG * 64;     // a tile of K or of V
    static constexpr int stage = 2 * side + 16;      // and the two scales
    static constexpr int depth = NG <= 2 ? 4 : 3;
    static constexpr int warp = depth * stage;
    static constexpr int joined = kWarps * kRows * (NG * 64 + 4) * 4;              // the warps' sums
    static constexpr int bytes = kWarps * warp > joined ? kWarps * warp : joined;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}

// Of four codes: the bytes that are NaN (0x7F, 0xFF), all bits set.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return ((((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u) * 0xFFu;
}

template <typename T, int NG>
__global__ void __launch_bounds__(kThreads) kv_decode_kernel(const AttnParams p) {
    constexpr bool TWO = sizeof(T) == 4;             // two pieces of q and of p
    constexpr int PIECES = TWO ? 2 : 1;
    using R = Ring<NG>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t warp_sum[kWarps];
    __shared__ int64_t found_base;
    __shared__ int found_seq;
    __shared__ unsigned order;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int P = 1 << p.page_log;
    uint8_t* const ring = smem + warp * R::warp;

    // all units, and where this CTA's range of them begins: a run of sequences per thread
    const int per = (p.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, p.B); ++b) {
        const Seq s = seq_of(p, b);
        mine += all_units(p, s);
        if (blockIdx.x == 0 && (s.len < 0 || p.starts[b + 1] < s.start || s.start < 0 || p.starts[b + 1] > p.T))
            record_error(p.err, kDevErrValue);
    }
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) sum += warp_sum[w];
        all += warp_sum[w];
    }
    // rows behind the last sequence
    {
        const int used = p.B > 0 ? min(max(p.starts[p.B], 0), p.T) : 0;
        const int values = p.heads * p.group * p.D;
        for (int row = used + blockIdx.x; row < p.T; row += gridDim.x)
            for (int e = tid; e < values; e += kThreads) {
                const int h = e / p.D;
                static_cast<T*>(p.out)[row * p.out_t + h * p.out_h + (e - h * p.D)] = kv_from<T>(0.0f);
            }
    }
    // (no more of them than units: each has one at least)
    const int64_t ctas = min((int64_t)gridDim.x, all);
    if (blockIdx.x >= ctas) return;
    int64_t at = all * blockIdx.x / ctas;
    const int64_t stop = all * (blockIdx.x + 1) / ctas;
    int64_t before = sum - mine;
    if (before <= at && at < sum) {
        int b = tid * per;
        for (;; ++b) {
            const int64_t w = all_units(p, seq_of(p, b));
            if (at < before + w) break;
            before += w;
        }
        found_seq = b;
        found_base = before;
    }
    __syncthreads();
    int b = found_seq;
    int64_t base = found_base;

    while (at < stop) {
        Seq s = seq_of(p, b);
        int64_t w = all_units(p, s);
        while (at >= base + w) {
            base += w;
            s = seq_of(p, ++b);
            w = all_units(p, s);
        }
        const bool bad = s.len < 0;
        if (bad) s.len = 0;
        const int units = units_of(p, s);
        const int seg = (int)((at - base) / units);  // q tile * heads + head
        const int64_t seg_begin = base + (int64_t)seg * units, seg_end = seg_begin + units;
        const int u0 = (int)(at - seg_begin), u1 = (int)(min(stop, seg_end) - seg_begin);
        const int head = seg % p.heads, row0 = seg / p.heads * kRows;
        const int rows = min(kRows, s.n * p.group - row0);
        const int pos0 = s.len - s.n;                // position of the sequence's first new token
        // tokens that some row of the segment sees
        const int sees_end = max(0, min(s.len, pos0 + (row0 + rows - 1) / p.group + 1));
        const int sees_begin = p.window ? max(0, pos0 + row0 / p.group - p.window + 1) : 0;
        const int tile0 = first_tile_token(p, s) + u0 * kUnit + warp * kTile;
        const int tiles = (u1 - u0);                 // of this warp, kUnit tokens apart
        const int32_t* pages = p.table + (int64_t)b * p.width;
        const float nan = __uint_as_float(0x7FC00000u);

        // copies of the warp's tile i; page: its page as the table has it
        auto page_of = [&](int i) {
            const int tok = tile0 + i * kUnit;
            return i < tiles && tok < sees_end && tok + kTile > sees_begin ? pages[tok >> p.page_log] : 0;
        };
        auto copy_tile = [&](int i, int page) {
            const int tok = tile0 + i * kUnit;
            if (i < tiles && tok < sees_end && tok + kTile > sees_begin) {
                const uint32_t dst = smem_u32(ring) + i % R::depth * R::stage;
                const bool ok = page >= 0 && page < p.pages;
                const int64_t unit = (int64_t)(ok ? page : 0) * p.heads + head;
                const int64_t from = ((unit << p.page_log) + (tok & (P - 1))) * p.D;
#pragma unroll
                for (int c = lane; c < kTile * NG * 4; c += 32) {
                    const int row = c / (NG * 4), piece = c % (NG * 4);
                    const bool in = ok && tok + row >= sees_begin && tok + row < sees_end && piece * 16 < p.D;
                    const int64_t off = in ? from + row * p.D + piece * 16 : 0;
                    const uint32_t to = dst + piece_at<NG>(row, piece);
                    copy16(to, p.k + off, in);
                    copy16(to + R::side, p.v + off, in);
                }
                if (lane < 2) {
                    const uint32_t to = dst + 2 * R::side + 4 * lane;
                    if (ok) copy4(to, (lane ? p.vs : p.ks) + unit);
                    else {
                        asm volatile("st.shared.f32 [%0], %1;" :: "r"(to), "f"(nan) : "memory");
                        record_error(p.err, kDevErrValue);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int next_page[R::depth];
#pragma unroll
        for (int i = 0; i < R::depth; ++i) next_page[i] = page_of(i);
        __syncthreads();                             // the shared memory of the segment before has been read
#pragma unroll
        for (int i = 0; i < R::depth - 1; ++i) copy_tile(i, next_page[i]);
        int page_ahead = next_page[R::depth - 1];

        // The rows g and g + 8 of the queries as FP16 pieces: of the 64 values of a
        // group a lane holds 16 in a row, four for each K = 16 step.
        uint32_t qa[PIECES][NG * 4][4];
        float factor[2];                             // a row's: scores are sums times factor times s_k, base 2
        int pos[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = min(row0 + g + 8 * r, row0 + rows - 1), i = row / p.group;
            const T* from = static_cast<const T*>(p.q) + (s.start + i) * p.q_t + (head * p.group + row - i * p.group) * p.q_h;
            pos[r] = pos0 + i;
            float x[NG * 16];
            float top = 0.0f;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int d = n * 64 + t * 16;
                if (d < p.D) {
                    kv_load8(from + d, p.wide, x + n * 16);
                    kv_load8(from + d + 8, p.wide, x + n * 16 + 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[n * 16 + e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[n * 16 + e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(14 - E), top = m 2^E
            const int E = max((int)(__float_as_uint(top) >> 23) - 127, -112);
            const float up = __uint_as_float((uint32_t)(14 - E + 127) << 23);
            factor[r] = __uint_as_float((uint32_t)(E - 14 + 127) << 23) * (p.scale * kLog2e);
#pragma unroll
            for (int k = 0; k < NG * 4; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {        // a0/a1: the first pair; a2/a3: the second
                    const float lo = x[4 * k + 2 * h] * up, hi = x[4 * k + 2 * h + 1] * up;
                    qa[0][k][r + 2 * h] = half2_bits(lo, hi);
                    if constexpr (TWO) qa[PIECES - 1][k][r + 2 * h] = half2_rest(lo, hi, qa[0][k][r + 2 * h]);
                }
        }

        float o[NG * 8][4];
#pragma unroll
        for (int n = 0; n < NG * 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
        float top[2] = {-INFINITY, -INFINITY};       // running maxima of the scores
        float ref[2] = {-INFINITY, -INFINITY};       // and of what o is held against
        float total[2] = {0.0f, 0.0f};               // this lane's sums of p

        for (int i = 0; i < tiles; ++i) {
            asm volatile("cp.async.wait_group %0;" :: "n"(R::depth - 2) : "memory");
            __syncwarp();
            copy_tile(i + R::depth - 1, page_ahead);
            page_ahead = page_of(i + R::depth);
            const int tok = tile0 + i * kUnit;
            if (tok >= sees_end || tok + kTile <= sees_begin) continue;
            const uint8_t* kt = ring + i % R::depth * R::stage;
            const uint8_t* vt = kt + R::side;
            const float k_scale = *reinterpret_cast<const float*>(kt + 2 * R::side);
            const float v_scale = *reinterpret_cast<const float*>(kt + 2 * R::side + 4);

            float sc[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = 0.0f;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    const uint4 w4 = *reinterpret_cast<const uint4*>(kt + piece_at<NG>(8 * n + g, 4 * gr + t));
                    const uint32_t wd[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t b0 = kv_half2((uint16_t)wd[k]), b1 = kv_half2((uint16_t)(wd[k] >> 16));
                        if constexpr (TWO) mma_f16(sc[n], qa[PIECES - 1][4 * gr + k], b0, b1);
                        mma_f16(sc[n], qa[0][4 * gr + k], b0, b1);
                    }
                }
            }
            // base-2 scores; what a row does not see is -infinity
            const bool edge = tok + kTile > pos0 + row0 / p.group + 1 || tok + kTile > s.len ||
                              (p.window && tok <= pos0 + (row0 + rows - 1) / p.group - p.window);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float f = factor[r] * k_scale;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& x = sc[n][2 * r + e];
                        x *= f;
                        if (edge) {
                            const int j = tok + 8 * n + 2 * t + e;
                            if (j > pos[r] || j >= s.len || (p.window && j <= pos[r] - p.window)) x = -INFINITY;
                        }
                    }
            }
            // a bound of log2(s_v): its exponent and one
            const int v_exp = (int)((__float_as_uint(v_scale) >> 23) & 0xFF) - 126;
            uint32_t pa[PIECES][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float m = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const float top_now = fmaxf(top[r], m), ref_now = fmaxf(ref[r], m + (float)(v_exp - 14));
                if (top_now > top[r]) total[r] *= exp2_of(top[r] - top_now);
                if (__any_sync(0xffffffffu, ref_now > ref[r])) {
                    const float c = ref_now > ref[r] ? exp2_of(ref[r] - ref_now) : 1.0f;
#pragma unroll
                    for (int n = 0; n < NG * 8; ++n) {
                        o[n][2 * r] *= c;
                        o[n][2 * r + 1] *= c;
                    }
                }
                top[r] = top_now;
                ref[r] = ref_now;
                const float m0 = top_now == -INFINITY ? 0.0f : top_now;
                const float f = top_now == -INFINITY ? 0.0f : v_scale * exp2_of(top_now - ref_now);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = exp2_of(sc[n][2 * r] - m0), p1 = exp2_of(sc[n][2 * r + 1] - m0);
                    total[r] += p0 + p1;
                    pa[0][r + 2 * n] = half2_bits(p0 * f, p1 * f);
                    if constexpr (TWO) pa[PIECES - 1][r + 2 * n] = half2_rest(p0 * f, p1 * f, pa[0][r + 2 * n]);
                }
            }
            // Values: of the 64 of a group a lane holds 8 in a row, of the four tokens 2t, 2t + 1, 2t + 8, 2t + 9.
            bool nan_seen = false;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                uint2 row[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    row[k] = *reinterpret_cast<const uint2*>(
                        vt + piece_at<NG>(2 * t + (k & 1) + 8 * (k >> 1), 4 * gr + (g >> 1)) + (g & 1) * 8);
                    if (edge) {
                        // A NaN counts in the rows that see its token only: 0 times NaN is NaN, so it is
                        // taken out here and put into those rows below.
                        if (nan_bytes(row[k].x) | nan_bytes(row[k].y)) {
                            nan_seen = true;
                            row[k].x &= ~nan_bytes(row[k].x);
                            row[k].y &= ~nan_bytes(row[k].y);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t a0 = j < 4 ? row[0].x : row[0].y, a1 = j < 4 ? row[1].x : row[1].y;
                    const uint32_t a2 = j < 4 ? row[2].x : row[2].y, a3 = j < 4 ? row[3].x : row[3].y;
                    const uint32_t sel = (j & 3) < 2 ? 0x5140 : 0x7362;
                    const uint32_t lo = __byte_perm(a0, a1, sel), hi = __byte_perm(a2, a3, sel);
                    const uint32_t b0 = kv_half2((uint16_t)(j & 1 ? lo >> 16 : lo));
                    const uint32_t b1 = kv_half2((uint16_t)(j & 1 ? hi >> 16 : hi));
                    if constexpr (TWO) mma_f16(o[gr * 8 + j], pa[PIECES - 1], b0, b1);
                    mma_f16(o[gr * 8 + j], pa[0], b0, b1);
                }
            }
            if (edge && __any_sync(0xffffffffu, nan_seen)) {
                for (int row = 0; row < kTile; ++row) {
                    const int j = tok + row;
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // values 64 gr + 8 (2t + e) .. + 7
                            const uint8_t* at8 = vt + piece_at<NG>(row, 4 * gr + t) + e * 8;
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                if ((at8[x] & 0x7F) == 0x7F) {
#pragma unroll
                                    for (int r = 0; r < 2; ++r)
                                        if (j <= pos[r] && j < s.len && !(p.window && j <= pos[r] - p.window))
                                            o[gr * 8 + x][2 * r + e] = nan;
                                }
                        }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            total[r] += __shfl_xor_sync(0xffffffffu, total[r], 1);
            total[r] += __shfl_xor_sync(0xffffffffu, total[r], 2);
        }
        __syncthreads();                             // all rings have been read
        // the warps' sums: [warp][row][4 + D]: maximum, sum, reference, and o
        const int pitch = NG * 64 + 4;
        float* const joined = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float* to = joined + (warp * kRows + g + 8 * r) * pitch;
            if (t == 0) {
                to[0] = top[r];
                to[1] = total[r];
                to[2] = ref[r];
            }
            to += 4;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float4*>(to + 64 * gr + 16 * t + 8 * e + 4 * h) =
                            make_float4(o[gr * 8 + 4 * h][2 * r + e], o[gr * 8 + 4 * h + 1][2 * r + e],
                                        o[gr * 8 + 4 * h + 2][2 * r + e], o[gr * 8 + 4 * h + 3][2 * r + e]);
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == units;
        // Adds `parts` of one layout up; row r, value d of each at from + part * step
        auto finish = [&](int r, int d, float m, float l, float ref_all, float sum_o) {
            const int row = row0 + r, i = row / p.group;
            float y = l > 0.0f || l != l ? sum_o / l * exp2_of(ref_all - m) : 0.0f;
            if (bad) y = nan;
            static_cast<T*>(p.out)[(s.start + i) * p.out_t + (head * p.group + row - i * p.group) * p.out_h + d] = kv_from<T>(y);
        };
        auto add_up = [&](const float* from, int64_t step, int parts, float& m, float& l, float& ref_all, int d, float& sum_o) {
            m = ref_all = -INFINITY;
            for (int k = 0; k < parts; ++k) {
                m = fmaxf(m, from[k * step]);
                ref_all = fmaxf(ref_all, from[k * step + 2]);
            }
            l = sum_o = 0.0f;
            for (int k = 0; k < parts; ++k) {
                const float mk = from[k * step], rk = from[k * step + 2];
                if (mk > -INFINITY || from[k * step + 1] != 0.0f) l += from[k * step + 1] * exp2_of(mk - m);
                const float ok = from[k * step + 4 + d];
                if (rk > -INFINITY || ok != 0.0f) sum_o += ok * exp2_of(rk - ref_all);
            }
        };
        const int part_pitch = p.D + 4;
        float* const slot = p.partial + (2 * (int64_t)blockIdx.x + (u0 == 0)) * kRows * part_pitch;
        for (int e = tid; e < rows * p.D; e += kThreads) {
            const int r = e / p.D, d = e - r * p.D;
            float m, l, ref_all, sum_o;
            add_up(joined + r * pitch, kRows * pitch, kWarps, m, l, ref_all, d, sum_o);
            if (whole) {
                finish(r, d, m, l, ref_all, sum_o);
            } else {
                float* to = slot + r * part_pitch;
                to[4 + d] = sum_o;
                if (d == 0) {
                    to[0] = m;
                    to[1] = l;
                    to[2] = ref_all;
                }
            }
        }
        if (!whole) {
            // CTAs that share the segment: c0, whose part is its range's last, to c1
            const int64_t c0 = ((seg_begin + 1) * ctas - 1) / all, c1 = (seg_end * ctas - 1) / all;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                order = atomicAdd(p.arrived + c0, 1u);
                __threadfence();
            }
            __syncthreads();
            if (order == (unsigned)(c1 - c0)) {
                if (tid == 0) p.arrived[c0] = 0;
                for (int e = tid; e < rows * p.D; e += kThreads) {
                    const int r = e / p.D, d = e - r * p.D;
                    // c0's slot is its odd one, the others' their even one
                    float m = -INFINITY, ref_all = -INFINITY, l = 0.0f, sum_o = 0.0f;
                    auto part = [&](int64_t c) { return p.partial + ((2 * c + (c == c0)) * kRows + r) * part_pitch; };
                    for (int64_t c = c0; c <= c1; ++c) {
                        m = fmaxf(m, __ldcg(part(c)));
                        ref_all = fmaxf(ref_all, __ldcg(part(c) + 2));
                    }
                    for (int64_t c = c0; c <= c1; ++c) {
                        const float* from = part(c);
                        const float mk = __ldcg(from), lk = __ldcg(from + 1), rk = __ldcg(from + 2), ok = __ldcg(from + 4 + d);
                        if (mk > -INFINITY || lk != 0.0f) l += lk * exp2_of(mk - m);
                        if (rk > -INFINITY || ok != 0.0f) sum_o += ok * exp2_of(rk - ref_all);
                    }
                    finish(r, d, m, l, ref_all, sum_o);
                }
            }
        }
        at = min(stop, seg_end);
    }
}

template <typename T, int NG>
cudaError_t launch_decode(AttnParams p, DeviceState* d, cudaStream_t stream) {
    auto kern = kv_decode_kernel<T, NG>;
    static int per_sm[kMaxDevices] = {};             // (g_mu is held)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!per_sm[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<NG>::bytes);
        int n = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, Ring<NG>::bytes);
        if (e != cudaSuccess) return e;
        per_sm[dev] = n < 1 ? 1 : n > kKvCtasPerSm ? kKvCtasPerSm : n;
    }
    kern<<<(unsigned)(d->sms * per_sm[dev]), kThreads, Ring<NG>::bytes, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const AttnParams& p, DeviceState* d, cudaStream_t stream) {
    if (p.D <= 64) return launch_decode<T, 1>(p, d, stream);
    if (p.D <= 128) return launch_decode<T, 2>(p, d, stream);
    if (p.D <= 192) return launch_decode<T, 3>(p, d, stream);
    return launch_decode<T, 4>(p, d, stream);
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" emu_status_t emu_kv_attention(int dtype, int64_t T, const emu_heads_t* q, const emu_heads_t* out,
                                         const emu_kv_cache_t* cache, int64_t B, const int32_t* table, int64_t width,
                                         const int32_t* starts, const int32_t* lengths, float scale, int64_t window,
                                         int64_t max_new, emu_stream_t stream_) {
    constexpr int64_t most = int64_t(1) << 40;
    if (dtype < EMU_F32 || dtype > EMU_F16 || !q || !out || !cache || !kv_cache_ok(*cache)) return EMU_ERR_INVALID_VALUE;
    if (T < 0 || T > kKvMaxRows || B < 0 || B > 1 << 20 || width < 0 || width > INT32_MAX / cache->page || window < 0 ||
        max_new < 0 || !(scale - scale == 0.0f))
        return EMU_ERR_INVALID_VALUE;
    if (q->heads < 1 || q->heads > 65536 || q->heads % cache->heads != 0 || out->heads != q->heads)
        return EMU_ERR_INVALID_VALUE;
    for (const emu_heads_t* h : {q, out})
        if (h->token_stride < -most || h->token_stride > most || h->head_stride < -most || h->head_stride > most ||
            (T > 0 && !h->data))
            return EMU_ERR_INVALID_VALUE;
    if (T > 0 && B > 0 && (!starts || !lengths || (width > 0 && !table))) return EMU_ERR_INVALID_VALUE;
    if (T == 0) return EMU_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    emu_status_t st = current_device(&d);
    if (st != EMU_OK) return st;
    // Made once, for the largest head and grid, so that no later call moves what a captured one reads.
    if (!d->kv_ws) {
        const size_t ctas = (size_t)d->sms * kKvCtasPerSm;
        const size_t flags = (ctas * sizeof(unsigned) + 255) / 256 * 256;
        const size_t bytes = flags + 2 * ctas * kRows * (256 + 4) * sizeof(float);
        void* ws = nullptr;
        if (cudaMalloc(&ws, bytes) != cudaSuccess) {
            cudaGetLastError();
            return EMU_ERR_ALLOC;
        }
        cudaError_t e = cudaMemset(ws, 0, flags);
        if (e == cudaSuccess) e = cudaDeviceSynchronize();       // whatever stream the calls are on
        if (e != cudaSuccess) {
            cudaFree(ws);
            return from_cuda(e);
        }
        d->kv_ws = ws;
        d->kv_flags = flags;
    }
    AttnParams p = {};
    p.q = q->data; p.q_t = q->token_stride; p.q_h = q->head_stride;
    p.out = out->data; p.out_t = out->token_stride; p.out_h = out->head_stride;
    p.T = (int)T; p.heads = (int)cache->heads; p.group = (int)(q->heads / cache->heads); p.D = (int)cache->D;
    p.page_log = kv_log2(cache->page);
    p.B = (int)B; p.width = (int)width;
    p.window = (int)(window > INT32_MAX / 2 ? 0 : window);
    p.k = static_cast<const uint8_t*>(cache->k); p.v = static_cast<const uint8_t*>(cache->v);
    p.ks = cache->k_scale; p.vs = cache->v_scale; p.pages = cache->pages;
    p.table = table; p.starts = starts; p.lengths = lengths;
    p.scale = scale;
    const int size = dtype == EMU_F32 ? 4 : 2;
    p.wide = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.q_t * size % 16 == 0 && p.q_h * size % 16 == 0;
    p.arrived = static_cast<unsigned*>(d->kv_ws);
    p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(d->kv_ws) + d->kv_flags);
    p.err = d->err;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    cudaError_t e;
    if (dtype == EMU_F32) e = launch_typed<float>(p, d, stream);
    else if (dtype == EMU_BF16) e = launch_typed<__nv_bfloat16>(p, d, stream);
    else e = launch_typed<__half>(p, d, stream);
    return from_cuda(e);
}
