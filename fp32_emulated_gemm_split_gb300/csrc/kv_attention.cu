// kv_attention.cu -- causal attention over keys and values kept in 8 bits
// (emu_kv_attention, include/emu_layers.h).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  k_j = s_k K_j, v_j = s_v V_j
//   over the tokens j that the query's position sees, K and V e4m3 codes, s_k and
//   s_v a number for each page and head
//
// A code is an FP16 value (4 significant bits, exponents -6..8), so one FP16 piece
// of K and V is exact, and FP32 queries and weights p need two pieces each, hi +
// lo (good to 2^-23), where a product of two FP32 operands would need nine of three:
// S = q_hi K + q_lo K, O = p_hi V + p_lo V, FP32 sums.  BF16 and FP16 queries are
// exact in one piece (a row is scaled by a power of two so that its largest value
// lies in 2^14..2^15; what falls below 2^-24 there is 2^-39 of the largest), and
// their outputs take p in one piece, rounded to 11 bits where the output keeps 8 or
// 11.  The page's s_v goes into p before its rounding: p s_v is held against a
// reference of its own, the running maximum of log2(p s_v), so that p keeps its
// bits however far the pages' scales are apart.
//
// Next tokens and drafts: bound by reading the cache.  The work is cut into units
// of tokens of one sequence and key head for a segment of 8 NR rows (a key head's
// query heads, of one token after another); the CTAs take equal consecutive ranges
// of all units.  A range's first and last segment may be shared with neighbours:
// their sums go to a slot in memory, and a second kernel adds them up in order.  (In
// the first one, by the last CTA to arrive, the sums' code took registers from the
// steps: 96 sequences 220 us, 192 without it.)  Within a CTA each warp takes every kWarps-th step of ST tokens through a ring of its own,
// filled by tensor copies: no barrier but at a segment's end.  Measured: next tokens of 96
// sequences (600,000 tokens, 8 heads of 128, 1.22 GB) 196 us, 6.2 TB/s, 92 % of a
// copy's rate; the copies alone 181 us.  A ring of three stages and two CTAs an SM: 235;
// steps of 16 tokens through registers, rows as the MMA's 16 (M): 332.
//
// The rows are the MMA's N, so that 8 of them fill it: S^T = K Q^T, O^T = V^T P^T,
// codes as the A operand, straight from their bytes.  The order of the values in a
// product's sum, of the rows of O^T and of the tokens is free, and chosen so that
// a lane reads 16 bytes at a time and no two lanes of a phase the same banks:
// token t(g) = (g >> 1) + 4 (g & 1) is row g of S^T, piece (g >> 1) + 4 (g & 1) of 16
// values of V belongs to rows g and g + 8 of O^T.
#include "kv_attention.cuh"

#include <type_traits>

namespace emu {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKvCtasPerSm = 4;                      // at most
// Rows of a sequence (16-bit types, heads up to 128; FP32: 16) up to which this file's kernel runs, in segments of 16 that
// each read the cache, all but the first from L2.  24 sequences of 3 to 7 tokens, 8 heads of 128 a key head: 75 us, in
// kv_prompt.cu 106, and in segments of 32 (queries in shared memory, steps of 16 tokens for their registers) 102.  Both
// kernels where all sequences have so many rows (us, this one's and kv_prompt.cu's): 24 sequences of 300 to 7000 tokens, 4 key
// heads of 128: 16 rows 38 / 82, 32 rows 62 / 82, 48 rows 91 / 85, 64 rows 119 / 89; 8 of 64: 51 / 108, 93 / 110, 142 / 116,
// 180 / 120; two of 60,000, 8 of 128: 62 / 158, 103 / 161, 147 / 163, 186 / 165.  FP32: 46 / 95, 79 / 97, 113 / 98, 151 / 98.
// They meet at 40 to 48 rows in either type where all sequences have as many; drafts of different lengths have fewer.
constexpr int kFewKvRows = 64;

// Steps that a warp adds up in an MMA's sums, 16-bit rows: each MMA rounds toward zero, some 2^-24 of the sum lost as it grows.
// Behind so many the sum goes to one in memory, to the nearest.  (FP32 rows add each step's sums to the nearest.)
constexpr int kChain = 256;                          // (whole batches)
constexpr int kMovedQuads = 33;                      // of a lane: o of 16 rows of 256, and its rows' references

// Steps start on multiples of ST tokens; the first one that any row of the sequence sees.
template <int ST>
__device__ __forceinline__ int first_token(const AttnParams& p, const Seq& s) {
    if (!p.window) return 0;
    return max(0, s.len - s.n - p.window + 1) & ~(ST - 1);
}
template <int ST>
__device__ __forceinline__ int units_of(const AttnParams& p, const Seq& s) {       // of one segment
    constexpr int unit = ST * kWarps;
    return max(1, (s.len - first_token<ST>(p, s) + unit - 1) / unit);
}
template <int ST, int ROWS>
__device__ __forceinline__ int64_t all_units(const AttnParams& p, const Seq& s) {  // of the sequence
    const int64_t rows = (int64_t)s.n * p.group;
    return (rows + ROWS - 1) / ROWS * p.heads * units_of<ST>(p, s);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, two neighbours of a row per lane, turned.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Where byte o of a run of codes lies in shared memory: rows of 128 bytes, their
// 16-byte pieces swizzled by the row (the tensor copies' 128-byte swizzle).
__device__ __forceinline__ uint32_t swizzled(uint32_t o) { return o ^ (o >> 3 & 0x70); }

// D in 64s (NG) as the lanes hold the values of O^T: blocks of 128 (16 bytes per
// lane group and token), and one of 64 (8 bytes) where NG is odd.
template <int NG>
struct Blocks {
    static constexpr int whole = NG / 2, count = (NG + 1) / 2;
    static constexpr int tiles(int b) { return b < whole ? 8 : 4; }      // MMA tiles of 16 values
    // first of the values that lane group g has in block b
    static __device__ __forceinline__ int first(int b, int g) {
        return b < whole ? 128 * b + 16 * ((g >> 1) + 4 * (g & 1)) : 128 * b + 8 * g;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// What a warp of kv_decode_kernel holds of a segment, and a step of ST tokens of it.
//
// DT: the values of a head where they are known when this is compiled (a lane's places in a
// tile are then the same in every tile, 16 DT bytes apart), or 0.
template <typename T, int NG, int DT, int NR, int ST>
struct Segment {
    static constexpr bool TWO = sizeof(T) == 4;      // two pieces of q and of p
    static constexpr int PIECES = TWO ? 2 : 1;
    static constexpr int SUB = ST / 16;              // tiles of 16 tokens in a step
    using Bl = Blocks<NG>;
    static_assert(DT % 64 == 0, "whole rows of 1024 bytes from tile to tile");

    uint32_t qb[PIECES][NR][NG * 4][2];              // the rows of the queries as FP16 pieces, 2^14 the largest value
    float factor[NR][2];                             // of rows 8 r + 2t, + 1: scores are sums times factor times s_k, base 2
    int pos[NR][2];                                  // and their positions
    float o[Bl::count * 8][NR][4];                   // (of a block of 64: the first four tiles)
    float top[NR][2], ref[NR][2], total[NR][2];      // running maxima of the scores, what o is held against, sums of p
    uint32_t k_at[NG][2], v_at[Bl::count][4];        // where a lane's codes lie in a stage
    int d_rt, len, window, side;

    // Adds o to this lane's sums in memory (`first`: begins them) and starts anew, or, at the end, the sums to o.
    __device__ __forceinline__ void move_sums(float4* sums, bool first, bool end) {
        float4* const held = sums + (kMovedQuads - 1) * 32;      // references
        float x[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) x[r][e] = 0.0f;
        if (!first) {
            const float4 h = *held;
            x[0][0] = share_of(h.x, ref[0][0]);
            x[0][1] = share_of(h.y, ref[0][1]);
            x[NR - 1][0] = NR > 1 ? share_of(h.z, ref[NR - 1][0]) : x[0][0];
            x[NR - 1][1] = NR > 1 ? share_of(h.w, ref[NR - 1][1]) : x[0][1];
        }
#pragma unroll
        for (int n = 0; n < Bl::count * 8; ++n)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float4* const at = sums + (n * NR + r) * 32;
                const float4 old = first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *at;
                float (&y)[4] = o[n][r];
                y[0] = fmaf(old.x, x[r][0], y[0]);
                y[1] = fmaf(old.y, x[r][1], y[1]);
                y[2] = fmaf(old.z, x[r][0], y[2]);
                y[3] = fmaf(old.w, x[r][1], y[3]);
                if (!end) {
                    *at = make_float4(y[0], y[1], y[2], y[3]);
                    y[0] = y[1] = y[2] = y[3] = 0.0f;
                }
            }
        if (!end) *held = make_float4(ref[0][0], ref[0][1], ref[NR - 1][0], ref[NR - 1][1]);
    }

    // EDGE: some row does not see some token of the step.
    template <bool EDGE>
    __device__ __forceinline__ void step(int tok, uint32_t kt, const float (&k_scale)[SUB], const float (&v_scale)[SUB]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, D = DT ? DT : d_rt;
        const int tau = (g >> 1) + 4 * (g & 1);      // this lane's token of S^T's rows 0..7
        const float nan = __uint_as_float(0x7FC00000u);
        float sc[SUB][NR][4];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            float other[NR][4];                  // a second chain of sums (TWO: of the low pieces)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[u][r][e] = other[r][e] = 0.0f;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                if (DT) {
                    lo = lds128(kt + k_at[gr][0] + u * 16 * DT);
                    hi = lds128(kt + k_at[gr][1] + u * 16 * DT);
                } else if (64 * gr + 16 * t < D) {
                    lo = lds128(kt + swizzled((16 * u + tau) * D + 64 * gr + 16 * t));
                    hi = lds128(kt + swizzled((16 * u + tau + 8) * D + 64 * gr + 16 * t));
                }
                const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a[4] = {kv_half2((uint16_t)wl[k]), kv_half2((uint16_t)wh[k]),
                                           kv_half2((uint16_t)(wl[k] >> 16)), kv_half2((uint16_t)(wh[k] >> 16))};
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        if constexpr (TWO) {
                            mma_f16(other[r], a, qb[PIECES - 1][r][4 * gr + k][0], qb[PIECES - 1][r][4 * gr + k][1]);
                            mma_f16(sc[u][r], a, qb[0][r][4 * gr + k][0], qb[0][r][4 * gr + k][1]);
                        } else {
                            mma_f16(k & 1 ? other[r] : sc[u][r], a, qb[0][r][4 * gr + k][0], qb[0][r][4 * gr + k][1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[u][r][e] += other[r][e];
        }
        // bounds of log2(s_v), its exponent and one, less 14: p s_v has 14 bits above 1 in FP16
        int v_exp[SUB];
#pragma unroll
        for (int u = 0; u < SUB; ++u) v_exp[u] = scale_bound(v_scale[u]);
        uint32_t pb[PIECES][SUB][NR][2];         // P^T: rows of tokens, turned
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float m0[2], f[SUB][2], fs[SUB][2], back[2] = {1.0f, 1.0f};
            uint32_t hidden = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m[SUB];
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    fs[u][e] = factor[r][e] * k_scale[u];
                    float a = sc[u][r][e] * fs[u][e], c = sc[u][r][e + 2] * fs[u][e];
                    if constexpr (EDGE) {
                        // what a row does not see is -infinity, and has no weight below
                        const int j = tok + 16 * u + tau, last = min(pos[r][e], len - 1);
                        const int from = window ? pos[r][e] - window : -1;
                        if (j > last || j <= from) a = -INFINITY, hidden |= 1u << (4 * u + e);
                        if (j + 8 > last || j + 8 <= from) c = -INFINITY, hidden |= 1u << (4 * u + 2 + e);
                    }
                    m[u] = fmaxf(a, c);
                }
                float m_all = m[0], over = m[0] + (float)v_exp[0];
                bool apart = false;
                if constexpr (SUB == 2) {
                    m_all = fmaxf(m[0], m[1]);
                    over = fmaxf(over, m[1] + (float)v_exp[1]);
                    apart = v_exp[0] != v_exp[1];
                }
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) m_all = fmaxf(m_all, __shfl_xor_sync(0xffffffffu, m_all, x));
                if (apart) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) over = fmaxf(over, __shfl_xor_sync(0xffffffffu, over, x));
                } else {
                    over = m_all + (float)v_exp[0];
                }
                const float top_now = fmaxf(top[r][e], m_all), ref_now = fmaxf(ref[r][e], over);
                if (top_now > top[r][e]) total[r][e] *= exp2_of(top[r][e] - top_now);
                const bool up = ref_now > ref[r][e];
                if (__any_sync(0xffffffffu, up)) {
                    const float c = up ? exp2_of(ref[r][e] - ref_now) : 1.0f;
#pragma unroll
                    for (int n = 0; n < Bl::count * 8; ++n) {
                        o[n][r][e] *= c;
                        o[n][r][e + 2] *= c;
                    }
                }
                top[r][e] = top_now;
                ref[r][e] = ref_now;
                m0[e] = top_now == -INFINITY ? 0.0f : top_now;
#pragma unroll
                for (int u = 0; u < SUB; ++u)
                    f[u][e] = top_now == -INFINITY ? 0.0f : v_scale[u] * exp2_of(top_now - ref_now);
            }
            if (v_scale[0] > kFarValue || v_scale[SUB - 1] > kFarValue) {        // (the same for all lanes)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (fmaxf(f[0][e], f[SUB - 1][e]) > kFarScale && top[r][e] > ref[r][e]) {
                        m0[e] = ref[r][e];
                        back[e] = exp2_of(ref[r][e] - top[r][e]);
#pragma unroll
                        for (int u = 0; u < SUB; ++u) f[u][e] = v_scale[u];
                    }
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float w2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // (one rounding, at the difference's size)
                        float x = exp2_of(fmaf(sc[u][r][e + 2 * h], fs[u][e], -m0[e]));
                        w2[e] = x * f[u][e];
                        if (EDGE && (hidden >> (4 * u + 2 * h + e) & 1)) x = w2[e] = 0.0f;
                        total[r][e] = fmaf(x, back[e], total[r][e]);
                    }
                    const uint32_t hi = half2_bits(w2[0], w2[1]);
                    pb[0][u][r][h] = turned(hi);
                    if constexpr (TWO) pb[PIECES - 1][u][r][h] = turned(half2_rest(w2[0], w2[1], hi));
                }
        }
        // Values: of a token a lane has 16 (8) in a row of each block, of the four tokens t, t + 4, t + 8, t + 12
        // of a tile; bytes 2j and 2j + 1 are rows g and g + 8 of the block's tile j.
        bool nan_seen = false;
        auto clean = [&](uint32_t& w) {
            // A NaN counts in the rows that see its token only: 0 times NaN is NaN, so it is taken out here
            // and put into those rows below.
            const uint32_t n = nan_bytes(w);
            nan_seen = nan_seen || n != 0;
            w &= ~n;
        };
#pragma unroll
        for (int bl = 0; bl < Bl::count; ++bl) {
            constexpr int WIDE = TWO ? 2 : 4;    // words of a token at a time (TWO: the step's own sums need the registers)
            const int d0 = Bl::first(bl, g);
#pragma unroll
            for (int w0 = 0; w0 < Bl::tiles(bl) / 2; w0 += WIDE) {
                const int words = min(WIDE, Bl::tiles(bl) / 2 - w0);
                float fresh[TWO ? 2 * WIDE : 1][NR][4];      // added to o in FP32, nearest
#pragma unroll
                for (int j = 0; j < (TWO ? 2 * WIDE : 1); ++j)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) fresh[j][r][e] = 0.0f;
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t row[4][WIDE];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // (4 w0 is 0 or 8: the half of a piece, which is not swizzled)
                        const uint32_t from = kt + 4 * w0 + (DT ? v_at[bl][k] + u * 16 * DT
                                                                 : swizzled((16 * u + t + 4 * k) * D + d0) + side);
                        if (words == 4) {
                            const uint4 x = lds128(from);
                            row[k][0] = x.x;
                            row[k][1] = x.y;
                            row[k][WIDE - 2] = x.z;
                            row[k][WIDE - 1] = x.w;
                        } else {
                            const uint2 x = lds64(from);
                            row[k][0] = x.x;
                            row[k][1] = x.y;
                        }
                        if (EDGE)
#pragma unroll
                            for (int x = 0; x < WIDE; ++x)
                                if (x < words) clean(row[k][x]);
                    }
#pragma unroll
                    for (int j = 0; j < 2 * WIDE; ++j) {
                        if (j >= 2 * words) continue;
                        const uint32_t sel = j & 1 ? 0x7362 : 0x5140;
                        const uint32_t x = __byte_perm(row[0][j / 2], row[1][j / 2], sel);
                        const uint32_t y = __byte_perm(row[2][j / 2], row[3][j / 2], sel);
                        const uint32_t a[4] = {kv_half2((uint16_t)x), kv_half2((uint16_t)(x >> 16)), kv_half2((uint16_t)y),
                                               kv_half2((uint16_t)(y >> 16))};
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            if constexpr (TWO) {
                                mma_f16(fresh[j][r], a, pb[PIECES - 1][u][r][0], pb[PIECES - 1][u][r][1]);
                                mma_f16(fresh[j][r], a, pb[0][u][r][0], pb[0][u][r][1]);
                            } else {
                                mma_f16(o[bl * 8 + 2 * w0 + j][r], a, pb[0][u][r][0], pb[0][u][r][1]);
                            }
                        }
                    }
                }
                if constexpr (TWO)
#pragma unroll
                    for (int j = 0; j < 2 * WIDE; ++j)
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (j < 2 * words) o[bl * 8 + 2 * w0 + j][r][e] += fresh[j][r][e];
            }
        }
        if (EDGE && __any_sync(0xffffffffu, nan_seen)) {
            for (int x = 0; x < ST; ++x) {
                const int j = tok + x;
#pragma unroll
                for (int bl = 0; bl < Bl::count; ++bl)
#pragma unroll
                    for (int c = 0; c < 2 * Bl::tiles(bl); ++c) {
                        const uint32_t at4 = kt + side + swizzled(x * D + Bl::first(bl, g) + (c & ~3));
                        uint32_t four;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(four) : "r"(at4) : "memory");
                        if ((four >> 8 * (c & 3) & 0x7F) == 0x7F) {
#pragma unroll
                            for (int r = 0; r < NR; ++r)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (j <= pos[r][e] && j < len && !(window && j <= pos[r][e] - window))
                                        o[bl * 8 + c / 2][r][e + 2 * (c & 1)] = nan;
                        }
                    }
            }
        }
    }
};

// Looks up the segment of unit w.at.
template <int ST, int ROWS>
__device__ __forceinline__ void find_segment(const AttnParams& p, Work& w) {
    Seq s = seq_of(p, w.seq);
    int64_t n = all_units<ST, ROWS>(p, s);
    while (w.at >= w.base + n) {
        w.base += n;
        s = seq_of(p, ++w.seq);
        n = all_units<ST, ROWS>(p, s);
    }
    w.bad = s.len < 0;
    if (w.bad) s.len = 0;
    w.start = s.start;
    w.len = s.len;
    w.pos0 = s.len - s.n;
    const int units = units_of<ST>(p, s);
    const int seg = (int)((w.at - w.base) / units);  // row tile * heads + head
    w.begin = w.base + (int64_t)seg * units;
    w.end = w.begin + units;
    const int u0 = (int)(w.at - w.begin);
    w.units = (int)(min(w.stop, w.end) - w.at);
    w.starts = u0 == 0;
    w.whole = w.units == units;
    w.head = seg % p.heads;
    w.row0 = seg / p.heads * ROWS;
    w.rows = min(ROWS, s.n * p.group - w.row0);
    w.token0 = first_token<ST>(p, s) + u0 * (ST * kWarps);
}

template <typename T, int NG, int DT, int NR, int ST>
__global__ void __launch_bounds__(kThreads, NG > 2 ? 1 : NR == 1 && (NG == 1 || sizeof(T) == 2) ? 3 : 2)
kv_decode_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    constexpr bool TWO = sizeof(T) == 4;             // two pieces of q and of p
    constexpr int PIECES = TWO ? 2 : 1;
    constexpr int ROWS = 8 * NR, SUB = ST / 16;      // rows of a segment; tiles of 16 tokens in a step
    constexpr int UNIT = ST * kWarps;
    constexpr int BATCH = 32 / SUB;                  // steps whose pages the lanes hold, one tile each
    static_assert(kChain % BATCH == 0, "sums are moved where a batch begins");
    using Bl = Blocks<NG>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps][4];
    __shared__ int64_t warp_sum[kWarps];
    __shared__ Work work;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int P = 1 << p.page_log, D = DT ? DT : p.D;
    static_assert(DT % 64 == 0, "whole rows of 1024 bytes from tile to tile");
    const uint32_t ring = smem_u32(smem) + warp * p.depth * 2 * p.side;
    const uint32_t bar0 = smem_u32(bars[warp]);
    if (lane == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(bar0 + 8 * i, SUB);
        fence_mbar_init();
    }
    const float nan = __uint_as_float(0x7FC00000u);
    griddep_launch_dependents();                     // (kv_join_kernel waits for this one's end)

    // all units, and where this CTA's range of them begins: a run of sequences per thread
    const int per = (p.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, p.B); ++b) {
        const Seq s = seq_of(p, b);
        mine += all_units<ST, ROWS>(p, s);
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
    // (no more CTAs than units: each has one at least)
    const int64_t ctas = min((int64_t)gridDim.x, all);
    if (blockIdx.x >= ctas) {
        if (tid == 0) p.shared[blockIdx.x].units = 0;
        return;
    }
    {
        const int64_t at = all * blockIdx.x / ctas;
        int64_t before = sum - mine;
        if (before <= at && at < sum) {              // (one thread)
            int b = tid * per;
            for (;; ++b) {
                const int64_t n = all_units<ST, ROWS>(p, seq_of(p, b));
                if (at < before + n) break;
                before += n;
            }
            work.all = all;
            work.ctas = ctas;
            work.at = at;
            work.stop = all * (blockIdx.x + 1) / ctas;
            work.base = before;
            work.seq = b;
            find_segment<ST, ROWS>(p, work);
        }
    }
    int stage_in = 0, stage_out = 0;                 // next stage to fill, to read
    uint32_t parity = 0;                             // of the stage to read, flips when the ring wraps
    bool dead = false;                               // a wait gave up: no more copies

    for (;;) {
        __syncthreads();                             // the segment is known, the shared memory of the one before read
        const int len = work.len, pos0 = work.pos0, head = work.head, row0 = work.row0, rows = work.rows, start = work.start;
        // tokens that some row of the segment sees; steps of this warp that have any
        const int pos_first = pos0 + row0 / p.group, pos_last = pos0 + (row0 + rows - 1) / p.group;
        const int sees_end = max(0, min(len, pos_last + 1));
        const int sees_begin = p.window ? max(0, pos_first - p.window + 1) : 0;
        int token0 = work.token0 + warp * ST;
        int steps = work.units;
        if (token0 + ST <= sees_begin) {
            const int skip = (sees_begin - token0 - ST) / UNIT + 1;
            token0 += skip * UNIT;
            steps -= skip;
        }
        steps = sees_end <= token0 ? 0 : min(steps, (sees_end - token0 + UNIT - 1) / UNIT);
        const int32_t* pages = p.table + (int64_t)work.seq * p.width;

        // A lane has one tile of each of BATCH steps: the page (-1: bad, -2: no row sees the tile) and its scales.
        auto page_of = [&](int i) {
            const int tok = token0 + i * UNIT + (SUB == 2 ? (lane & 1) * 16 : 0);
            // (where one copy brings the whole step, the step counts)
            const int from = p.copy_tokens > 16 ? token0 + i * UNIT : tok, to = from + p.copy_tokens;
            if (i >= steps || from >= sees_end || to <= sees_begin) return -2;
            const int page = pages[from >> p.page_log];
            return page >= 0 && page < p.pages ? page : -1;
        };
        auto scales_of = [&](int page, float& ks, float& vs) {
            const int64_t unit = (int64_t)max(page, 0) * p.heads + head;
            ks = page >= 0 ? p.ks[unit] : page == -1 ? nan : 0.0f;
            vs = page >= 0 ? p.vs[unit] : page == -1 ? nan : 0.0f;
            if (page == -1) record_error(p.err, kDevErrValue);
        };
        const int my_step = lane / SUB, my_sub = lane % SUB;     // of a batch, of a step
        // where one copy brings both tiles, one lane has the keys', the other the values'
        const bool joint = p.copy_tokens > 16;
        int page_now = page_of(my_step), page_next = page_of(BATCH + my_step);
        // The step's copies, by the lanes that have its tiles; each arrives once.
        auto copy_step = [&](int i, int page) {
            if (i >= steps) return;
            if (my_step == i % BATCH && !dead) {
                const uint32_t bar = bar0 + 8 * stage_in, dst = ring + stage_in * 2 * p.side + (joint ? 0 : my_sub * 16 * D);
                const int tok = token0 + i * UNIT + (joint ? 0 : my_sub * 16);
                const int row = (int)(((((int64_t)page * p.heads + head) << p.page_log) + (tok & (P - 1))) * D >> 7);
                const uint32_t bytes = p.copy_tokens * D;
                mbar_arrive_expect_tx(bar, page < 0 ? 0 : joint ? bytes : 2 * bytes);
                if (page >= 0) {
                    if (!joint || my_sub == 0) tma_load_3d(dst, &map_k, bar, 0, row, 0);
                    if (!joint || my_sub == 1) tma_load_3d(dst + p.side, &map_v, bar, 0, row, 0);
                }
            }
            stage_in = stage_in + 1 == p.depth ? 0 : stage_in + 1;
        };
        for (int i = 0; i < p.depth - 1; ++i) copy_step(i, page_now);
        float ks_now, vs_now, ks_next = 0.0f, vs_next = 0.0f;
        scales_of(page_now, ks_now, vs_now);

        // The rows of the queries as FP16 pieces: of the 64 values of a group a lane
        // holds 16 in a row, four for each K = 16 step.
        Segment<T, NG, DT, NR, ST> sg;
        sg.d_rt = D;
        sg.len = len;
        sg.window = p.window;
        sg.side = p.side;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = min(row0 + 8 * r + g, row0 + rows - 1), i = row / p.group;
            const T* from = static_cast<const T*>(p.q) + (start + i) * p.q_t + (head * p.group + row - i * p.group) * p.q_h;
            float x[NG * 16];
            float top = 0.0f;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int d = n * 64 + t * 16;
                if (d < D) {
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
            const float mine_factor = score_factor(top, E, p.scale);
#pragma unroll
            for (int k = 0; k < NG * 4; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float lo = x[4 * k + 2 * h] * up, hi = x[4 * k + 2 * h + 1] * up;
                    sg.qb[0][r][k][h] = half2_bits(lo, hi);
                    if constexpr (TWO) sg.qb[PIECES - 1][r][k][h] = half2_rest(lo, hi, sg.qb[0][r][k][h]);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sg.factor[r][e] = __shfl_sync(0xffffffffu, mine_factor, 4 * (2 * t + e));
                sg.pos[r][e] = pos0 + min(row0 + 8 * r + 2 * t + e, row0 + rows - 1) / p.group;
            }
        }

#pragma unroll
        for (int n = 0; n < Bl::count * 8; ++n)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) sg.o[n][r][e] = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sg.top[r][e] = sg.ref[r][e] = -INFINITY;
                sg.total[r][e] = 0.0f;
            }
        const int tau = (g >> 1) + 4 * (g & 1);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int h = 0; h < 2; ++h) sg.k_at[gr][h] = swizzled((tau + 8 * h) * D + 64 * gr + 16 * t);
#pragma unroll
        for (int bl = 0; bl < Bl::count; ++bl)
#pragma unroll
            for (int k = 0; k < 4; ++k) sg.v_at[bl][k] = swizzled((t + 4 * k) * D + Bl::first(bl, g)) + p.side;

        float4* const sums = p.moved + (size_t)(blockIdx.x * kWarps + warp) * (kMovedQuads * 32) + lane;
        for (int i = 0; i < steps; ++i) {
            const int in_batch = i % BATCH;
            if (in_batch == 0 && i > 0) {
                if (!TWO && i % kChain == 0) sg.move_sums(sums, i == kChain, false);
                page_now = page_next;
                ks_now = ks_next;
                vs_now = vs_next;
                page_next = page_of(i + BATCH + my_step);
            }
            if (in_batch == BATCH / 2) scales_of(page_next, ks_next, vs_next);
            if (!dead && __any_sync(0xffffffffu, !mbar_wait(bar0 + 8 * stage_out, parity, p.err, kDevErrTimeout))) {
                // the copies in flight may still land: once more for each
                dead = true;
                for (int k = 0; k < min(p.depth - 1, steps - i); ++k) {
                    const int st = (stage_out + k) % p.depth;
                    mbar_wait(bar0 + 8 * st, parity ^ (stage_out + k >= p.depth), p.err, kDevErrTimeout);
                }
            }
            __syncwarp();                            // all lanes have read the stage that is filled now
            const int ahead = i + p.depth - 1;
            copy_step(ahead, ahead / BATCH == i / BATCH ? page_now : page_next);
            float k_scale[SUB], v_scale[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                k_scale[u] = __shfl_sync(0xffffffffu, ks_now, in_batch * SUB + u);
                v_scale[u] = __shfl_sync(0xffffffffu, vs_now, in_batch * SUB + u);
            }
            const int tok = token0 + i * UNIT;
            const uint32_t kt = ring + stage_out * 2 * p.side;
            if (++stage_out == p.depth) {
                stage_out = 0;
                parity ^= 1;
            }
            // (an edge: some row does not see some token of the step)
            if (tok + ST > pos_first + 1 || tok + ST > len || (p.window && tok <= pos_last - p.window))
                sg.template step<true>(tok, kt, k_scale, v_scale);
            else
                sg.template step<false>(tok, kt, k_scale, v_scale);
        }
        if (!TWO && steps > kChain) sg.move_sums(sums, false, true);
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sg.total[r][e] += __shfl_xor_sync(0xffffffffu, sg.total[r][e], x);
        __syncthreads();                             // all rings have been read, and none has copies in flight
        // the warps' sums: [warp][row][4 + D]: maximum, sum, reference, and o
        const int pitch = NG * 64 + 4;
        float* const joined = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* to = joined + (warp * ROWS + 8 * r + 2 * t + e) * pitch;
                if (g == 0) {
                    to[0] = sg.top[r][e];
                    to[1] = sg.total[r][e];
                    to[2] = sg.ref[r][e];
                }
#pragma unroll
                for (int bl = 0; bl < Bl::count; ++bl)
#pragma unroll
                    for (int j = 0; j < Bl::tiles(bl); j += 2)
                        *reinterpret_cast<float4*>(to + 4 + Bl::first(bl, g) + 2 * j) =
                            make_float4(sg.o[bl * 8 + j][r][e], sg.o[bl * 8 + j][r][e + 2], sg.o[bl * 8 + j + 1][r][e],
                                        sg.o[bl * 8 + j + 1][r][e + 2]);
            }
        __syncthreads();
        // the warps' sums added up: the rows, or this CTA's part of a segment that it shares
        const int quads = D / 4, part_pitch = D + 4;
        float* const slot = p.partial + (2 * (int64_t)blockIdx.x + work.starts) * (p.slot_rows * part_pitch);
        for (int i = tid; i < rows * quads; i += kThreads) {
            const int r = i / quads, d = (i - r * quads) * 4;
            const float* from = joined + r * pitch;
            float m = -INFINITY, ref_all = -INFINITY, l = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                m = fmaxf(m, from[k * ROWS * pitch]);
                ref_all = fmaxf(ref_all, from[k * ROWS * pitch + 2]);
            }
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float* f = from + k * ROWS * pitch;
                l += f[1] * weight_of(f[0], f[1], m);
                add_to(v, share_of(f[2], ref_all), *reinterpret_cast<const float4*>(f + 4 + d));
            }
            if (work.whole) {
                write_row<T>(p, work, r, d, m, l, ref_all, v);
            } else {
                float* to = slot + r * part_pitch;
                *reinterpret_cast<float4*>(to + 4 + d) = v;
                if (d == 0) *reinterpret_cast<float4*>(to) = make_float4(m, l, ref_all, 0.0f);
            }
        }
        // the next segment's copies come after what was read and written here
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if (work.end >= work.stop) break;
        __syncthreads();
        if (tid == 0) {
            work.at = work.end;
            find_segment<ST, ROWS>(p, work);
        }
    }
    // a segment that begins here and is shared is added up by kv_join_kernel
    if (tid == 0) {
        if (work.whole || !work.starts) work.units = 0;
        p.shared[blockIdx.x] = work;
    }
}

// What parts of a segment's row add up to: a lane has four values of o, of more than 128 eight.
struct RowSum {
    float m, l, ref;
    float4 v[2];
    __device__ __forceinline__ void clear() {
        m = ref = -INFINITY;
        l = 0.0f;
        v[0] = v[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    // Holds the sums against a maximum and a reference at least as large.
    __device__ __forceinline__ void lift(float m_new, float ref_new) {
        l *= weight_of(m, l, m_new);
        const float x = share_of(ref, ref_new);
        m = m_new;
        ref = ref_new;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 o = v[h];
            v[h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            add_to(v[h], x, o);
        }
    }
};

// Adds the parts of the segments that CTAs share up in order, and the rows before the first and
// behind the last sequence become zero.  Block (x, y): the segment that CTA x began; where it has few parts
// (most do: two or three), its rows kJoinWarps y on, a warp each; where it has many, its rows
// y, y + gridDim.y and so on, the parts dealt to the warps.
constexpr int kJoinWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_join_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float4 sums[kJoinWarps][64];
    __shared__ float stat[kJoinWarps][3];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = p.D, c0 = blockIdx.x;
    griddep_wait();
    {
        const int first = p.B > 0 ? min(max(p.starts[0], 0), p.T) : 0;
        const int used = p.B > 0 ? min(max(p.starts[p.B], first), p.T) - first : 0, values = p.heads * p.group * D;
        for (int i = blockIdx.x + blockIdx.y * gridDim.x; i < p.T - used; i += gridDim.x * gridDim.y) {
            const int row = i < first ? i : i + used;
            for (int e = tid; e < values; e += kJoinWarps * 32) {
                const int h = e / D;
                static_cast<T*>(p.out)[row * p.out_t + h * p.out_h + (e - h * D)] = kv_from<T>(0.0f);
            }
        }
    }
    const Work& w = p.shared[c0];
    if (w.units == 0) return;
    // from c0's part, its odd slot, to that of the segment's last unit; theirs are the even ones
    const int parts = (int)((w.end * w.ctas - 1) / w.all) - c0 + 1;
    const int pitch = D + 4, d0 = lane * 4;
    auto add_row = [&](RowSum& s, int r, int first, int step) {
        s.clear();
        auto at = [&](int k) { return p.partial + ((2 * ((int64_t)c0 + k) + (k == 0)) * p.slot_rows + r) * pitch; };
        for (int k0 = first; k0 < parts; k0 += 4 * step) {
            float4 head[4], x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + i * step;
                const float* from = at(min(k, parts - 1));
                head[i] = *reinterpret_cast<const float4*>(from);
                x[i] = *reinterpret_cast<const float4*>(from + 4 + min(d0, D - 4));
                if (D > 128) y[i] = *reinterpret_cast<const float4*>(from + 4 + min(128 + d0, D - 4));
            }
            float m = s.m, ref = s.ref;
#pragma unroll
            for (int i = 0; i < 4; ++i) {            // (the last part twice changes no maximum)
                m = fmaxf(m, head[i].x);
                ref = fmaxf(ref, head[i].z);
            }
            s.lift(m, ref);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k0 + i * step < parts) {
                    s.l += head[i].y * weight_of(head[i].x, head[i].y, m);
                    const float share = share_of(head[i].z, ref);
                    add_to(s.v[0], share, x[i]);
                    if (D > 128) add_to(s.v[1], share, y[i]);
                }
        }
    };
    RowSum s;
    if (parts <= 16) {
        for (int r = blockIdx.y * kJoinWarps + warp; r < w.rows; r += gridDim.y * kJoinWarps) {
            add_row(s, r, 0, 1);
            if (d0 < D) write_row<T>(p, w, r, d0, s.m, s.l, s.ref, s.v[0]);
            if (128 + d0 < D) write_row<T>(p, w, r, 128 + d0, s.m, s.l, s.ref, s.v[1]);
        }
        return;
    }
    for (int r = blockIdx.y; r < w.rows; r += gridDim.y) {
        add_row(s, r, warp, kJoinWarps);
        if (lane == 0) {
            stat[warp][0] = s.m;
            stat[warp][1] = s.l;
            stat[warp][2] = s.ref;
        }
        sums[warp][lane] = s.v[0];
        sums[warp][lane + 32] = s.v[1];
        __syncthreads();
        if (tid * 4 < D) {
            float m = -INFINITY, ref = -INFINITY, l = 0.0f;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k) {
                m = fmaxf(m, stat[k][0]);
                ref = fmaxf(ref, stat[k][2]);
            }
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k) {
                l += stat[k][1] * weight_of(stat[k][0], stat[k][1], m);
                add_to(o, share_of(stat[k][2], ref), sums[k][tid]);
            }
            write_row<T>(p, w, r, tid * 4, m, l, ref, o);
        }
        __syncthreads();
    }
}

template <typename T, int NG, int DT, int NR>
cudaError_t launch_decode(AttnParams p, const emu_kv_cache_t& c, int64_t max_rows, DeviceState* d, cudaStream_t stream) {
    constexpr int ST = NG <= 2 ? 32 : 16, ROWS = 8 * NR;
    auto kern = kv_decode_kernel<T, NG, DT, NR, ST>;
    // the ring: up to 64 KB a CTA, two stages at least and four at most; a lane reads the values of a token in NG
    // whole 64s, of the last one past its end
    p.side = ((ST - 1) * p.D + NG * 64 + 1023) / 1024 * 1024;
    p.depth = (64 << 10) / (kWarps * 2 * p.side);
    p.depth = p.depth < 2 ? 2 : p.depth > 4 ? 4 : p.depth;
    p.copy_tokens = ST < c.page ? ST : (int)c.page;
    const int ring = kWarps * p.depth * 2 * p.side, joined = kWarps * ROWS * (NG * 64 + 4) * 4;
    const int smem = ring > joined ? ring : joined;
    CUtensorMap map_k = {}, map_v = {};
    if (c.pages > 0) {                               // (no page, no copy)
        const int64_t rows = c.pages * c.heads * c.page * c.D / 128;
        const int box = p.copy_tokens * p.D / 128;
        if (make_plane_map(&map_k, c.k, false, rows, 64, 64, 1, 64, box) != EMU_OK ||
            make_plane_map(&map_v, c.v, false, rows, 64, 64, 1, 64, box) != EMU_OK)
            return cudaErrorInvalidValue;
    }
    // CTAs resident at once, by ring size (g_mu is held)
    static int per_sm[kMaxDevices][17] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    int& fit = per_sm[dev][p.D / 16];
    if (!fit) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
        int n = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, smem);
        if (e != cudaSuccess) return e;
        fit = n < 1 ? 1 : n > kKvCtasPerSm ? kKvCtasPerSm : n;
    }
    p.slot_rows = ROWS;
    const unsigned ctas = (unsigned)(d->sms * fit);
    kern<<<ctas, kThreads, smem, stream>>>(p, map_k, map_v);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int dtype = sizeof(T) == 4 ? EMU_F32 : std::is_same<T, __half>::value ? EMU_F16 : EMU_BF16;
    // Blocks for a segment's rows: eight rows each, or one where so few segments share the CTAs that they have many parts.
    const unsigned rows = max_rows < ROWS ? (unsigned)max_rows : ROWS;
    const bool many = (int64_t)p.heads * (p.B < p.T ? p.B : p.T) * 4 < ctas;
    return launch_join(dtype, p, ctas, many ? rows : (rows + 7) / 8, stream);
}

template <typename T, int NR>
cudaError_t launch_rows(const AttnParams& p, const emu_kv_cache_t& c, int64_t max_rows, DeviceState* d, cudaStream_t stream) {
    if (p.D == 64) return launch_decode<T, 1, 64, NR>(p, c, max_rows, d, stream);
    if (p.D == 128) return launch_decode<T, 2, 128, NR>(p, c, max_rows, d, stream);
    if (p.D == 256) return launch_decode<T, 4, 256, NR>(p, c, max_rows, d, stream);
    if (p.D < 64) return launch_decode<T, 1, 0, NR>(p, c, max_rows, d, stream);
    if (p.D < 128) return launch_decode<T, 2, 0, NR>(p, c, max_rows, d, stream);
    if (p.D <= 192) return launch_decode<T, 3, 0, NR>(p, c, max_rows, d, stream);
    return launch_decode<T, 4, 0, NR>(p, c, max_rows, d, stream);
}

template <typename T>
cudaError_t launch_join_typed(const AttnParams& p, unsigned ctas, unsigned rows, cudaStream_t stream) {
    cudaLaunchConfig_t how = {};
    how.gridDim = dim3(ctas, rows);
    how.blockDim = dim3(kJoinWarps * 32);
    how.stream = stream;
    cudaLaunchAttribute dependent = {};
    dependent.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dependent.val.programmaticStreamSerializationAllowed = 1;
    how.attrs = &dependent;
    how.numAttrs = 1;
    return cudaLaunchKernelEx(&how, kv_join_kernel<T>, p);
}

template <typename T>
cudaError_t launch_typed(const AttnParams& p, const emu_kv_cache_t& c, int64_t max_rows, DeviceState* d, cudaStream_t stream) {
    return max_rows <= 8 ? launch_rows<T, 1>(p, c, max_rows, d, stream) : launch_rows<T, 2>(p, c, max_rows, d, stream);
}

}  // namespace

cudaError_t launch_join(int dtype, const AttnParams& p, unsigned ctas, unsigned rows, cudaStream_t stream) {
    if (dtype == EMU_F32) return launch_join_typed<float>(p, ctas, rows, stream);
    if (dtype == EMU_BF16) return launch_join_typed<__nv_bfloat16>(p, ctas, rows, stream);
    return launch_join_typed<__half>(p, ctas, rows, stream);
}

}  // namespace emu

using namespace emu;

extern "C" emu_status_t emu_kv_attention(int dtype, int64_t T, const emu_heads_t* q, const emu_heads_t* out,
                                         const emu_kv_cache_t* cache, int64_t B, const int32_t* table, int64_t width,
                                         const int32_t* starts, const int32_t* lengths, float scale, int64_t window,
                                         int64_t max_new, emu_stream_t stream_) {
    constexpr int64_t most = int64_t(1) << 40;
    if (dtype < EMU_F32 || dtype > EMU_F16 || !q || !out || !cache || !kv_cache_ok(*cache)) return EMU_ERR_INVALID_VALUE;
    // (a tile's end, 128 tokens on, and what rounds up to one stay below 2^31)
    if (T < 0 || T > kKvMaxRows || B < 0 || B > 1 << 20 || width < 0 || width > (INT32_MAX - 255) / cache->page || window < 0 ||
        max_new < 0 || !(scale - scale == 0.0f))
        return EMU_ERR_INVALID_VALUE;
    if (q->heads < 1 || q->heads > 65536 || q->heads % cache->heads != 0 || out->heads != q->heads)
        return EMU_ERR_INVALID_VALUE;
    for (const emu_heads_t* h : {q, out})
        if (h->token_stride < -most || h->token_stride > most || h->head_stride < -most || h->head_stride > most ||
            (T > 0 && !h->data))
            return EMU_ERR_INVALID_VALUE;
    if (T > 0 && B > 0 && (!starts || !lengths || (width > 0 && !table))) return EMU_ERR_INVALID_VALUE;
    if (T * (q->heads / cache->heads) > INT32_MAX - 256) return EMU_ERR_INVALID_VALUE;
    if (T == 0) return EMU_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    emu_status_t st = current_device(&d);
    if (st != EMU_OK) return st;
    // Made once, for the largest head and grid, so that no later call moves what a captured one reads.
    const size_t ctas = (size_t)d->sms * kKvCtasPerSm;
    const size_t few = 2 * ctas * 16 * (256 + 4) * sizeof(float), many = 2 * (size_t)d->sms * kKvSlotRows * (128 + 4) * sizeof(float);
    const size_t slots = few > many ? few : many;
    const size_t moved = ctas * kWarps * kMovedQuads * 32 * sizeof(float4);      // (kv_prompt.cu: 2 SMs 128 x 128 values, fewer)
    static_assert(kKvCtasPerSm * kWarps * kMovedQuads * 32 * sizeof(float4) >= 2 * 128 * 128 * sizeof(float), "sums of both kernels");
    if (!d->kv_ws && cudaMalloc(&d->kv_ws, slots + moved + ctas * sizeof(Work)) != cudaSuccess) {
        cudaGetLastError();
        d->kv_ws = nullptr;
        return EMU_ERR_ALLOC;
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
    p.wide_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.out_t * size % 16 == 0 && p.out_h * size % 16 == 0;
    p.partial = static_cast<float*>(d->kv_ws);
    p.moved = reinterpret_cast<float4*>(static_cast<uint8_t*>(d->kv_ws) + slots);
    p.shared = reinterpret_cast<Work*>(static_cast<uint8_t*>(d->kv_ws) + slots + moved);
    p.err = d->err;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int64_t max_rows = (max_new > 0 && max_new < T ? max_new : T) * p.group;
    cudaError_t e;
    if (max_rows > (dtype == EMU_F32 ? 16 : kFewKvRows) && p.D <= 128) e = launch_prompt(dtype, p, max_rows, d->sms, stream);
    else if (dtype == EMU_F32) e = launch_typed<float>(p, *cache, max_rows, d, stream);
    else if (dtype == EMU_BF16) e = launch_typed<__nv_bfloat16>(p, *cache, max_rows, d, stream);
    else e = launch_typed<__half>(p, *cache, max_rows, d, stream);
    return from_cuda(e);
}
