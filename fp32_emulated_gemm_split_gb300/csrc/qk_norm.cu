// qk_norm.cu -- norm of each query and key head with the position rotation
// in the same pass, forward and backward (include/emu_layers.h).
//
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps),   y = R(p) n
//   dn = R(p)^T dy,  dw = sum dn x r,  dx = r (dn w - x r^2 mean(dn w x))
//
// Bound by HBM: the forward reads and writes each head once, the backward
// reads x and dy and writes dx.  Everything else stays in registers, so the
// layout is made for that.  Halves: the values of a head are taken as D/2 pairs,
// the rotated ones (j, j + rot/2), the rest (rot + j, rot + rest/2 + j); a lane
// holds V neighbouring pairs (two loads of V values).  Neighbouring pairs (2j,
// 2j + 1): a lane holds 2 V values in a row.  So a rotation needs no other lane,
// and D/2/V lanes (rounded up to a power of two, at most a warp) hold a head.  A
// warp walks a range of heads, 32 / lanes of them at a time: the weights, and a
// token's cosines and sines, are read once and kept in registers.
//
// What a round costs beyond the bytes are its instructions: values stay packed
// in pairs as they lie in memory (fma.rn.f32x2), and where the layout allows it
// no copy or load is guarded (a lane without a chunk, or a head past the end,
// does another's and stores nothing).
//
// The weights' gradients are summed per lane over the tokens of its warp,
// then over the block in shared memory, and one row per block goes to the
// workspace; a second kernel adds the rows in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"

namespace emu {
namespace {

constexpr int kMaxD = 512;                   // values of a head

struct Heads {
    const void* in;
    const void* dy;          // backward: the gradient of the output
    void* out;               // forward: y; backward: dx
    int64_t in_t, in_h, dy_t, dy_h, out_t, out_h;
    const float* w;
    int heads;
    int per_token;           // rounds of a token
    int per_warp, one_more;  // rounds of a warp; the first one_more warps do one more
};

struct QkParams {
    Heads side[2];           // queries, keys
    int64_t T;
    int D, rot, lanes;       // lanes per head, a power of two
    float eps;
    const float *cos, *sin;
    int64_t table_rows;
    const int32_t* positions;
    float* partial;          // backward: [block][2][D] sums of dw
    int* err;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// N neighbouring elements as one access of their size (at most 16 bytes)
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

// Packed pairs of FP32 values (half the instructions), and the 16-bit pairs
// of a 32-bit word as such: one or two instructions per pair.
__device__ __forceinline__ uint64_t pk(float lo, float hi) {
    return pack_f32x2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }
template <typename T> __device__ __forceinline__ uint64_t widen(uint32_t w);
template <> __device__ __forceinline__ uint64_t widen<__nv_bfloat16>(uint32_t w) {
    return pack_f32x2(w << 16, w & 0xFFFF0000u);
}
template <> __device__ __forceinline__ uint64_t widen<__half>(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pk(f.x, f.y);
}
template <typename T> __device__ __forceinline__ uint32_t narrow(float lo, float hi);
template <> __device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t narrow<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Where the chunk of lane position c (pairs c V .. c V + V - 1) lies: first and
// second vectors' offsets in the head, and whether they exist.  An odd rest (V =
// 1 only) leaves the last pair without a second element.
template <int V, bool PAIRS>
struct Chunk {
    int a, b, j;             // offsets of the vectors; rotary index
    bool rotated, has_a, has_b;
    Chunk() = default;
    __device__ __forceinline__ Chunk(int c, int D, int rot) {
        const int p = c * V, half = rot / 2, rest = D - rot, q = p - half;
        rotated = p < half;
        j = p;
        if (PAIRS) {
            a = 2 * p;
            b = a + V;
            has_a = a < D;
            has_b = b < D;
        } else if (rotated) {
            a = p;
            b = p + half;
            has_a = has_b = true;
        } else {
            const int up = (rest + 1) / 2;
            a = rot + q;
            b = rot + up + q;
            has_a = q < up;
            has_b = q < up && up + q < rest;
        }
    }
};

// A lane's chunk as it lies in memory: two vectors (of neighbouring pairs: in a row).
template <typename T, int V>
struct alignas(sizeof(T) * V >= 16 || V == 1 ? sizeof(T) * V : 2 * sizeof(T) * V) Raw {
    Vec<T, V> a, b;
};
template <typename T, int V, int NC, bool PAIRS>
__device__ __forceinline__ void load_chunks(const T* head, const Chunk<V, PAIRS> (&ck)[NC], bool in,
                                            Raw<T, V> (&r)[NC]) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        r[n] = {};
        if (in && ck[n].has_a) r[n].a = *reinterpret_cast<const Vec<T, V>*>(head + ck[n].a);
        if (in && ck[n].has_b) r[n].b = *reinterpret_cast<const Vec<T, V>*>(head + ck[n].b);
    }
}

// One access for both vectors where they lie in a row and make up to 16 bytes.
template <typename T, int V, bool PAIRS>
constexpr bool kJoined = PAIRS && V > 1 && 2 * V * sizeof(T) <= 16;

// The same by asynchronous copies into this thread's own slots of shared
// memory (GUARD: zeros where there is nothing), and back: a thread reads only
// what it copied itself, so its own wait for the copies is all the order needed.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool in) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;"
                     :: "r"(dst), "l"(src), "n"(BYTES), "r"(in ? BYTES : 0) : "memory");
}
template <typename T, int V, int NC, bool PAIRS, bool GUARD>
__device__ __forceinline__ void copy_chunks(const T* head, const Chunk<V, PAIRS> (&ck)[NC], bool in,
                                            uint32_t slot, uint32_t step) {
    constexpr int B = sizeof(T) * V;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const bool a = !GUARD || (in && ck[n].has_a), b = !GUARD || (in && ck[n].has_b);
        if constexpr (kJoined<T, V, PAIRS>) {
            copy_async<2 * B>(slot + n * step, a ? head + ck[n].a : head, a);
        } else {
            copy_async<B>(slot + 2 * n * step, a ? head + ck[n].a : head, a);
            copy_async<B>(slot + (2 * n + 1) * step, b ? head + ck[n].b : head, b);
        }
    }
}
template <typename T, int V, int NC, bool PAIRS>
__device__ __forceinline__ void read_chunks(const uint8_t* slot, uint32_t step, Raw<T, V> (&r)[NC]) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        if constexpr (kJoined<T, V, PAIRS>) {
            r[n] = *reinterpret_cast<const Raw<T, V>*>(slot + n * step);
        } else {
            r[n].a = *reinterpret_cast<const Vec<T, V>*>(slot + 2 * n * step);
            r[n].b = *reinterpret_cast<const Vec<T, V>*>(slot + (2 * n + 1) * step);
        }
    }
}

// A lane's NC V pairs of values, packed: for wide chunks as they lie in memory,
// those of a chunk's first vector and then of its second; V = 1: the first
// elements of two chunks and then their second ones (neighbouring pairs: a
// chunk's own two).
template <typename T, int V, int NC, bool PAIRS>
__device__ __forceinline__ void unpack(const Raw<T, V> (&r)[NC], uint64_t (&x)[NC * V]) {
    if constexpr (V == 1 && PAIRS) {
#pragma unroll
        for (int n = 0; n < NC; ++n) x[n] = pk(to_f32(r[n].a.v[0]), to_f32(r[n].b.v[0]));
    } else if constexpr (V == 1) {
#pragma unroll
        for (int n = 0; n < NC; n += 2) {
            x[n] = pk(to_f32(r[n].a.v[0]), to_f32(r[n + 1].a.v[0]));
            x[n + 1] = pk(to_f32(r[n].b.v[0]), to_f32(r[n + 1].b.v[0]));
        }
    } else {
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Vec<T, V>& from = i < V / 2 ? r[n].a : r[n].b;
                const int at = i % (V / 2);
                if constexpr (sizeof(T) == 4) x[n * V + i] = pk(from.v[2 * at], from.v[2 * at + 1]);
                else x[n * V + i] = widen<T>(reinterpret_cast<const uint32_t*>(from.v)[at]);
            }
    }
}

template <typename T, int V, int NC, bool PAIRS, bool GUARD>
__device__ __forceinline__ void store_chunks(T* head, const Chunk<V, PAIRS> (&ck)[NC], const uint64_t (&x)[NC * V]) {
    if constexpr (V == 1) {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const float a = PAIRS ? lo_of(x[n]) : n & 1 ? hi_of(x[n - 1]) : lo_of(x[n]);
            const float b = PAIRS ? hi_of(x[n]) : n & 1 ? hi_of(x[n]) : lo_of(x[n + 1]);
            if (ck[n].has_a) head[ck[n].a] = from_f32<T>(a);
            if (ck[n].has_b) head[ck[n].b] = from_f32<T>(b);
        }
    } else {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            Raw<T, V> r;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                Vec<T, V>& to = i < V / 2 ? r.a : r.b;
                const int at = i % (V / 2);
                const uint64_t v = x[n * V + i];
                if constexpr (sizeof(T) == 4) {
                    to.v[2 * at] = lo_of(v);
                    to.v[2 * at + 1] = hi_of(v);
                } else {
                    reinterpret_cast<uint32_t*>(to.v)[at] = narrow<T>(lo_of(v), hi_of(v));
                }
            }
            if constexpr (kJoined<T, V, PAIRS>) {
                if (!GUARD || ck[n].has_a) *reinterpret_cast<Raw<T, V>*>(head + ck[n].a) = r;
            } else {
                if (!GUARD || ck[n].has_a) *reinterpret_cast<Vec<T, V>*>(head + ck[n].a) = r.a;
                if (!GUARD || ck[n].has_b) *reinterpret_cast<Vec<T, V>*>(head + ck[n].b) = r.b;
            }
        }
    }
}

// Turns a lane's pairs, coefficients k1 and k2:
//   halves: first' = first k1[first] + second k2[second], second' = second k1[second] + first k2[first]
//   neighbouring pairs: (a, b)' = (a, b) k1 + (b, a) k2
// and makes the coefficients from a lane's cosines c and sines s (of the turn, or
// of its reverse with -s) and weights (as pairs; null: ones).
template <int V, int NC>
struct Halves {                                      // the k-th first and second vector's pair
    static constexpr int a(int k) { return V == 1 ? 2 * k : k / (V / 2) * V + k % (V / 2); }
    static constexpr int b(int k) { return V == 1 ? 2 * k + 1 : a(k) + V / 2; }
};
template <int V, int NC, bool PAIRS>
__device__ __forceinline__ void make_turn(const float* c, const float* s, float sign, const uint64_t* w,
                                          uint64_t (&k1)[NC * V], uint64_t (&k2)[NC * V]) {
    using H = Halves<V, NC>;
    if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < NC * V; ++e) {
            const float wa = w ? lo_of(w[e]) : 1.0f, wb = w ? hi_of(w[e]) : 1.0f, sn = sign * s[e];
            k1[e] = pk(wa * c[e], wb * c[e]);
            k2[e] = pk(-wb * sn, wa * sn);
        }
    } else {
#pragma unroll
        for (int k = 0; k < NC * V / 2; ++k) {
            const uint64_t cc = pk(c[2 * k], c[2 * k + 1]), sp = pk(sign * s[2 * k], sign * s[2 * k + 1]);
            const uint64_t sm = pk(-sign * s[2 * k], -sign * s[2 * k + 1]);
            k1[H::a(k)] = w ? mul_f32x2(w[H::a(k)], cc) : cc;
            k1[H::b(k)] = w ? mul_f32x2(w[H::b(k)], cc) : cc;
            k2[H::a(k)] = w ? mul_f32x2(w[H::a(k)], sp) : sp;
            k2[H::b(k)] = w ? mul_f32x2(w[H::b(k)], sm) : sm;
        }
    }
}
template <int V, int NC, bool PAIRS>
__device__ __forceinline__ void turn(uint64_t (&x)[NC * V], const uint64_t (&k1)[NC * V], const uint64_t (&k2)[NC * V]) {
    using H = Halves<V, NC>;
    if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < NC * V; ++e)
            x[e] = fma_f32x2(pk(hi_of(x[e]), lo_of(x[e])), k2[e], mul_f32x2(x[e], k1[e]));
    } else {
#pragma unroll
        for (int k = 0; k < NC * V / 2; ++k) {
            const uint64_t a = x[H::a(k)], b = x[H::b(k)];
            x[H::a(k)] = fma_f32x2(b, k2[H::b(k)], mul_f32x2(a, k1[H::a(k)]));
            x[H::b(k)] = fma_f32x2(a, k2[H::a(k)], mul_f32x2(b, k1[H::b(k)]));
        }
    }
}

// Cosines and sines of a chunk at position `pos` (NaN out of the table; 1, 0
// where nothing is rotated).
template <int V, bool PAIRS>
__device__ __forceinline__ void load_turn(const QkParams& p, int64_t pos, bool pos_ok,
                                          const Chunk<V, PAIRS>& ck, float* cs, float* sn) {
    const float bad = __uint_as_float(0x7FC00000u);
    Vec<float, V> c, s;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c.v[i] = ck.rotated ? bad : 1.0f;
        s.v[i] = ck.rotated ? bad : 0.0f;
    }
    if (ck.rotated && pos_ok) {
        const int64_t o = pos * (p.rot / 2) + ck.j;
        // (V = 8: two 16-byte loads)
        constexpr int L = V < 4 ? V : 4;
#pragma unroll
        for (int i = 0; i < V; i += L) {
            const Vec<float, L> cl = *reinterpret_cast<const Vec<float, L>*>(p.cos + o + i);
            const Vec<float, L> sl = *reinterpret_cast<const Vec<float, L>*>(p.sin + o + i);
#pragma unroll
            for (int l = 0; l < L; ++l) {
                c.v[i + l] = cl.v[l];
                s.v[i + l] = sl.v[l];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        cs[i] = c.v[i];
        sn[i] = s.v[i];
    }
}

// The weights of a lane's chunks, as pairs like its values (ones where w is null).
template <int V, int NC, bool PAIRS>
__device__ __forceinline__ void load_weights(const float* w, const Chunk<V, PAIRS> (&ck)[NC], uint64_t (&out)[NC * V]) {
    Raw<float, V> r[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            r[n].a.v[i] = w && ck[n].has_a ? w[ck[n].a + i] : 1.0f;
            r[n].b.v[i] = w && ck[n].has_b ? w[ck[n].b + i] : 1.0f;
        }
    unpack<float, V, NC, PAIRS>(r, out);
}

// Rounds of heads in flight per warp: shared memory holds them, so that HBM's
// latency is covered by bytes on the way and not by registers.
constexpr int kWarps = 8;                    // per block
template <typename T, int V, int NC, bool PAIRS, bool BWD, int HU>
struct Ring {
    static constexpr int copy = (kJoined<T, V, PAIRS> ? 2 : 1) * V * (int)sizeof(T);
    static constexpr bool used = copy >= 4;          // (cp.async copies 4, 8 or 16 bytes)
    static constexpr int per_tensor = (kJoined<T, V, PAIRS> ? 1 : 2) * NC;   // copies per lane and head
    static constexpr int per_head = per_tensor * (BWD ? 2 : 1);
    static constexpr int per_round = per_head * HU;
    static constexpr int step = kWarps * 32 * copy;  // from one copy's slots to the next
    static constexpr int depth = 3;
    static constexpr int bytes = used ? depth * per_round * step : 0;
};

// V pairs per chunk, NC chunks per lane and head, HU heads per lane and round.
// The rounds of heads (32 / lanes times HU at a time) of all tokens are shared evenly by the warps in consecutive ranges,
// first those of one side and then of the other.  (One range over both sides, most
// warps on one of them: 8 tokens no faster, 4099 12.0 -> 11.0, but 16384 tokens
// 61.0 -> 62.5 and 12001 37.3 -> 39.5.)
//
// Forward, with the weights folded into the cosines and sines once per token:
//   y_a = r (a (w_a c) - b (w_b s)),  y_b = r (b (w_b c) + a (w_a s)).
//
// LAYOUT kWhole: a head's chunks fit its lanes and whole rounds make up both
// sides: nothing is guarded (a lane without a chunk does the last one's and
// neither adds nor stores it).  kTail (forward): a head past the end reads the
// first one and is not stored.  kAny: every access is guarded.
enum { kAny, kTail, kWhole };
template <typename T, int V, int NC, bool PAIRS, bool BWD, int BPS, int LAYOUT, int HU>
__global__ void __launch_bounds__(kWarps * 32, BPS) qk_norm_kernel(const QkParams p) {
    static_assert(LAYOUT == kAny || NC == 1, "one chunk per lane");
    static_assert(!(BWD && LAYOUT == kTail), "what is read twice would count in dw");
    constexpr bool GUARD = LAYOUT == kAny;
    extern __shared__ __align__(16) uint8_t smem[];              // the rings; backward: then [warp][2][D]
    constexpr int E = NC * V;                                    // pairs a lane holds
    static_assert(E % 2 == 0, "pairs of values");
    using R = Ring<T, V, NC, PAIRS, BWD, HU>;
    constexpr uint32_t kStep = R::step;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / p.lanes, pos_in = lane % p.lanes;   // head of the warp's group, lane in it
    const int groups = 32 / p.lanes, at_once = groups * HU;      // heads of a warp's round: u groups + sub
    const int self = blockIdx.x * kWarps + warp;
    const float inv_d = 1.0f / p.D;
    uint8_t* mine = smem + threadIdx.x * R::copy;
    float* dw_sum = reinterpret_cast<float*>(smem + R::bytes);
    Chunk<V, PAIRS> ck[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n)
        ck[n] = Chunk<V, PAIRS>(GUARD ? pos_in + n * p.lanes : min(pos_in, p.D / (2 * V) - 1), p.D, p.rot);
    const bool mine_counts = GUARD || pos_in < p.D / (2 * V);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
        const Heads& hd = p.side[s];
        // this warp's range of the T x per_token rounds (divided on the host: the
        // 64-bit divisions took 0.3 to 1 us of a call here)
        const int per_token = hd.per_token;
        const int64_t begin = (int64_t)self * hd.per_warp + min(self, hd.one_more);
        int left = hd.per_warp + (self < hd.one_more);
        uint64_t w[E], dw[BWD ? E : 1];
        if constexpr (BWD)
#pragma unroll
            for (int e = 0; e < E; ++e) dw[e] = 0;
        int t = left > 0 ? begin <= UINT32_MAX ? int((uint32_t)begin / per_token) : int(begin / per_token) : 0;
        int round = left > 0 ? int(begin - (int64_t)t * per_token) : 0;
        // the copies' own walk over the rounds, R::depth ahead
        int to_copy = left, copy_at = round, filled = 0;
        const int64_t step_in = at_once * hd.in_h, step_dy = at_once * hd.dy_h;
        const int64_t wrap_in = hd.in_t - per_token * step_in, wrap_dy = hd.dy_t - per_token * step_dy;
        const T* copy_in = static_cast<const T*>(hd.in) + t * hd.in_t + round * step_in + sub * hd.in_h;
        const T* copy_dy = static_cast<const T*>(hd.dy) + t * hd.dy_t + round * step_dy + sub * hd.dy_h;
        auto copy_round = [&]() {
            if (to_copy > 0) {
                --to_copy;
                const uint32_t slot = smem_u32(mine) + filled * (R::per_round * kStep);
#pragma unroll
                for (int u = 0; u < HU; ++u) {
                    // (a head past the end: any address in range)
                    const bool in = LAYOUT == kWhole || copy_at * at_once + u * groups + sub < hd.heads;
                    copy_chunks<T, V, NC, PAIRS, GUARD>(in ? copy_in + u * groups * hd.in_h : static_cast<const T*>(hd.in),
                                                        ck, in, slot + u * R::per_head * kStep, kStep);
                    if constexpr (BWD)
                        copy_chunks<T, V, NC, PAIRS, GUARD>(in ? copy_dy + u * groups * hd.dy_h
                                                               : static_cast<const T*>(hd.dy),
                                                            ck, in, slot + (u * R::per_head + R::per_tensor) * kStep, kStep);
                }
                filled = filled + 1 == R::depth ? 0 : filled + 1;
                copy_in += step_in;
                if (BWD) copy_dy += step_dy;
                if (++copy_at == per_token) {                    // the next token
                    copy_at = 0;
                    copy_in += wrap_in;
                    if (BWD) copy_dy += wrap_dy;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if constexpr (R::used)
            for (int i = 0; i < R::depth; ++i) copy_round();
        int read = 0;
        // position, cosines and sines are read one token ahead
        auto pos_of = [&](int tok) { return p.rot > 0 && tok < p.T ? p.positions[tok] : 0; };
        float c[E], sn[E];
        auto turn_of = [&](int pos) {
            const bool ok = pos >= 0 && pos < p.table_rows;
            if (!ok && p.rot > 0 && lane == 0) record_error(p.err, kDevErrValue);
#pragma unroll
            for (int n = 0; n < NC; ++n) load_turn<V, PAIRS>(p, pos, ok, ck[n], c + n * V, sn + n * V);
        };
        // (after the first copies, none of which waits for these)
        const int pos = left > 0 ? pos_of(t) : 0;
        int next_pos = left > 0 ? pos_of(t + 1) : 0;
        load_weights<V, NC, PAIRS>(left > 0 ? hd.w : nullptr, ck, w);
        if (left > 0) turn_of(pos);
        while (left > 0) {
            const int here = min(left, per_token - round);       // rounds of this token
            left -= here;
            uint64_t k1[E], k2[E];
            make_turn<V, NC, PAIRS>(c, sn, BWD ? -1.0f : 1.0f, BWD ? nullptr : w, k1, k2);
            if (left > 0) {
                turn_of(next_pos);
                next_pos = pos_of(t + 2);
            }
            T* out = static_cast<T*>(hd.out) + t * hd.out_t + (round * at_once + sub) * hd.out_h;
            const int64_t step_out = at_once * hd.out_h;
            // every lane of the warp runs every round (the sums are shuffles)
            for (int i = 0; i < here; ++i, out += step_out) {
                Raw<T, V> rx[HU][NC], rd[HU][NC];
                auto live = [&](int u) {
                    return LAYOUT == kWhole || (round + i) * at_once + u * groups + sub < hd.heads;
                };
                if constexpr (R::used) {
                    asm volatile("cp.async.wait_group %0;" :: "n"(R::depth - 1) : "memory");
                    const uint8_t* slot = mine + read * (R::per_round * kStep);
#pragma unroll
                    for (int u = 0; u < HU; ++u) {
                        read_chunks<T, V, NC, PAIRS>(slot + u * R::per_head * kStep, kStep, rx[u]);
                        if constexpr (BWD)
                            read_chunks<T, V, NC, PAIRS>(slot + (u * R::per_head + R::per_tensor) * kStep, kStep, rd[u]);
                    }
                    read = read + 1 == R::depth ? 0 : read + 1;
                    copy_round();                                // into the slots just read
                } else {
#pragma unroll
                    for (int u = 0; u < HU; ++u) {
                        const int64_t h = (round + i) * at_once + u * groups + sub;
                        load_chunks<T, V, NC, PAIRS>(static_cast<const T*>(hd.in) + t * hd.in_t + h * hd.in_h, ck,
                                                     live(u), rx[u]);
                        if constexpr (BWD)
                            load_chunks<T, V, NC, PAIRS>(static_cast<const T*>(hd.dy) + t * hd.dy_t + h * hd.dy_h, ck,
                                                         live(u), rd[u]);
                    }
                }
                uint64_t x[HU][E], dn[BWD ? HU : 1][E];
                float ss[HU], sd[HU];
#pragma unroll
                for (int u = 0; u < HU; ++u) {
                    uint64_t q = 0;
                    unpack<T, V, NC, PAIRS>(rx[u], x[u]);
#pragma unroll
                    for (int e = 0; e < E; ++e) q = fma_f32x2(x[u][e], x[u][e], q);
                    ss[u] = mine_counts ? lo_of(q) + hi_of(q) : 0.0f;
                    if constexpr (BWD) {
                        // dn, the output's gradient turned back; its sum with w x
                        uint64_t z = 0;
                        unpack<T, V, NC, PAIRS>(rd[u], dn[u]);
                        turn<V, NC, PAIRS>(dn[u], k1, k2);
#pragma unroll
                        for (int e = 0; e < E; ++e) z = fma_f32x2(mul_f32x2(dn[u][e], w[e]), x[u][e], z);
                        sd[u] = mine_counts ? lo_of(z) + hi_of(z) : 0.0f;
                    }
                }
                for (int o = p.lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
                    for (int u = 0; u < HU; ++u) {
                        ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
                        if constexpr (BWD) sd[u] += __shfl_xor_sync(0xffffffffu, sd[u], o);
                    }
                }
#pragma unroll
                for (int u = 0; u < HU; ++u) {
                    const float r = rsqrtf(fmaf(ss[u], inv_d, p.eps));
                    const uint64_t rr = pk(r, r);
                    if constexpr (BWD) {
                        const float m = sd[u] * inv_d * r * r;
                        const uint64_t nm = pk(-m, -m);
                        // (a head past the end has no norm where eps is 0: 0 times infinity)
                        const bool counts = live(u);
#pragma unroll
                        for (int e = 0; e < E; ++e) {            // r (dn w - x m)
                            if (counts) dw[e] = fma_f32x2(dn[u][e], mul_f32x2(x[u][e], rr), dw[e]);
                            x[u][e] = mul_f32x2(rr, fma_f32x2(x[u][e], nm, mul_f32x2(dn[u][e], w[e])));
                        }
                    } else {
                        turn<V, NC, PAIRS>(x[u], k1, k2);
#pragma unroll
                        for (int e = 0; e < E; ++e) x[u][e] = mul_f32x2(rr, x[u][e]);
                    }
                    if (live(u) && mine_counts)
                        store_chunks<T, V, NC, PAIRS, GUARD>(out + u * groups * hd.out_h, ck, x[u]);
                }
            }
            round = 0;
            ++t;
        }
        if constexpr (R::used) asm volatile("cp.async.wait_group 0;" ::: "memory");
        if constexpr (BWD) {
            // over the warp's heads (lanes without a head added nothing)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float lo = lo_of(dw[e]), hi = hi_of(dw[e]);
                for (int o = p.lanes; o < 32; o <<= 1) {
                    lo += __shfl_xor_sync(0xffffffffu, lo, o);
                    hi += __shfl_xor_sync(0xffffffffu, hi, o);
                }
                dw[e] = pk(lo, hi);
            }
            if (sub == 0 && mine_counts) store_chunks<float, V, NC, PAIRS, GUARD>(dw_sum + (warp * 2 + s) * p.D, ck, dw);
        }
    }
    if constexpr (BWD) {
        // over the block's warps, in order
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * p.D; e += blockDim.x) {
            float v = 0.0f;
            for (int wp = 0; wp < kWarps; ++wp) v += dw_sum[wp * 2 * p.D + e];
            p.partial[(int64_t)blockIdx.x * 2 * p.D + e] = v;
        }
    }
}

// dwq and dwk: 32 columns per block, the first kernel's rows dealt to its 32
// warps and the warps' sums added in order.
__global__ void __launch_bounds__(1024) qk_norm_dw(const float* __restrict__ partial, int blocks, int D,
                                                   float* dwq, float* dwk) {
    __shared__ float part[32][33];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (e < 2 * D)
#pragma unroll 8
        for (int b = warp; b < blocks; b += 32) v += partial[(int64_t)b * 2 * D + e];
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && e < 2 * D) {
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) v += part[w][lane];
        float* dw = e < D ? dwq : dwk;
        if (dw) dw[e < D ? e : e - D] = v;
    }
}

template <bool BWD>
constexpr int kBlocksPerSm = 2;
template <typename T, bool BWD>
constexpr int kHeadsPerLane = sizeof(T) == 2 && !BWD ? 2 : 1;

template <typename T, int V, int NC, bool PAIRS, bool BWD, int BPS, int LAYOUT, int HU>
cudaError_t launch_one(QkParams p, int blocks, cudaStream_t stream) {
    constexpr int ring = Ring<T, V, NC, PAIRS, BWD, HU>::bytes, per_value = BWD ? kWarps * 2 * (int)sizeof(float) : 0;
    const int smem = ring + per_value * p.D;
    auto kern = qk_norm_kernel<T, V, NC, PAIRS, BWD, BPS, LAYOUT, HU>;
    for (Heads& h : p.side) {
        const int at_once = 32 / p.lanes * HU, warps = blocks * kWarps;
        h.per_token = (h.heads + at_once - 1) / at_once;
        h.per_warp = int(p.T * h.per_token / warps);
        h.one_more = int(p.T * h.per_token % warps);
    }
    if (ring + per_value * kMaxD > 48 << 10) {
        // the limit, raised once per device (g_mu is held)
        static bool done[kMaxDevices] = {};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && (dev >= kMaxDevices || !done[dev])) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring + per_value * kMaxD);
            if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
        }
        if (e != cudaSuccess) return e;
    }
    kern<<<blocks, kWarps * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

// The widest chunk that the head's layout allows: four pairs per lane position
// where both parts of the head are whole chunks and every row starts on a
// boundary of four elements (and the tables on 16 bytes); one pair otherwise.
// Measured, forward / backward, us: bfloat16, 16384 tokens x 40 heads x 128, 62 /
// 91 with four pairs, 67 / 112 with eight (whose cosines, sines and weights
// alone take 64 registers); float32, 8192 x 24 x 128, 39 / 56.  Two blocks per
// SM: 62 / 91; three 64 / 107; four 68 / 107.  Two heads per lane and round in
// the 16-bit forward pass: float16, neighbouring pairs, 12001 x 28 x 96, 42 ->
// 38; values packed as they lie and no guards: 37 / 62 -> 30 / 50 (a round took
// 327 instructions, two thirds of all issue slots).  Three chunks per lane where
// that leaves fewer lanes idle (96: 4 lanes of 3): 46 / 68, registers spilled.
// (Bytes at the HBM's rate: 49 / 74, 30 / 45, 19 / 29.)  Before the rings the
// loads waited in registers: 89 us forward.
template <typename T, bool PAIRS, bool BWD>
cudaError_t launch_typed(QkParams p, int max_blocks, int* blocks, cudaStream_t stream) {
    constexpr int V = 4;
    bool wide = p.rot % (2 * V) == 0 && (p.D - p.rot) % (2 * V) == 0;
    constexpr int kWide = kJoined<T, V, PAIRS> ? 2 * V : V;          // values of an access
    auto whole = [&](const void* q, int64_t ts, int64_t hs) {
        return reinterpret_cast<uintptr_t>(q) % (kWide * sizeof(T)) == 0 && ts % kWide == 0 && hs % kWide == 0;
    };
    for (const Heads& h : p.side)
        if (h.heads > 0)
            wide = wide && whole(h.in, h.in_t, h.in_h) && whole(h.out, h.out_t, h.out_h) &&
                   (!BWD || whole(h.dy, h.dy_t, h.dy_h));
    if (p.rot > 0)
        wide = wide && reinterpret_cast<uintptr_t>(p.cos) % 16 == 0 &&
               reinterpret_cast<uintptr_t>(p.sin) % 16 == 0;
    const int chunks = wide ? p.D / (2 * V) : p.rot / 2 + (p.D - p.rot + 1) / 2;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes < chunks) p.lanes *= 2;
    const int nc = (chunks + p.lanes - 1) / p.lanes;
    // a warp per round until they fill the GPU
    constexpr int BPS = kBlocksPerSm<BWD>, HU = kHeadsPerLane<T, BWD>;
    const int at_once = 32 / p.lanes * (wide && nc == 1 ? HU : 1);
    const int most = p.side[0].heads > p.side[1].heads ? p.side[0].heads : p.side[1].heads;
    const int64_t want = (p.T * ((most + at_once - 1) / at_once) + kWarps - 1) / kWarps;
    *blocks = (int)(want < max_blocks ? want : max_blocks);
    if (wide) {
        const bool whole_rounds = p.side[0].heads % at_once == 0 && p.side[1].heads % at_once == 0;
        if (nc == 1 && whole_rounds) return launch_one<T, V, 1, PAIRS, BWD, BPS, kWhole, HU>(p, *blocks, stream);
        if (nc == 1) return launch_one<T, V, 1, PAIRS, BWD, BPS, BWD ? kAny : kTail, HU>(p, *blocks, stream);
        return launch_one<T, V, 2, PAIRS, BWD, 1, kAny, 1>(p, *blocks, stream);
    }
    if (nc <= 2) return launch_one<T, 1, 2, PAIRS, BWD, BPS, kAny, 1>(p, *blocks, stream);
    return launch_one<T, 1, 8, PAIRS, BWD, 1, kAny, 1>(p, *blocks, stream);
}

template <bool BWD>
cudaError_t launch_any(int dtype, bool pairs, const QkParams& p, int max_blocks, int* blocks,
                       cudaStream_t stream) {
    auto go = [&](auto t) {
        using T = decltype(t);
        return pairs ? launch_typed<T, true, BWD>(p, max_blocks, blocks, stream)
                     : launch_typed<T, false, BWD>(p, max_blocks, blocks, stream);
    };
    if (dtype == EMU_F32) return go(float{});
    if (dtype == EMU_BF16) return go(__nv_bfloat16{});
    return go(__half{});
}

constexpr int64_t kMaxStride = int64_t(1) << 40;

bool heads_ok(const emu_heads_t& h, int64_t T) {
    if (h.heads < 0 || h.heads > 65536) return false;
    if (h.token_stride < -kMaxStride || h.token_stride > kMaxStride || h.head_stride < -kMaxStride ||
        h.head_stride > kMaxStride)
        return false;
    return h.heads == 0 || T == 0 || h.data != nullptr;
}

emu_status_t check_qk(int dtype, int64_t T, int64_t D, int64_t rot, int interleaved, float eps,
                      const emu_heads_t& q, const emu_heads_t& k, const emu_heads_t& qo,
                      const emu_heads_t& ko, const float* cos, const float* sin,
                      int64_t table_rows, const int32_t* positions) {
    if (dtype < EMU_F32 || dtype > EMU_F16 || (interleaved != 0 && interleaved != 1))
        return EMU_ERR_INVALID_VALUE;
    if (T < 0 || T > INT32_MAX / 64 || D < 1 || D > kMaxD || rot < 0 || rot > D || rot % 2 != 0 || !(eps >= 0.0f))
        return EMU_ERR_INVALID_VALUE;
    if (!heads_ok(q, T) || !heads_ok(k, T) || !heads_ok(qo, T) || !heads_ok(ko, T) ||
        qo.heads != q.heads || ko.heads != k.heads)
        return EMU_ERR_INVALID_VALUE;
    if (table_rows < 0 || table_rows > INT32_MAX) return EMU_ERR_INVALID_VALUE;
    if (rot > 0 && T > 0 && (!positions || (table_rows > 0 && (!cos || !sin)))) return EMU_ERR_INVALID_VALUE;
    return EMU_OK;
}

Heads make_side(const emu_heads_t& in, const emu_heads_t& out, const float* w, const emu_heads_t* dy) {
    Heads h = {};
    h.in = in.data; h.in_t = in.token_stride; h.in_h = in.head_stride;
    h.out = out.data; h.out_t = out.token_stride; h.out_h = out.head_stride;
    if (dy) { h.dy = dy->data; h.dy_t = dy->token_stride; h.dy_h = dy->head_stride; }
    h.w = w;
    h.heads = (int)in.heads;
    return h;
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_qk_norm_rope(int dtype, int64_t T, int64_t D, int64_t rot, int interleaved,
                              float eps, const emu_heads_t* heads, const float* wq,
                              const float* wk, const float* cos, const float* sin,
                              int64_t table_rows, const int32_t* positions, emu_stream_t stream) {
    if (!heads) return EMU_ERR_INVALID_VALUE;
    const emu_heads_t &q = heads[0], &k = heads[1];
    emu_status_t st = check_qk(dtype, T, D, rot, interleaved, eps, q, k, heads[2], heads[3], cos,
                               sin, table_rows, positions);
    if (st != EMU_OK) return st;
    if (T == 0 || q.heads + k.heads == 0) return EMU_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    st = current_device(&d);
    if (st != EMU_OK) return st;
    QkParams p = {};
    p.side[0] = make_side(q, heads[2], wq, nullptr);
    p.side[1] = make_side(k, heads[3], wk, nullptr);
    p.T = T; p.D = (int)D; p.rot = (int)rot; p.eps = eps;
    p.cos = cos; p.sin = sin; p.table_rows = table_rows; p.positions = positions;
    p.err = d->err;
    int blocks = 0;
    return from_cuda(launch_any<false>(dtype, interleaved != 0, p, d->sms * kBlocksPerSm<false>, &blocks,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

emu_status_t emu_qk_norm_rope_bwd(int dtype, int64_t T, int64_t D, int64_t rot, int interleaved,
                                  float eps, const emu_heads_t* heads, const float* wq,
                                  const float* wk, const float* cos, const float* sin,
                                  int64_t table_rows, const int32_t* positions, float* dwq,
                                  float* dwk, emu_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (!heads) return EMU_ERR_INVALID_VALUE;
    const emu_heads_t &q = heads[0], &k = heads[1];
    emu_status_t st = check_qk(dtype, T, D, rot, interleaved, eps, q, k, heads[2], heads[3], cos,
                               sin, table_rows, positions);
    if (st != EMU_OK) return st;
    if (!heads_ok(heads[4], T) || !heads_ok(heads[5], T) || heads[4].heads != q.heads ||
        heads[5].heads != k.heads)
        return EMU_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    st = current_device(&d);
    if (st != EMU_OK) return st;
    const int max_blocks = d->sms * kBlocksPerSm<true>;
    st = ensure_buffer(&d->ws, &d->ws_bytes, (size_t)max_blocks * 2 * D * sizeof(float));
    if (st != EMU_OK) return st;
    QkParams p = {};
    p.side[0] = make_side(q, heads[2], wq, &heads[4]);
    p.side[1] = make_side(k, heads[3], wk, &heads[5]);
    p.T = T; p.D = (int)D; p.rot = (int)rot; p.eps = eps;
    p.cos = cos; p.sin = sin; p.table_rows = table_rows; p.positions = positions;
    p.partial = static_cast<float*>(d->ws);
    p.err = d->err;
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (T > 0 && q.heads + k.heads > 0)
        e = launch_any<true>(dtype, interleaved != 0, p, max_blocks, &blocks, stream);
    if (e == cudaSuccess && (dwq || dwk)) {
        qk_norm_dw<<<(unsigned)((2 * D + 31) / 32), 1024, 0, stream>>>(p.partial, blocks,
                                                                             (int)D, dwq, dwk);
        e = cudaGetLastError();
    }
    return from_cuda(e);
}

}  // extern "C"
