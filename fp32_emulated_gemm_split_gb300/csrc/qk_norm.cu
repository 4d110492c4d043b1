// qk_norm.cu -- norm of each query and key head with the position rotation
// in the same pass, forward and backward (include/emu_layers.h).
//
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps),   y = R(p) n
//   dn = R(p)^T dy,  dw = sum dn x r,  dx = r (dn w - x r^2 mean(dn w x))
//
// Bound by HBM: the forward reads and writes each head once, the backward
// reads x and dy and writes dx.  Everything else stays in registers, so the
// layout is made for that: the values of a head are taken as D/2 pairs, the
// rotated ones (j, j + rot/2) or (2j, 2j + 1), the rest (rot + j, rot + rest/2
// + j); a lane holds V neighbouring pairs (two 16-byte loads for V = 16 bytes
// of the type), so a rotation needs no other lane, and D/2/V lanes (rounded
// up to a power of two, at most a warp) hold a head.  A warp takes one token
// and a range of its heads, 32 / lanes of them at a time: its cosines, sines
// and weights are read once and kept in registers.
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

struct Heads {
    const void* in;
    const void* dy;          // backward: the gradient of the output
    void* out;               // forward: y; backward: dx
    int64_t in_t, in_h, dy_t, dy_h, out_t, out_h;
    const float* w;
    int heads;
};

struct QkParams {
    Heads side[2];           // queries, keys
    int64_t T;
    int D, rot, lanes;       // lanes per head, a power of two
    int segments;            // ranges of heads that a token is cut into
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

// Where the pair chunk of lane position c (pairs c V .. c V + V - 1) lies:
// first and second elements' offsets in the head, and whether they exist.
// An odd rest (V = 1 only) leaves the last pair without a second element.
template <int V, bool PAIRS>
struct Chunk {
    int a, b, j;             // offsets of the first elements; rotary index
    bool rotated, has_a, has_b;
    __device__ __forceinline__ Chunk(int c, int D, int rot) {
        const int p = c * V, half = rot / 2, rest = D - rot, q = p - half;
        rotated = p < half;
        j = p;
        if (rotated) {
            a = PAIRS ? 2 * p : p;
            b = PAIRS ? 2 * p + V : p + half;
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

// The chunk as it lies in memory, and its 2 V values as x[i] (first elements)
// and x[V + i] (second).  Rotated neighbouring pairs lie as a0 b0 a1 b1 ..: two
// vectors in a row.
template <typename T, int V>
struct Raw {
    Vec<T, V> a, b;
};
template <typename T, int V, bool PAIRS>
__device__ __forceinline__ Raw<T, V> load_chunk(const T* head, const Chunk<V, PAIRS>& ck, bool in) {
    Raw<T, V> r = {};
    if (in && ck.has_a) r.a = *reinterpret_cast<const Vec<T, V>*>(head + ck.a);
    if (in && ck.has_b) r.b = *reinterpret_cast<const Vec<T, V>*>(head + ck.b);
    return r;
}
template <typename T, int V, bool PAIRS>
__device__ __forceinline__ void unpack_chunk(const Raw<T, V>& r, const Chunk<V, PAIRS>& ck, float (&x)[2 * V]) {
    if (PAIRS && ck.rotated) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = to_f32(2 * i < V ? r.a.v[(2 * i) % V] : r.b.v[(2 * i) % V]);
            x[V + i] = to_f32(2 * i + 1 < V ? r.a.v[(2 * i + 1) % V] : r.b.v[(2 * i + 1) % V]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = to_f32(r.a.v[i]);
            x[V + i] = to_f32(r.b.v[i]);
        }
    }
}

template <typename T, int V, bool PAIRS>
__device__ __forceinline__ void store_chunk(T* head, const Chunk<V, PAIRS>& ck, const float (&y)[2 * V]) {
    Vec<T, V> a, b;
    if (PAIRS && ck.rotated) {
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
            const T v = from_f32<T>(y[(e & 1) * V + e / 2]);
            if (e < V) a.v[e % V] = v;
            else b.v[e % V] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a.v[i] = from_f32<T>(y[i]);
            b.v[i] = from_f32<T>(y[V + i]);
        }
    }
    if (ck.has_a) *reinterpret_cast<Vec<T, V>*>(head + ck.a) = a;
    if (ck.has_b) *reinterpret_cast<Vec<T, V>*>(head + ck.b) = b;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Cosines and sines of a chunk at position `pos` (NaN out of the table; 1, 0
// where nothing is rotated).
template <int V, bool PAIRS>
__device__ __forceinline__ void load_turn(const QkParams& p, int64_t pos, bool pos_ok,
                                          const Chunk<V, PAIRS>& ck, float (&cs)[V], float (&sn)[V]) {
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

template <int V, bool PAIRS>
__device__ __forceinline__ void load_weight(const float* w, const Chunk<V, PAIRS>& ck, float (&x)[2 * V]) {
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) x[i] = 1.0f;
    if (w && ck.has_a)
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = w[PAIRS && ck.rotated ? ck.a + 2 * i : ck.a + i];
    if (w && ck.has_b)
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[V + i] = w[PAIRS && ck.rotated ? ck.a + 2 * i + 1 : ck.b + i];
}

constexpr int kWarps = 8;                    // per block

// V pairs per chunk, NC chunks per lane, U rounds of heads read ahead of
// their arithmetic (HBM's latency: each round is 32 bytes per lane and tensor).
template <typename T, int V, int NC, bool PAIRS, bool BWD, int U>
__global__ void __launch_bounds__(kWarps * 32, 2) qk_norm_kernel(const QkParams p) {
    extern __shared__ float dw_sum[];                            // backward: [warp][2][D]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / p.lanes, pos_in = lane % p.lanes;   // head of the warp's group, lane in it
    const int at_once = 32 / p.lanes;
    const int64_t items = p.T * p.segments;
    const float inv_d = 1.0f / p.D;
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
        const Heads& hd = p.side[s];
        float w[NC][2 * V], dw[BWD ? NC : 1][BWD ? 2 * V : 1];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            load_weight<V, PAIRS>(hd.w, Chunk<V, PAIRS>(pos_in + n * p.lanes, p.D, p.rot), w[n]);
            if constexpr (BWD)
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) dw[n][i] = 0.0f;
        }
        const int per = (hd.heads + p.segments - 1) / p.segments;
        for (int64_t it = (int64_t)blockIdx.x * kWarps + warp; it < items;
             it += (int64_t)gridDim.x * kWarps) {
            const int64_t t = it / p.segments;
            const int seg = int(it - t * p.segments);
            const int h_end = min(hd.heads, (seg + 1) * per);
            if (seg * per >= h_end) continue;
            const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
            const bool pos_ok = pos >= 0 && pos < p.table_rows;
            if (!pos_ok && p.rot > 0 && lane == 0) record_error(p.err, kDevErrValue);
            float cs[NC][V], sn[NC][V];
#pragma unroll
            for (int n = 0; n < NC; ++n)
                load_turn<V, PAIRS>(p, pos, pos_ok, Chunk<V, PAIRS>(pos_in + n * p.lanes, p.D, p.rot), cs[n], sn[n]);
            const T* in = static_cast<const T*>(hd.in) + t * hd.in_t;
            const T* dy = static_cast<const T*>(hd.dy) + t * hd.dy_t;
            T* out = static_cast<T*>(hd.out) + t * hd.out_t;
            // every lane of the warp runs every round (the sums are shuffles)
            for (int h0 = seg * per; h0 < h_end; h0 += U * at_once) {
                Raw<T, V> rx[U][NC], rd[BWD ? U : 1][BWD ? NC : 1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * at_once + sub;
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        const Chunk<V, PAIRS> ck(pos_in + n * p.lanes, p.D, p.rot);
                        rx[u][n] = load_chunk<T, V, PAIRS>(in + h * hd.in_h, ck, h < h_end);
                        if constexpr (BWD) rd[u][n] = load_chunk<T, V, PAIRS>(dy + h * hd.dy_h, ck, h < h_end);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * at_once + sub;
                    float x[NC][2 * V], d[BWD ? NC : 1][BWD ? 2 * V : 1];
                    float ss = 0.0f, sd = 0.0f;
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        const Chunk<V, PAIRS> ck(pos_in + n * p.lanes, p.D, p.rot);
                        unpack_chunk<T, V, PAIRS>(rx[u][n], ck, x[n]);
#pragma unroll
                        for (int i = 0; i < 2 * V; ++i) ss = fmaf(x[n][i], x[n][i], ss);
                        if constexpr (BWD) {
                            unpack_chunk<T, V, PAIRS>(rd[u][n], ck, d[n]);
#pragma unroll
                            for (int i = 0; i < V; ++i) {        // turned back
                                const float a = d[n][i], b = d[n][V + i];
                                d[n][i] = fmaf(a, cs[n][i], b * sn[n][i]);
                                d[n][V + i] = fmaf(b, cs[n][i], -(a * sn[n][i]));
                            }
#pragma unroll
                            for (int i = 0; i < 2 * V; ++i) sd = fmaf(d[n][i] * w[n][i], x[n][i], sd);
                        }
                    }
                    ss = lanes_sum(ss, p.lanes);
                    const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                    if constexpr (BWD) {
                        sd = lanes_sum(sd, p.lanes);
                        const float m = r * r * (sd * inv_d);
                        const bool live = h < h_end;
#pragma unroll
                        for (int n = 0; n < NC; ++n) {
                            const Chunk<V, PAIRS> ck(pos_in + n * p.lanes, p.D, p.rot);
#pragma unroll
                            for (int i = 0; i < 2 * V; ++i) {
                                if (live) dw[n][i] = fmaf(d[n][i], x[n][i] * r, dw[n][i]);
                                d[n][i] = r * fmaf(d[n][i], w[n][i], -(x[n][i] * m));
                            }
                            if (live) store_chunk<T, V, PAIRS>(out + h * hd.out_h, ck, d[n]);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NC; ++n) {
                            const Chunk<V, PAIRS> ck(pos_in + n * p.lanes, p.D, p.rot);
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const float a = x[n][i] * r * w[n][i], b = x[n][V + i] * r * w[n][V + i];
                                x[n][i] = fmaf(a, cs[n][i], -(b * sn[n][i]));
                                x[n][V + i] = fmaf(b, cs[n][i], a * sn[n][i]);
                            }
                            if (h < h_end) store_chunk<T, V, PAIRS>(out + h * hd.out_h, ck, x[n]);
                        }
                    }
                }
            }
        }
        if constexpr (BWD) {
            // over the warp's heads
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const Chunk<V, PAIRS> ck(pos_in + n * p.lanes, p.D, p.rot);
#pragma unroll
                for (int i = 0; i < 2 * V; ++i) {
                    float v = dw[n][i];
                    for (int o = p.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    const bool second = i >= V;
                    if (sub == 0 && (second ? ck.has_b : ck.has_a)) {
                        const int e = PAIRS && ck.rotated ? ck.a + 2 * (i % V) + (second ? 1 : 0)
                                                          : (second ? ck.b + i - V : ck.a + i);
                        dw_sum[(warp * 2 + s) * p.D + e] = v;
                    }
                }
            }
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

constexpr int kBlocksPerSm = 2;

template <typename T, int V, int NC, bool PAIRS, bool BWD, int U>
cudaError_t launch_one(const QkParams& p, int blocks, cudaStream_t stream) {
    const size_t smem = BWD ? (size_t)kWarps * 2 * p.D * sizeof(float) : 0;
    qk_norm_kernel<T, V, NC, PAIRS, BWD, U><<<blocks, kWarps * 32, smem, stream>>>(p);
    return cudaGetLastError();
}

// The widest chunk that the head's layout allows: V pairs per lane position
// where both parts of the head are whole chunks and every row starts on a
// boundary of V elements (and the tables on 16 bytes); one pair otherwise.
template <typename T, bool PAIRS, bool BWD>
cudaError_t launch_typed(QkParams p, int max_blocks, int* blocks, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    bool wide = p.rot % (2 * V) == 0 && (p.D - p.rot) % (2 * V) == 0;
    auto whole = [&](const void* q, int64_t ts, int64_t hs) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ts % V == 0 && hs % V == 0;
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
    // few tokens: cut each one's heads into ranges until the warps fill the GPU
    const int rounds = (p.side[0].heads * p.lanes + 31) / 32 + (p.side[1].heads * p.lanes + 31) / 32;
    p.segments = 1;
    while (p.segments * 2 <= rounds && p.T * p.segments < (int64_t)max_blocks * kWarps) p.segments *= 2;
    const int64_t want = (p.T * p.segments + kWarps - 1) / kWarps;
    *blocks = (int)(want < max_blocks ? want : max_blocks);
    constexpr int U = BWD ? 2 : 4;
    if (wide) {
        if (nc == 1) return launch_one<T, V, 1, PAIRS, BWD, U>(p, *blocks, stream);
        return launch_one<T, V, 2, PAIRS, BWD, U / 2>(p, *blocks, stream);
    }
    if (nc <= 2) return launch_one<T, 1, 2, PAIRS, BWD, U>(p, *blocks, stream);
    return launch_one<T, 1, 8, PAIRS, BWD, 1>(p, *blocks, stream);
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
    if (T < 0 || T > INT32_MAX || D < 1 || D > 512 || rot < 0 || rot > D || rot % 2 != 0 || !(eps >= 0.0f))
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
    return from_cuda(launch_any<false>(dtype, interleaved != 0, p, d->sms * kBlocksPerSm, &blocks,
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
    const int max_blocks = d->sms * kBlocksPerSm;
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
