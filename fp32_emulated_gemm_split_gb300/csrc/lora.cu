// lora.cu -- a projection with the low-rank adapters of many requests at once
// (include/emu_layers.h):  Y = X W^T + bias + scale_i (X A_i^T) B_i^T.
//
// Three steps: S[t] = A_i X[t] for every token with an adapter (down), Y[t] =
// bias + scale_i B_i S[t] (up), and the shared projection added to it by the
// emulated GEMM (beta = 1).  The adapters' steps group the tokens by adapter as
// they go: a block takes one adapter and one window of tokens, scans the
// window's indices, and works on the tokens of its own in order, so an
// adapter's rows are read once for all of them and no sorted copy of the tokens
// is made.  K is cut into slices so that few tokens, too, fill the GPU; the up
// step adds the slices in order.  Every output element is one fixed sum: where
// a token stands in the batch cannot change its result.
//
// Both steps are FP32 on the CUDA cores, in packed pairs (fma.rn.f32x2: twice
// the rate of single FMAs).  They are 2 R (K + N) of a token's 2 N K operations,
// under 1 % at rank 16 and N = K = 4096, at a third of the GEMM's rate.
#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"

namespace emu {
namespace {

struct LoraParams {
    int64_t M, N, K;
    int R, adapters;
    const float* X;
    int64_t ldx;
    const float *A, *B, *scale, *bias;
    const int32_t* index;
    float* S;                // slices x M x R
    int64_t slice;           // values of K per slice (a multiple of 64)
    int slices;
    float* Y;
    int64_t ldy;
    int* err;
};

constexpr int kWindow = 2048;                // tokens scanned by a block

// The tokens of window `win` whose adapter is `a` (a == adapters: those
// without one), in order, as offsets in the window; returns how many.  Called
// by all T threads of a block.
template <int T>
__device__ __forceinline__ int tokens_of(const LoraParams& p, int a, int64_t win, uint16_t* list) {
    __shared__ int warp_n[T / 32];
    constexpr int kPer = kWindow / T;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = win * kWindow;
    const int in = p.M - t0 < kWindow ? int(p.M - t0) : kWindow;
    // thread i looks at tokens i kPer .. i kPer + kPer - 1
    unsigned mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = threadIdx.x * kPer + j;
        if (i < in) {
            const int32_t v = p.index ? p.index[t0 + i] : -1;
            const bool none = v < 0 || v >= p.adapters;
            if (a == p.adapters ? none : v == a) mine |= 1u << j;
            if (a == p.adapters && none && v != -1) record_error(p.err, kDevErrValue);
        }
    }
    const int n = __popc(mine);
    int upto = n;                            // of this warp's lanes, this one included
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) warp_n[warp] = upto;
    __syncthreads();
    int at = upto - n, total = 0;
    for (int w = 0; w < T / 32; ++w) {
        if (w < warp) at += warp_n[w];
        total += warp_n[w];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (mine >> j & 1) list[at++] = (uint16_t)(threadIdx.x * kPer + j);
    __syncthreads();
    return total;
}

// ------------------------------------------------------------- down, dots --
//
// Few tokens: S[t][r] over one slice of K.  A warp takes two rows of A and
// four tokens at a time, its lanes stride over the slice (V neighbouring
// values each).  Bound by the latency of reading A's rows once.
constexpr int kDotWarps = 8, kDotTok = 4, kDotRows = 2;

template <int V>
__global__ void __launch_bounds__(kDotWarps * 32) lora_down_dots(const LoraParams p) {
    __shared__ uint16_t list[kWindow];
    const int a = blockIdx.x;
    const int64_t win = blockIdx.y;
    const int n = tokens_of<kDotWarps * 32>(p, a, win, list);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t k0 = blockIdx.z * p.slice, k1 = min(p.K, k0 + p.slice);
    float* S = p.S + blockIdx.z * p.M * p.R;
    for (int i0 = 0; i0 < n; i0 += kDotTok) {
        const float* row[kDotTok];
#pragma unroll
        for (int j = 0; j < kDotTok; ++j)    // past the end: the first token again, not stored
            row[j] = p.X + (win * kWindow + list[i0 + j < n ? i0 + j : i0]) * p.ldx;
        for (int r = warp * kDotRows; r < p.R; r += kDotWarps * kDotRows) {
            const float* ar = p.A + ((int64_t)a * p.R + r) * p.K;
            const float* ar1 = r + 1 < p.R ? ar + p.K : ar;
            float acc[kDotRows][kDotTok] = {};
#pragma unroll 2
            for (int64_t k = k0 + lane * V; k < k1; k += 32 * V) {
                float w[kDotRows][V], x[V];
                if constexpr (V == 4) {
                    *reinterpret_cast<float4*>(w[0]) = *reinterpret_cast<const float4*>(ar + k);
                    *reinterpret_cast<float4*>(w[1]) = *reinterpret_cast<const float4*>(ar1 + k);
                } else {
                    w[0][0] = ar[k];
                    w[1][0] = ar1[k];
                }
#pragma unroll
                for (int j = 0; j < kDotTok; ++j) {
                    if constexpr (V == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(row[j] + k);
                    else x[0] = row[j][k];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        acc[0][j] = fmaf(w[0][v], x[v], acc[0][j]);
                        acc[1][j] = fmaf(w[1][v], x[v], acc[1][j]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kDotRows; ++q)
#pragma unroll
                for (int j = 0; j < kDotTok; ++j) {
                    float v = acc[q][j];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    if (lane == 0 && i0 + j < n && r + q < p.R)
                        S[(win * kWindow + list[i0 + j]) * p.R + r + q] = v;
                }
        }
    }
}

// ------------------------------------------------------------ down, tiles --
//
// Many tokens: tiles of 64 tokens x 16 rows of A per warp, over one slice of
// K.  The block stages 64 values of K of its 64 tokens and of 16 G rows of A at
// a time in shared memory (two buffers, filled by cp.async); its 8 warps are G
// groups of 16 rows times 8 / G parts of each stage.  A lane owns 8 tokens x 4
// rows, each sum as a pair over even and odd k, which is how 16-byte loads
// along K leave the operands; rows are padded by four values, so the eight
// token groups of a load fall into different banks.  Bound by shared-memory
// loads: 12 of them per 64 packed FMAs.
constexpr int kTileTok = 64, kTileK = 64, kTileRow = kTileK + 4, kTileWarps = 8;
constexpr int kTileGroups = 4;               // z blocks that share a window's tiles

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(float* dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
constexpr int tile_smem(int G) { return 2 * (kTileTok + 16 * G) * kTileRow * 4; }

template <int V, int G>
__global__ void __launch_bounds__(kTileWarps * 32) lora_down_tiles(const LoraParams p) {
    extern __shared__ __align__(16) float stage[];   // [2][64 + 16 G][kTileRow]
    __shared__ uint16_t list[kWindow];
    constexpr int kRows = kTileTok + 16 * G, kParts = kTileWarps / G;
    const int a = blockIdx.x;
    const int64_t win = blockIdx.y;
    const int n = tokens_of<kTileWarps * 32>(p, a, win, list);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = warp % G, part = warp / G;
    const int tg = lane & 7, rg = lane >> 3;         // tokens tg + 8 i, rows rg + 4 j
    const int slice = blockIdx.z / kTileGroups;
    const int64_t k0 = slice * p.slice, k1 = min(p.K, k0 + p.slice);
    const int steps = int((k1 - k0 + kTileK - 1) / kTileK);
    float* S = p.S + slice * p.M * p.R;
    for (int i0 = (blockIdx.z % kTileGroups) * kTileTok; i0 < n; i0 += kTileGroups * kTileTok) {
        for (int r0 = 0; r0 < p.R; r0 += 16 * G) {
            auto fill = [&](int st) {
                float* dst = stage + (st & 1) * kRows * kTileRow;
                const int64_t k = k0 + (int64_t)st * kTileK;
                constexpr int per = kTileK / V;      // copies per row
                for (int e = tid; e < kRows * per; e += kTileWarps * 32) {
                    const int row = e / per, c = (e % per) * V;
                    const float* src;
                    bool in;
                    if (row < kTileTok) {
                        in = i0 + row < n;
                        src = p.X + (win * kWindow + list[in ? i0 + row : 0]) * p.ldx;
                    } else {
                        const int r = r0 + row - kTileTok;
                        in = r < p.R;
                        src = p.A + ((int64_t)a * p.R + (in ? r : 0)) * p.K;
                    }
                    in = in && k + c < k1;
                    if constexpr (V == 4) cp_async16(dst + row * kTileRow + c, src + (in ? k + c : 0), in);
                    else cp_async4(dst + row * kTileRow + c, src + (in ? k + c : 0), in);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            uint64_t acc[8][4] = {};
            fill(0);
            for (int st = 0; st < steps; ++st) {
                if (st + 1 < steps) {
                    fill(st + 1);
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                } else {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                }
                __syncthreads();
                const float* xs = stage + (st & 1) * kRows * kTileRow + tg * kTileRow;
                const float* as = stage + (st & 1) * kRows * kTileRow + (kTileTok + 16 * group + rg) * kTileRow;
#pragma unroll
                for (int c = 4 * part; c < kTileK; c += 4 * kParts) {
                    ulonglong2 av[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) av[j] = *reinterpret_cast<const ulonglong2*>(as + 4 * j * kTileRow + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(xs + 8 * i * kTileRow + c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[i][j] = fma_f32x2(x.x, av[j].x, acc[i][j]);
                            acc[i][j] = fma_f32x2(x.y, av[j].y, acc[i][j]);
                        }
                    }
                }
                __syncthreads();                     // the buffer is filled again
            }
            // the parts of K meet in shared memory, added in order
            float* sum = stage;                      // [part][group][64 tokens][16 rows]
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[((part * G + group) * kTileTok + tg + 8 * i) * 16 + rg + 4 * j] =
                        __uint_as_float(uint32_t(acc[i][j])) + __uint_as_float(uint32_t(acc[i][j] >> 32));
            __syncthreads();
            for (int e = tid; e < kTileTok * 16 * G; e += kTileWarps * 32) {
                const int t = e / (16 * G), r = e % (16 * G);
                float v = 0.0f;
#pragma unroll
                for (int q = 0; q < kParts; ++q)
                    v += sum[((q * G + r / 16) * kTileTok + t) * 16 + r % 16];
                if (i0 + t < n && r0 + r < p.R) S[(win * kWindow + list[i0 + t]) * p.R + r0 + r] = v;
            }
            __syncthreads();
        }
    }
}

// --------------------------------------------------------------------- up --
//
// Y[t][n] = bias[n] + scale sum_r B[n][r] S[t][r]: a thread takes C columns,
// kUpThreads apart (a warp writes 128 neighbouring bytes), keeps kUpRank
// values of each one's row of B in registers and walks up to kUpTok of the
// window's tokens of its adapter, whose S the block has put in shared memory
// (times the scale, the slices of K added in order); higher ranks take more
// passes, which add to Y.  Bound by the writes of Y.
constexpr int kUpThreads = 128, kUpRank = 16, kUpTok = 64, kUpGroups = 4;

template <int C>
__global__ void __launch_bounds__(kUpThreads) lora_up(const LoraParams p) {
    __shared__ uint16_t list[kWindow];
    __shared__ __align__(16) float s[kUpTok][kUpRank];
    const int a = blockIdx.x;
    const int64_t win = blockIdx.y;
    const int cnt = tokens_of<kUpThreads>(p, a, win, list);
    const int64_t n0 = (int64_t)(blockIdx.z / kUpGroups) * (C * kUpThreads) + threadIdx.x;
    const int R = a == p.adapters ? 0 : p.R;
    const float scale = R > 0 && p.scale ? p.scale[a] : 1.0f;
    float bias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t n = n0 + c * kUpThreads;
        bias[c] = p.bias && n < p.N ? p.bias[n] : 0.0f;
    }
    for (int i0 = (blockIdx.z % kUpGroups) * kUpTok; i0 < cnt; i0 += kUpGroups * kUpTok) {
        const int nt = min(kUpTok, cnt - i0);
        int r0 = 0;
        do {
            for (int e = threadIdx.x; e < nt * kUpRank; e += kUpThreads) {
                const int t = e / kUpRank, r = r0 + e % kUpRank;
                float v = 0.0f;
                if (r < R) {
                    const float* src = p.S + (win * kWindow + list[i0 + t]) * p.R + r;
                    for (int q = 0; q < p.slices; ++q) v += src[q * p.M * p.R];
                }
                s[t][e % kUpRank] = scale * v;
            }
            float w[C][kUpRank];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t n = n0 + c * kUpThreads;
                const float* b = p.B + ((int64_t)a * p.N + n) * p.R + r0;
#pragma unroll
                for (int r = 0; r < kUpRank; ++r) w[c][r] = n < p.N && r0 + r < R ? b[r] : 0.0f;
            }
            __syncthreads();
#pragma unroll 2
            for (int t = 0; t < nt; ++t) {
                float* y = p.Y + (win * kWindow + list[i0 + t]) * p.ldy + n0;
                float v[C];
#pragma unroll
                for (int c = 0; c < C; ++c)
                    v[c] = r0 == 0 ? bias[c] : n0 + c * kUpThreads < p.N ? y[c * kUpThreads] : 0.0f;
#pragma unroll
                for (int r = 0; r < kUpRank; r += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(&s[t][r]);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        v[c] = fmaf(w[c][r], x.x, v[c]);
                        v[c] = fmaf(w[c][r + 1], x.y, v[c]);
                        v[c] = fmaf(w[c][r + 2], x.z, v[c]);
                        v[c] = fmaf(w[c][r + 3], x.w, v[c]);
                    }
                }
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (n0 + c * kUpThreads < p.N) y[c * kUpThreads] = v[c];
            }
            __syncthreads();
            r0 += kUpRank;
        } while (r0 < R);
    }
}

// Up to this many tokens take the dots: a tile's 64 tokens would mostly be
// empty, and what counts is reading each adapter's rows from many SMs at once.
constexpr int64_t kDotTokens = 256;

template <int V>
cudaError_t launch_down(const LoraParams& p, unsigned windows, cudaStream_t stream) {
    if (p.M <= kDotTokens) {
        lora_down_dots<V><<<dim3(p.adapters, windows, p.slices), kDotWarps * 32, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const dim3 grid(p.adapters, windows, p.slices * kTileGroups);
    // rows of A per stage: as the rank needs, at most 64
    auto go = [&](auto kern, int smem) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<grid, kTileWarps * 32, smem, stream>>>(p);
        return cudaGetLastError();
    };
    if (p.R <= 16) return go(lora_down_tiles<V, 1>, tile_smem(1));
    if (p.R <= 32) return go(lora_down_tiles<V, 2>, tile_smem(2));
    return go(lora_down_tiles<V, 4>, tile_smem(4));
}

// Slices of K: enough blocks for every SM to have two, slices of at least 256
// values, at most 16 (the up step reads each).
int64_t slices_of(int64_t M, int64_t K, int64_t adapters, int sms) {
    const int64_t tiles = M <= kDotTokens ? (M < adapters ? M : adapters) : (M + kTileTok - 1) / kTileTok;
    int64_t n = (2 * sms + tiles - 1) / tiles;
    n = n > 16 ? 16 : n;
    const int64_t most = (K + 255) / 256;
    return n < most ? n : most;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" emu_status_t emu_lora(int64_t M, int64_t N, int64_t K, const float* X, int64_t ldx,
                                 const float* W, int64_t ldw, const void* Wp, int64_t ldwp,
                                 const float* bias, int64_t R, int64_t adapters, const float* A,
                                 const float* B, const float* scale, const int32_t* index, float* Y,
                                 int64_t ldy, emu_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (M < 0 || N < 0 || K < 0 || R < 0 || adapters < 0) return EMU_ERR_INVALID_VALUE;
    if (M > 32768 * (int64_t)kWindow || N > 65535 / kUpGroups * (int64_t)kUpThreads || K > INT32_MAX - 64 ||
        R > 65536 || adapters > (1 << 20))
        return EMU_ERR_INVALID_VALUE;
    if (ldx < 1 || ldx < K || ldy < 1 || ldy < N || (W && (ldw < 1 || ldw < K)))
        return EMU_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return EMU_OK;
    if (!Y) return EMU_ERR_INVALID_VALUE;
    if (K > 0 && (!X || !Wp || !aligned16(Wp) || ldwp < K || ldwp % 8 != 0 || ldwp > INT32_MAX))
        return EMU_ERR_INVALID_VALUE;
    const bool adapted = R > 0 && adapters > 0 && K > 0;
    if (adapted && (!A || !B || !index)) return EMU_ERR_INVALID_VALUE;
    if (((double)M + N) * (K + 8.0) > 5e17 || (double)M * R > 5e17) return EMU_ERR_ALLOC;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    emu_status_t st = current_device(&d);
    if (st != EMU_OK) return st;
    const int64_t ldp = plane_ld(K);
    const int64_t slices = adapted ? slices_of(M, K, adapters, d->sms) : 0;
    const size_t xp_bytes = ((size_t)6 * M * ldp + 1023) / 1024 * 1024;
    st = ensure_buffer(&d->ws, &d->ws_bytes, xp_bytes + (adapted ? (size_t)slices * M * R * 4 : 0));
    if (st != EMU_OK) return st;
    LoraParams p = {};
    p.M = M; p.N = N; p.K = K;
    p.R = adapted ? (int)R : 0;
    p.adapters = adapted ? (int)adapters : 0;
    p.X = X; p.ldx = ldx; p.A = A; p.B = B; p.scale = scale; p.bias = bias;
    p.index = adapted ? index : nullptr;
    p.S = reinterpret_cast<float*>(static_cast<uint8_t*>(d->ws) + xp_bytes);
    p.Y = Y; p.ldy = ldy; p.err = d->err;
    const unsigned windows = (unsigned)((M + kWindow - 1) / kWindow);
    cudaError_t e = cudaSuccess;
    if (adapted) {
        p.slices = (int)slices;
        p.slice = ((K + slices - 1) / slices + 63) / 64 * 64;
        e = K % 4 == 0 && ldx % 4 == 0 && aligned16(X) && aligned16(A) ? launch_down<4>(p, windows, stream)
                                                                      : launch_down<1>(p, windows, stream);
        if (e != cudaSuccess) return from_cuda(e);
    }
    // columns per thread: four where there are tokens to share them
    const int cols = M <= kDotTokens ? 1 : 4;
    const dim3 up((unsigned)p.adapters + 1, windows,
                  (unsigned)((N + cols * kUpThreads - 1) / (cols * kUpThreads)) * kUpGroups);
    if (cols == 1) lora_up<1><<<up, kUpThreads, 0, stream>>>(p);
    else lora_up<4><<<up, kUpThreads, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || K == 0) return from_cuda(e);
    e = launch_split_pieces(kModeBf16x9, X, M, K, ldx, 0, d->ws, ldp, stream);
    if (e != cudaSuccess) return from_cuda(e);
    if (few_rows_ok(M, W, ldw)) {
        TcGemmParams q = {};
        q.alpha = q.beta = 1.0f;
        q.C = Y; q.ldc = ldy;
        return gemm_few_rows(W, ldw, nullptr, 0, M, N, K, d->ws, ldp, q, d, stream);
    }
    return gemm_on_pieces(kModeBf16x9, PieceSet{d->ws, ldp, 0, 0}, PieceSet{Wp, ldwp, 0, 0}, M, N, K,
                          1.0f, 1.0f, Y, ldy, d, stream);
}
