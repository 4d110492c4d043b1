// lora.cu -- a projection with the low-rank adapters of many requests at once
// (include/emu_layers.h):  Y = X W^T + bias + scale_i (X A_i^T) B_i^T.
//
// Three steps: S[t] = A_i X[t] for every token with an adapter (down), Y[t] =
// bias + scale_i B_i S[t] (up), and the shared projection added to it by the
// emulated GEMM (beta = 1).  K is cut into slices so that few tokens, too, fill
// the GPU; the up step adds the slices in order.
//
// Up to kFewTokens tokens a block takes four neighbouring tokens and one after
// another the adapters among them: an adapter's rows come from L2 again for
// every four tokens, and no grouping has to run first.  Beyond that one block
// groups the tokens by adapter (lora_group) into tiles of up to 64, and the
// steps' blocks take a tile each.  Every element of the adapter's term is one
// fixed sum, so neither the order of the tokens in the batch nor that of a tile
// changes it.  The projection's last rounding may depend on a token's place: whole
// tiles, tiles that share K and the last rows of a ragged batch (ragged_rows) add
// their partial sums in different orders.
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
    // the grouping (many tokens): the tokens by adapter, and its tiles
    int32_t* order;
    int4* tiles;             // adapter (== adapters: none), first place in order, tokens
    int32_t* ntiles;
};

constexpr int64_t kFewTokens = 256;          // up to here: no grouping
constexpr int kTileTok = 64;                 // tokens of a tile
constexpr int kMaxAdapters = 8191;           // lora_group counts them in shared memory

// The adapter of token t, `adapters` for none.
__device__ __forceinline__ int adapter_of(const LoraParams& p, int64_t t) {
    const int32_t v = p.index ? p.index[t] : -1;
    if (v >= 0 && v < p.adapters) return v;
    if (v != -1) record_error(p.err, kDevErrValue);
    return p.adapters;
}

// Sum of v over the block's threads before this one (1024 threads).
__device__ __forceinline__ int block_before(int v, int* warp_sum, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int before = upto - v, all = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    __syncthreads();
    *total = all;
    return before;
}

// Groups the tokens by adapter and cuts the groups into tiles.  One block; the
// tokens are counted and placed with shared-memory atomics (their order inside
// a group is not fixed and does not matter).
__global__ void __launch_bounds__(1024) lora_group(const LoraParams p) {
    __shared__ int count[kMaxAdapters + 1];  // tokens, then the next free place
    __shared__ int warp_sum[32];
    const int groups = p.adapters + 1, tid = threadIdx.x;
    griddep_launch_dependents();
    for (int a = tid; a < groups; a += 1024) count[a] = 0;
    __syncthreads();
    for (int64_t t = tid; t < p.M; t += 1024) atomicAdd(&count[adapter_of(p, t)], 1);
    __syncthreads();
    const int per = (groups + 1023) / 1024;
    int tokens = 0, tiles = 0;
    for (int a = tid * per; a < min(groups, (tid + 1) * per); ++a) {
        tokens += count[a];
        tiles += (count[a] + kTileTok - 1) / kTileTok;
    }
    int all, all_tiles;
    int at = block_before(tokens, warp_sum, &all);
    int tile = block_before(tiles, warp_sum, &all_tiles);
    for (int a = tid * per; a < min(groups, (tid + 1) * per); ++a) {
        const int n = count[a];
        for (int i = 0; i < n; i += kTileTok) p.tiles[tile++] = make_int4(a, at + i, min(kTileTok, n - i), 0);
        count[a] = at;
        at += n;
    }
    if (tid == 0) *p.ntiles = all_tiles;
    __syncthreads();
    for (int64_t t = tid; t < p.M; t += 1024) p.order[atomicAdd(&count[adapter_of(p, t)], 1)] = (int32_t)t;
    griddep_wait();                          // complete only after the split ahead, which may run beside it
}

// ------------------------------------------------------------- down, dots --
//
// Few tokens: S[t][r] over one slice of K.  A block takes TOK neighbouring
// tokens, a warp two rows of A (the block 16 of them), its lanes stride over
// the slice (V neighbouring values each).  Bound by the latency of reading A's
// rows once.
constexpr int kDotWarps = 8, kDotRows = 2;
constexpr int kDotTok = 4;                   // tokens per block, 1 up to kSingleTokens of them
constexpr int64_t kSingleTokens = 64;

template <int V, int TOK>
__global__ void __launch_bounds__(kDotWarps * 32) lora_down_dots(const LoraParams p) {
    griddep_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * TOK;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slice = blockIdx.z;
    const int64_t k0 = slice * p.slice, k1 = min(p.K, k0 + p.slice);
    float* S = p.S + slice * p.M * p.R;
    const int r = (blockIdx.y * kDotWarps + warp) * kDotRows;
    if (r >= p.R) return;
    int own[TOK];
    const float* row[TOK];
#pragma unroll
    for (int j = 0; j < TOK; ++j) {      // past the end: the first token again, not stored
        const int64_t t = t0 + j < p.M ? t0 + j : t0;
        own[j] = t0 + j < p.M ? adapter_of(p, t) : p.adapters;
        row[j] = p.X + t * p.ldx;
    }
    for (unsigned left = (1u << TOK) - 1; left != 0;) {
        // the first token left, and those with the same adapter
        int a = p.adapters;
#pragma unroll
        for (int j = TOK - 1; j >= 0; --j)
            if (left >> j & 1) a = own[j];
        unsigned now = 0;
#pragma unroll
        for (int j = 0; j < TOK; ++j)
            if (own[j] == a) now |= 1u << j;
        left &= ~now;
        if (a == p.adapters) continue;
        const float* ar = p.A + ((int64_t)a * p.R + r) * p.K;
        const float* ar1 = r + 1 < p.R ? ar + p.K : ar;
        float acc[kDotRows][TOK] = {};
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
            for (int j = 0; j < TOK; ++j) {
                if (!(now >> j & 1)) continue;       // the block's own, uniform
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
            for (int j = 0; j < TOK; ++j) {
                float v = acc[q][j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0 && (now >> j & 1) && r + q < p.R) S[(t0 + j) * p.R + r + q] = v;
            }
    }
}

// ------------------------------------------------------------ down, tiles --
//
// Many tokens: tiles of 64 tokens x 16 rows of A per warp, over one slice of
// K.  The block stages 64 values of K of its 64 tokens and of 16 G rows of A at
// a time in shared memory (kTileStages buffers, filled by cp.async); its 8 warps are G
// groups of 16 rows times 8 / G parts of each stage.  A lane owns 8 tokens x 4
// rows, each sum as a pair over even and odd k, which is how 16-byte loads
// along K leave the operands; rows are padded by four values, so the eight
// token groups of a load fall into different banks.  Bound by shared-memory
// loads: 12 of them per 64 packed FMAs.
constexpr int kTileK = 64, kTileRow = kTileK + 4, kTileWarps = 8;
constexpr int kTileStages = 4;

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(float* dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
constexpr int tile_smem(int G) { return kTileStages * (kTileTok + 16 * G) * kTileRow * 4; }

template <int V, int G>
__global__ void __launch_bounds__(kTileWarps * 32) lora_down_tiles(const LoraParams p) {
    extern __shared__ __align__(16) float stage[];   // [kTileStages][64 + 16 G][kTileRow]
    constexpr int kRows = kTileTok + 16 * G, kParts = kTileWarps / G;
    griddep_launch_dependents();
    griddep_wait();                                  // the grouping
    if ((int)blockIdx.x >= *p.ntiles) return;
    const int4 tile = p.tiles[blockIdx.x];
    const int a = tile.x, n = tile.z;
    if (a == p.adapters) return;
    const int32_t* list = p.order + tile.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = warp % G, part = warp / G;
    const int tg = lane & 7, rg = lane >> 3;         // tokens tg + 8 i, rows rg + 4 j
    const int slice = blockIdx.y;
    const int64_t k0 = slice * p.slice, k1 = min(p.K, k0 + p.slice);
    const int steps = int((k1 - k0 + kTileK - 1) / kTileK);
    float* S = p.S + slice * p.M * p.R;
    {
        for (int r0 = 0; r0 < p.R; r0 += 16 * G) {
            // a thread's copies of a stage: the same rows every time, kTileK
            // further along; their sources are worked out once
            constexpr int per = kTileK / V, kCopies = kRows * per / (kTileWarps * 32);
            static_assert(kRows * per % (kTileWarps * 32) == 0 && (kTileWarps * 32) % per == 0, "whole rows");
            const int col = tid % per * V;
            const float* src[kCopies];
            unsigned live = 0;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int row = tid / per + i * (kTileWarps * 32 / per);
                bool in;
                if (row < kTileTok) {
                    in = row < n;
                    src[i] = p.X + (int64_t)list[in ? row : 0] * p.ldx;
                } else {
                    const int r = r0 + row - kTileTok;
                    in = r < p.R;
                    src[i] = p.A + ((int64_t)a * p.R + (in ? r : 0)) * p.K;
                }
                if (in) live |= 1u << i;
            }
            auto fill = [&](int st) {
                if (st < steps) {                    // (an empty group keeps the count)
                    float* dst = stage + (st % kTileStages) * kRows * kTileRow + tid / per * kTileRow + col;
                    const int64_t k = k0 + (int64_t)st * kTileK + col;
                    const bool here = k < k1;
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const bool in = here && (live >> i & 1);
                        float* to = dst + i * (kTileWarps * 32 / per) * kTileRow;
                        if constexpr (V == 4) cp_async16(to, in ? src[i] + k : src[i], in);
                        else cp_async4(to, in ? src[i] + k : src[i], in);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            uint64_t acc[8][4] = {};
            for (int st = 0; st < kTileStages - 1; ++st) fill(st);
            for (int st = 0; st < steps; ++st) {
                asm volatile("cp.async.wait_group %0;" :: "n"(kTileStages - 2) : "memory");
                __syncthreads();                     // stage st is here, st - 1 is free again
                fill(st + kTileStages - 1);
                const float* xs = stage + (st % kTileStages) * kRows * kTileRow + tg * kTileRow;
                const float* as = stage + (st % kTileStages) * kRows * kTileRow + (kTileTok + 16 * group + rg) * kTileRow;
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
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
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
                if (t < n && r0 + r < p.R) S[(int64_t)list[t] * p.R + r0 + r] = v;
            }
            __syncthreads();
        }
    }
}

// --------------------------------------------------------------------- up --
//
// Y[t][n] = bias[n] + scale sum_r B[n][r] S[t][r]: a thread takes C columns,
// kUpThreads apart (a warp writes 128 neighbouring bytes), keeps RK values of
// each one's row of B in registers (as pairs of neighbouring ranks) and walks
// its tokens, whose S the block has put in shared
// memory (times the scale, the slices of K added in order); higher ranks take
// more passes, which add to Y.  Bound by the writes of Y, for few tokens by the
// latency of reading B.
constexpr int kUpThreads = 128;

// The block's rows of B (C kUpThreads columns of Y, RK ranks) pass through
// shared memory, `bs`: read straight into registers, a warp's 16-byte loads each
// touched 32 lines.  Rows are padded by four values: a thread reads its own.
template <int C, int RK>
constexpr int up_smem() { return C * kUpThreads * (RK + 4); }

// Tokens list[0..nt) (or t0, t0 + 1, .. where list is null) of adapter a;
// the block's columns are n0 - threadIdx.x + 0 .. C kUpThreads - 1.  place:
// room for the tokens' rows of Y.
template <int C, int RK, int V>
__device__ __forceinline__ void up_tokens(const LoraParams& p, int a, const int32_t* list, int64_t t0,
                                          int nt, int64_t n0, float (*s)[RK], float* bs, int32_t* place) {
    const int R = a == p.adapters ? 0 : p.R;
    const float scale = R > 0 && p.scale ? p.scale[a] : 1.0f;
    for (int t = threadIdx.x; t < nt; t += kUpThreads) place[t] = list ? list[t] : (int32_t)(t0 + t);
    int r0 = 0;
    do {
        if (R > 0) {
            const int64_t first = n0 - threadIdx.x;
            for (int e = threadIdx.x; e < C * kUpThreads * (RK / V); e += kUpThreads) {
                const int row = e / (RK / V), r = (e % (RK / V)) * V;
                const bool in = first + row < p.N && r0 + r < R;
                const float* src = p.B + ((int64_t)a * p.N + (in ? first + row : 0)) * p.R + (in ? r0 + r : 0);
                float* dst = bs + row * (RK + 4) + r;
                if constexpr (V == 4) cp_async16(dst, src, in);
                else {
                    cp_async4(dst, src, in);
                    cp_async4(dst + 1, in && r0 + r + 1 < R ? src + 1 : src, in && r0 + r + 1 < R);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        griddep_wait();                      // S (B and the indices are the caller's)
        for (int e = threadIdx.x * V; e < nt * RK; e += kUpThreads * V) {
            const int t = e / RK, r = r0 + e % RK;
            float v[V] = {};
            if (r < R) {
                const float* src = p.S + (list ? list[t] : t0 + t) * p.R + r;
#pragma unroll 4
                for (int q = 0; q < p.slices; ++q, src += p.M * p.R) {
                    if constexpr (V == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                    } else {
                        v[0] += src[0];
                        if (r + 1 < R) v[1] += src[1];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) s[t][e % RK + i] = scale * v[i];
        }
        float bias[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t n = n0 + c * kUpThreads;
            bias[c] = p.bias && n < p.N ? p.bias[n] : 0.0f;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // the columns' values of B, as pairs of neighbouring ranks
        uint64_t w[C][RK / 2] = {};
        if (R > 0)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int r = 0; r < RK; r += 4) {
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(
                        bs + (threadIdx.x + c * kUpThreads) * (RK + 4) + r);
                    w[c][r / 2] = x.x;
                    w[c][r / 2 + 1] = x.y;
                }
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
            float* y = p.Y + place[t] * p.ldy + n0;
            uint64_t v[C];
#pragma unroll
            for (int c = 0; c < C; ++c)
                v[c] = pack_f32x2(__float_as_uint(r0 == 0 ? bias[c]
                                                  : n0 + c * kUpThreads < p.N ? y[c * kUpThreads] : 0.0f), 0u);
#pragma unroll
            for (int r = 0; r < RK; r += 4) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&s[t][r]);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    v[c] = fma_f32x2(w[c][r / 2], x.x, v[c]);
                    v[c] = fma_f32x2(w[c][r / 2 + 1], x.y, v[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (n0 + c * kUpThreads < p.N)
                    y[c * kUpThreads] = __uint_as_float(uint32_t(v[c])) + __uint_as_float(uint32_t(v[c] >> 32));
        }
        __syncthreads();
        r0 += RK;
    } while (r0 < R);
}

// Few tokens: TOK neighbouring ones per block, runs of one adapter together.
template <int V, int TOK>
__global__ void __launch_bounds__(kUpThreads) lora_up_few(const LoraParams p) {
    __shared__ __align__(16) float s[TOK][32];
    __shared__ __align__(16) float bs[up_smem<1, 32>()];
    __shared__ int32_t place[TOK];
    griddep_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * TOK, end = min(p.M, t0 + TOK);
    const int64_t n0 = (int64_t)blockIdx.y * kUpThreads + threadIdx.x;
    for (int64_t t = t0; t < end;) {
        const int a = adapter_of(p, t);
        int nt = 1;
        while (t + nt < end && adapter_of(p, t + nt) == a) ++nt;
        up_tokens<1, 32, V>(p, a, nullptr, t, nt, n0, s, bs, place);
        t += nt;
    }
}

// Many tokens: `part` tokens of a tile per block (z picks them), RK ranks per
// pass: as the rank needs, 32 where it is more than 16.
template <int V, int RK>
__global__ void __launch_bounds__(kUpThreads) lora_up_tiles(const LoraParams p, int part) {
    __shared__ __align__(16) float s[kTileTok][RK];
    __shared__ __align__(16) float bs[up_smem<2, RK>()];
    __shared__ int32_t place[kTileTok];
    griddep_launch_dependents();
    griddep_wait();                          // the grouping and S
    if ((int)blockIdx.x >= *p.ntiles) return;
    const int4 tile = p.tiles[blockIdx.x];
    const int first = blockIdx.z * part;
    if (first >= tile.z) return;
    up_tokens<2, RK, V>(p, tile.x, p.order + tile.y + first, 0, min(part, tile.z - first),
                        (int64_t)blockIdx.y * (2 * kUpThreads) + threadIdx.x, s, bs, place);
}

// Tiles that the grouping makes at most.
int64_t max_tiles(int64_t M, int64_t adapters) {
    return M / kTileTok + (M < adapters + 1 ? M : adapters + 1);
}

// Launch as a programmatic dependent of the kernel ahead in the stream (pdl):
// this call's own, whose results the kernel waits for itself.
template <typename Kern, typename... More>
cudaError_t launch_after(Kern kern, dim3 grid, int threads, int smem, bool pdl, const LoraParams& p,
                         cudaStream_t stream, More... more) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p, more...);
}

template <int V>
cudaError_t launch_down(const LoraParams& p, cudaStream_t stream) {
    if (p.M <= kFewTokens) {
        const unsigned rows = (p.R + kDotWarps * kDotRows - 1) / (kDotWarps * kDotRows);
        if (p.M <= kSingleTokens)
            lora_down_dots<V, 1><<<dim3((unsigned)p.M, rows, p.slices), kDotWarps * 32, 0, stream>>>(p);
        else
            lora_down_dots<V, kDotTok><<<dim3((unsigned)((p.M + kDotTok - 1) / kDotTok), rows, p.slices),
                                         kDotWarps * 32, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)max_tiles(p.M, p.adapters), p.slices);
    // rows of A per stage: as the rank needs, at most 64
    auto go = [&](auto kern, int smem) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        return launch_after(kern, grid, kTileWarps * 32, smem, true, p, stream);
    };
    if (p.R <= 16) return go(lora_down_tiles<V, 1>, tile_smem(1));
    if (p.R <= 32) return go(lora_down_tiles<V, 2>, tile_smem(2));
    return go(lora_down_tiles<V, 4>, tile_smem(4));
}

// Slices of K, at least 256 values each, at most 16 (the up step reads each):
// for the dots enough for two blocks per SM (131 tokens, 40 adapters of rank 32,
// the whole call, us: one 83, two 78, four 84), for the tiles four, two of which
// run at a time, so that an uneven last round costs little.
int64_t slices_of(int64_t M, int64_t K, int64_t R, int sms) {
    const int64_t blocks = M <= kSingleTokens ? M * ((R + 15) / 16)
                           : M <= kFewTokens  ? (M + kDotTok - 1) / kDotTok * ((R + 15) / 16)
                                              : M / kTileTok;
    int64_t n = ((M <= kFewTokens ? 2 : 4) * sms + blocks - 1) / blocks;
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
    if (M > INT32_MAX || N > 65535 * (int64_t)kUpThreads || K > INT32_MAX - 64 || R > 65536 ||
        adapters > kMaxAdapters)
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
    const int64_t slices = adapted ? slices_of(M, K, R, d->sms) : 0;
    // workspace: X's pieces, S's slices, and the grouping
    const bool few = M <= kFewTokens;
    auto up16 = [](size_t b) { return (b + 1023) / 1024 * 1024; };
    const size_t xp_bytes = up16((size_t)6 * M * ldp);
    const size_t s_bytes = up16((size_t)slices * M * R * 4);
    const size_t o_bytes = few ? 0 : up16((size_t)M * 4);
    const size_t t_bytes = few ? 0 : (size_t)max_tiles(M, adapters) * sizeof(int4) + 16;
    st = ensure_buffer(&d->ws, &d->ws_bytes, xp_bytes + s_bytes + o_bytes + t_bytes);
    if (st != EMU_OK) return st;
    LoraParams p = {};
    p.M = M; p.N = N; p.K = K;
    p.R = adapted ? (int)R : 0;
    p.adapters = adapted ? (int)adapters : 0;
    p.X = X; p.ldx = ldx; p.A = A; p.B = B; p.scale = scale; p.bias = bias;
    p.index = adapted ? index : nullptr;
    uint8_t* ws = static_cast<uint8_t*>(d->ws) + xp_bytes;
    p.S = reinterpret_cast<float*>(ws);
    p.order = reinterpret_cast<int32_t*>(ws + s_bytes);
    p.ntiles = reinterpret_cast<int32_t*>(ws + s_bytes + o_bytes);
    p.tiles = reinterpret_cast<int4*>(ws + s_bytes + o_bytes + 16);
    p.Y = Y; p.ldy = ldy; p.err = d->err;
    // The order, each step launched as a programmatic dependent of the one
    // before: X's pieces and the grouping, side by side; the adapters' steps; the
    // GEMM.  For few tokens the dots come first, the pieces are made beside them.
    cudaError_t e = cudaSuccess;
    if (!few) {
        if (K > 0) e = launch_split_pieces(kModeBf16x9, X, M, K, ldx, 0, d->ws, ldp, stream);
        if (e == cudaSuccess) e = launch_after(lora_group, dim3(1), 1024, 0, K > 0, p, stream);
        if (e != cudaSuccess) return from_cuda(e);
    }
    if (adapted) {
        p.slices = (int)slices;
        p.slice = ((K + slices - 1) / slices + 63) / 64 * 64;
        e = K % 4 == 0 && ldx % 4 == 0 && aligned16(X) && aligned16(A) ? launch_down<4>(p, stream)
                                                                      : launch_down<1>(p, stream);
        if (e != cudaSuccess) return from_cuda(e);
    }
    const bool wide = R % 4 == 0 && aligned16(B);
    if (few && K > 0) {
        e = launch_split_pieces(kModeBf16x9, X, M, K, ldx, 0, d->ws, ldp, stream, adapted);
        if (e != cudaSuccess) return from_cuda(e);
    }
    const bool after = adapted || !few || K > 0;
    if (few) {
        auto go = [&](auto kern, int tok) {
            const dim3 grid((unsigned)((M + tok - 1) / tok), (unsigned)((N + kUpThreads - 1) / kUpThreads));
            return launch_after(kern, grid, kUpThreads, 0, after, p, stream);
        };
        e = M <= kSingleTokens ? (wide ? go(lora_up_few<4, 1>, 1) : go(lora_up_few<2, 1>, 1))
                               : (wide ? go(lora_up_few<4, kDotTok>, kDotTok) : go(lora_up_few<2, kDotTok>, kDotTok));
    } else {
        const unsigned tiles = (unsigned)max_tiles(M, p.adapters);
        const unsigned cols = (unsigned)((N + 2 * kUpThreads - 1) / (2 * kUpThreads));
        // a tile's tokens go to four blocks where the tiles are too few to fill
        // the GPU (341 tokens, 632 columns, rank 64: 27 blocks took 84 us)
        const int part = (int64_t)tiles * cols < 8 * d->sms ? kTileTok / 4 : kTileTok;
        const dim3 grid(tiles, cols, kTileTok / part);
        auto go = [&](auto kern) { return launch_after(kern, grid, kUpThreads, 0, after, p, stream, part); };
        e = p.R > 16 ? (wide ? go(lora_up_tiles<4, 32>) : go(lora_up_tiles<2, 32>))
                     : (wide ? go(lora_up_tiles<4, 16>) : go(lora_up_tiles<2, 16>));
    }
    if (e != cudaSuccess || K == 0) return from_cuda(e);
    // rows that stream the FP32 weight: all of them, or what whole tiles leave
    const int64_t stream_rows = !few_rows_ok(1, W, ldw) ? 0 : M <= kFewRows ? M : ragged_rows(M, N, K);
    const int64_t rows = M - stream_rows;
    if (stream_rows > 0) {
        TcGemmParams q = {};
        q.alpha = q.beta = 1.0f;
        q.C = Y + rows * ldy; q.ldc = ldy;
        st = gemm_few_rows(W, ldw, nullptr, 0, stream_rows, N, K,
                           static_cast<uint16_t*>(d->ws) + rows * ldp, ldp, M, q, d, stream);
        if (st != EMU_OK || rows == 0) return st;
    }
    return gemm_on_pieces(kModeBf16x9, PieceSet{d->ws, ldp, M, 0}, PieceSet{Wp, ldwp, 0, 0}, rows, N, K,
                          1.0f, 1.0f, Y, ldy, d, stream);
}
