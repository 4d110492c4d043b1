// lora.cu -- a projection with the low-rank adapters of many requests at once
// (include/emu_layers.h):  Y = X W^T + bias + scale_i (X A_i^T) B_i^T.
//
// Three steps: S[t] = scale_i A_i X[t] for every token with an adapter
// (lora_down), Y[t] = bias + B_i S[t] (lora_up), and the shared projection
// added to it by the emulated GEMM (beta = 1).  The adapters' steps group the
// tokens by adapter as they go: a block takes one adapter and one window of
// tokens, scans the window's indices, and works on the tokens of its own in
// order, so an adapter's rows are read once for all of them and no sorted copy
// of the tokens is made.  Every output element is one thread's sum in a fixed
// order: the grouping cannot change a result.
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
    float* S;                // M x R
    float* Y;
    int64_t ldy;
    int* err;
};

constexpr int kWindow = 512;                 // tokens scanned by a block
constexpr int kTok = 16;                     // tokens per step of lora_down
constexpr int kDownWarps = 8, kUpThreads = 128, kUpRank = 16;

// The tokens of window `win` whose adapter is `a` (a == adapters: those
// without one), in order, as offsets in the window; returns how many.  Called
// by all threads of a block of at most 16 warps.
__device__ __forceinline__ int tokens_of(const LoraParams& p, int a, int64_t win, uint16_t* list) {
    __shared__ int warp_n[16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t t0 = win * kWindow;
    int n = 0;
    for (int o = 0; o < kWindow && t0 + o < p.M; o += blockDim.x) {
        const int i = o + threadIdx.x;
        bool mine = false;
        if (i < kWindow && t0 + i < p.M) {
            const int32_t v = p.index ? p.index[t0 + i] : -1;
            const bool none = v < 0 || v >= p.adapters;
            mine = a == p.adapters ? none : v == a;
            if (a == p.adapters && none && v != -1) record_error(p.err, kDevErrValue);
        }
        const unsigned m = __ballot_sync(0xffffffffu, mine);
        if (lane == 0) warp_n[warp] = __popc(m);
        __syncthreads();
        int before = n;
        for (int w = 0; w < warp; ++w) before += warp_n[w];
        if (mine) list[before + __popc(m & ((1u << lane) - 1))] = (uint16_t)i;
        for (int w = 0; w < warps; ++w) n += warp_n[w];
        __syncthreads();
    }
    return n;
}

// S[t][r] = scale sum_k X[t][k] A[r][k]: a warp takes one row r of A and kTok
// tokens, its lanes stride over K (4 neighbouring values each when V = 4).
template <int V>
__global__ void __launch_bounds__(kDownWarps * 32) lora_down(const LoraParams p) {
    __shared__ uint16_t list[kWindow];
    const int a = blockIdx.x;
    const int64_t win = blockIdx.y;
    const int n = tokens_of(p, a, win, list);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float s = p.scale ? p.scale[a] : 1.0f;
    const float* Aa = p.A + (int64_t)a * p.R * p.K;
    for (int i0 = blockIdx.z * kTok; i0 < n; i0 += gridDim.z * kTok) {
        const int nt = min(kTok, n - i0);
        const float* row[kTok];
#pragma unroll
        for (int j = 0; j < kTok; ++j)       // past the end: the first token again, not stored
            row[j] = p.X + (win * kWindow + list[i0 + (j < nt ? j : 0)]) * p.ldx;
        for (int r = warp; r < p.R; r += kDownWarps) {
            const float* ar = Aa + (int64_t)r * p.K;
            float acc[kTok];
#pragma unroll
            for (int j = 0; j < kTok; ++j) acc[j] = 0.0f;
            for (int64_t k = lane * V; k < p.K; k += 32 * V) {
                float w[V];
                if constexpr (V == 4) *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(ar + k);
                else w[0] = ar[k];
#pragma unroll
                for (int j = 0; j < kTok; ++j) {
                    float x[V];
                    if constexpr (V == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(row[j] + k);
                    else x[0] = row[j][k];
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[j] = fmaf(w[v], x[v], acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                float v = acc[j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0 && j < nt) p.S[(win * kWindow + list[i0 + j]) * p.R + r] = s * v;
            }
        }
    }
}

// Y[t][n] = bias[n] + sum_r B[n][r] S[t][r]: a thread takes one column n,
// keeps kUpRank values of B's row in registers and walks the window's tokens
// of its adapter; higher ranks take several passes that add to Y.
__global__ void __launch_bounds__(kUpThreads) lora_up(const LoraParams p) {
    __shared__ uint16_t list[kWindow];
    const int a = blockIdx.x;
    const int64_t win = blockIdx.y;
    const int cnt = tokens_of(p, a, win, list);
    if (cnt == 0) return;
    const int64_t n = (int64_t)blockIdx.z * kUpThreads + threadIdx.x;
    if (n >= p.N) return;
    const float bias = p.bias ? p.bias[n] : 0.0f;
    const int R = a == p.adapters ? 0 : p.R;
    const float* b = p.B + ((int64_t)a * p.N + n) * p.R;
    int r0 = 0;
    do {
        float w[kUpRank];
#pragma unroll
        for (int r = 0; r < kUpRank; ++r) w[r] = r0 + r < R ? b[r0 + r] : 0.0f;
        for (int i = 0; i < cnt; ++i) {
            const int64_t t = win * kWindow + list[i];
            float* y = p.Y + t * p.ldy + n;
            float v = r0 == 0 ? bias : *y;
            const float* s = p.S + t * p.R + r0;
#pragma unroll
            for (int r = 0; r < kUpRank; ++r)
                if (r0 + r < R) v = fmaf(w[r], s[r], v);
            *y = v;
        }
        r0 += kUpRank;
    } while (r0 < R);
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
    if (M > 65535 * (int64_t)kWindow || N > 65535 * (int64_t)kUpThreads || K > INT32_MAX - 64 ||
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
    const size_t xp_bytes = ((size_t)6 * M * ldp + 1023) / 1024 * 1024;
    st = ensure_buffer(&d->ws, &d->ws_bytes, xp_bytes + (adapted ? (size_t)M * R * 4 : 0));
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
        const dim3 grid((unsigned)adapters, windows, kWindow / kTok / 2);
        if (K % 4 == 0 && ldx % 4 == 0 && aligned16(X) && aligned16(A))
            lora_down<4><<<grid, kDownWarps * 32, 0, stream>>>(p);
        else
            lora_down<1><<<grid, kDownWarps * 32, 0, stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return from_cuda(e);
    }
    lora_up<<<dim3((unsigned)p.adapters + 1, windows, (unsigned)((N + kUpThreads - 1) / kUpThreads)),
              kUpThreads, 0, stream>>>(p);
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
