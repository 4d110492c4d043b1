// gated.cu -- the gated feed-forward H = act(X Wg^T) * (X Wu^T) and its
// gradients (include/emu_layers.h): host entry points and the backward's
// elementwise kernel.
//
// Forward: X is split into its BF16 pieces, and one GEMM over the packed
// pieces of both weights forms 128 columns of each projection per 256-wide
// tile, so that a thread of the epilogue holds matching columns of both and
// writes their gated product (gemm_kblock.cu, kEpiGated).  Few rows of X
// leave that GEMM bound by the weights' bytes with most of its 256-row tiles
// empty: there the FP32 weights themselves are streamed (4 bytes a value
// instead of the pieces' 6) and split on chip, with X's pieces as the narrow
// operand (gemm_few.cu).
//
// Backward: dG = dH U act'(G), dU = dH act(G), then dX = [dG dU] [Wg; Wu] and
// [dWg; dWu] = [dG dU]^T X.  Both products read [dG dU] split into BF16
// pieces row by row -- dX as K-major pieces of its left operand, the weight
// gradients as M-major ones -- so one kernel forms the two gradients and
// their pieces in one pass and no FP32 copy of them is ever written.  The
// weights' packed pieces, K-major in the forward product, are N-major in
// dX's; X's row-wise pieces are N-major in the weight gradients.
#include <cstring>

#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"
#include "gated.cuh"

namespace emu {

static_assert(kActSilu == int(EMU_ACT_SILU) && kActGelu == int(EMU_ACT_GELU) &&
                  kActGeluTanh == int(EMU_ACT_GELU_TANH) && kActRelu == int(EMU_ACT_RELU) &&
                  kActSigmoid == int(EMU_ACT_SIGMOID),
              "kernel activations follow emu_act_t");

namespace {

// Rows of one projection in the packed pieces: a multiple of 32, so that the
// up projection's part of every row of [dG dU] starts on a 64-byte boundary
// and the row, of twice as many elements, is whole 64-element chunks.
inline int64_t gated_rows(int64_t F) { return (F + 31) / 32 * 32; }

// [dG dU] of G, U and dH as three planes of BF16 pieces, M rows of 2 Fp
// elements (dG from column 0, dU from column Fp, zeros in the gaps F..Fp-1).
// A thread takes 8 columns of one row: six 16-byte loads, six 16-byte stores
// (24 bytes read or written per element pair: bound by HBM).
template <int ACT>
__global__ void __launch_bounds__(256) gated_grad_split(int64_t M, int64_t F, int64_t Fp,
                                                        const float* __restrict__ dH, int64_t lddh,
                                                        const float* __restrict__ G,
                                                        const float* __restrict__ U, int64_t ldg,
                                                        bool vec, uint16_t* __restrict__ P) {
    griddep_launch_dependents();
    const int64_t groups = Fp / 8, total = M * groups, ld = 2 * Fp, plane = M * ld;
    for (int64_t t = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; t < total;
         t += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = t / groups, f = (t - m * groups) * 8;
        float g[8], u[8], d[8];
        if (vec && f + 8 <= F) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                *reinterpret_cast<float4*>(g + 4 * h) = __ldcs(reinterpret_cast<const float4*>(G + m * ldg + f) + h);
                *reinterpret_cast<float4*>(u + 4 * h) = __ldcs(reinterpret_cast<const float4*>(U + m * ldg + f) + h);
                *reinterpret_cast<float4*>(d + 4 * h) = __ldcs(reinterpret_cast<const float4*>(dH + m * lddh + f) + h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = f + j < F;
                g[j] = in ? G[m * ldg + f + j] : 0.0f;
                u[j] = in ? U[m * ldg + f + j] : 0.0f;
                d[j] = in ? dH[m * lddh + f + j] : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 a = gated_act_grad<ACT>(g[j]);
            g[j] = d[j] * u[j] * a.y;                    // dG
            u[j] = d[j] * a.x;                           // dU
        }
        uint16_t* dst = P + m * ld + f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float* v = half ? u : g;
            uint4 o0, o1, o2;
            split_bf16x3_pair(v[0], v[1], o0.x, o1.x, o2.x);
            split_bf16x3_pair(v[2], v[3], o0.y, o1.y, o2.y);
            split_bf16x3_pair(v[4], v[5], o0.z, o1.z, o2.z);
            split_bf16x3_pair(v[6], v[7], o0.w, o1.w, o2.w);
            *reinterpret_cast<uint4*>(dst + half * Fp) = o0;
            *reinterpret_cast<uint4*>(dst + half * Fp + plane) = o1;
            *reinterpret_cast<uint4*>(dst + half * Fp + 2 * plane) = o2;
        }
    }
    griddep_wait();          // complete only after the kernel ahead (see split.cu)
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Shared limits of the entry points: sizes, and that the packed pieces are
// what TMA can read.
emu_status_t check_sizes(int act, int64_t M, int64_t F, int64_t K) {
    if (act < EMU_ACT_SILU || act > EMU_ACT_SIGMOID) return EMU_ERR_INVALID_VALUE;
    if (M < 0 || F < 0 || K < 0 || M > INT32_MAX || F > INT32_MAX / 4 || K > INT32_MAX - 64)
        return EMU_ERR_INVALID_VALUE;
    return EMU_OK;
}
bool pieces_ok(const void* Wp, int64_t ldwp, int64_t K) {
    return Wp && aligned16(Wp) && ldwp >= K && ldwp % 64 == 0 && ldwp <= INT32_MAX;
}
// Elements of the pieces that one call stages, below 2^59 (so that no size
// product wraps; no allocation that large can succeed).
bool small_enough(int64_t M, int64_t F, int64_t K) {
    const double e = (double)M * (2.0 * F + 64) + ((double)M + 2.0 * F + 64) * (K + 64.0);
    return e < 5e17;
}

emu_status_t gated_forward(int act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                           const float* Wg, int64_t ldwg, const float* Wu, int64_t ldwu,
                           const void* Wp, int64_t ldwp, float* H, int64_t ldh, float* G, float* U,
                           int64_t ldg, DeviceState* d, cudaStream_t stream) {
    const int64_t ldp = plane_ld(K), Fp = gated_rows(F);
    emu_status_t st = ensure_buffer(&d->ws, &d->ws_bytes, (size_t)6 * M * ldp);
    if (st != EMU_OK) return st;
    cudaError_t e = launch_split_pieces(kModeBf16x9, X, M, K, ldx, 0, d->ws, ldp, stream);
    if (e != cudaSuccess) return from_cuda(e);
    // rows that stream the FP32 weights: all of them, or what whole tiles leave
    const int64_t few = !few_rows_ok(1, Wg, ldwg) || !few_rows_ok(1, Wu, ldwu) ? 0
                        : M <= kFewRows                                        ? M
                                                                               : ragged_rows(M, 2 * F, K);
    const int64_t rows = M - few;
    TcGemmParams p = {};
    p.act = act;
    if (few > 0) {
        p.C = H + rows * ldh; p.ldc = ldh;
        if (G) {
            p.G = G + rows * ldg; p.U = U + rows * ldg; p.ldg = ldg;
        }
        st = gemm_few_rows(Wg, ldwg, Wu, ldwu, few, F, K, static_cast<uint16_t*>(d->ws) + rows * ldp, ldp,
                           M, p, d, stream);
        if (st != EMU_OK || rows == 0) return st;
    }
    p.C = H; p.ldc = ldh;
    p.G = G; p.U = U; p.ldg = ldg;
    CUtensorMap mapA, mapB;
    st = make_plane_map(&mapA, d->ws, false, rows, K, ldp, 3, 64, 128, M);
    if (st != EMU_OK) return st;
    st = make_plane_map(&mapB, Wp, false, 2 * Fp, K, ldwp, 3, 64, 128);
    if (st != EMU_OK) return st;
    p.err = d->err;
    p.M = (int)rows; p.N = (int)F; p.K = (int)K;
    p.num_kb = (int)((K + 63) / 64);
    p.tiles_m = (int)((rows + 255) / 256);
    p.tiles_n = (int)((F + 127) / 128);
    p.up_row = (int)Fp;
    CUtensorMap mapH = mapB, mapG = mapB, mapU = mapB;   // placeholders where stored directly
    p.tma_store = make_c_map(&mapH, H, rows, F, ldh) ? 1 : 0;
    if (G)
        p.tma_gu = make_c_map(&mapG, G, rows, F, ldg) && make_c_map(&mapU, U, rows, F, ldg) ? 1 : 0;
    st = plan_tail(p, gemm_gated_clusters(d->sms), handover_half_blocks(kModeBf16x9), 256, 256, d);
    if (st != EMU_OK) return st;
    return from_cuda(launch_gemm_gated(mapA, mapB, mapH, mapG, mapU, p, d->sms, stream));
}

}  // namespace
}  // namespace emu

using namespace emu;

extern "C" {

int64_t emu_gated_rows(int64_t F) { return F < 0 || F > INT32_MAX / 4 ? -1 : gated_rows(F); }

emu_status_t emu_gated_pack(int64_t F, int64_t K, const float* Wg, int64_t ldwg, const float* Wu,
                            int64_t ldwu, void* Wp, int64_t ldwp, emu_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    emu_status_t st = check_sizes(EMU_ACT_SILU, 0, F, K);
    if (st != EMU_OK) return st;
    if (ldwg < 1 || ldwg < K || ldwu < 1 || ldwu < K) return EMU_ERR_INVALID_VALUE;
    if (F == 0 || K == 0) return EMU_OK;
    if (!Wg || !Wu || !pieces_ok(Wp, ldwp, K) || !small_enough(0, F, K)) return EMU_ERR_INVALID_VALUE;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    st = current_device(&d);
    if (st != EMU_OK) return st;
    const int64_t Fp = gated_rows(F);
    uint16_t* P = static_cast<uint16_t*>(Wp);
    cudaError_t e = cudaSuccess;
    // the gaps' rows meet zeros of [dG dU] in dX's product: they hold zeros too
    // (six of them, behind every F rows of the planes' halves)
    if (Fp > F)
        e = cudaMemset2DAsync(P + F * ldwp, Fp * ldwp * 2, 0, (Fp - F) * ldwp * 2, 6, stream);
    if (e == cudaSuccess)
        e = launch_split_pieces(kModeBf16x9, Wg, F, K, ldwg, 0, P, ldwp, stream, false, 2 * Fp);
    if (e == cudaSuccess)                                // may run beside the gate's split
        e = launch_split_pieces(kModeBf16x9, Wu, F, K, ldwu, 0, P + Fp * ldwp, ldwp, stream, true,
                                2 * Fp);
    return from_cuda(e);
}

emu_status_t emu_gated(int act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                       const float* Wg, int64_t ldwg, const float* Wu, int64_t ldwu,
                       const void* Wp, int64_t ldwp, float* H, int64_t ldh, float* G, float* U,
                       int64_t ldg, emu_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    emu_status_t st = check_sizes(act, M, F, K);
    if (st != EMU_OK) return st;
    if (ldx < 1 || ldx < K || ldh < 1 || ldh < F || (!G != !U) || (G && (ldg < 1 || ldg < F)))
        return EMU_ERR_INVALID_VALUE;
    if ((!Wg != !Wu) || (Wg && (ldwg < 1 || ldwg < K || ldwu < 1 || ldwu < K)))
        return EMU_ERR_INVALID_VALUE;
    if (M == 0 || F == 0) return EMU_OK;
    if (!H || (K > 0 && (!X || !pieces_ok(Wp, ldwp, K)))) return EMU_ERR_INVALID_VALUE;
    if (!small_enough(M, F, K)) return EMU_ERR_ALLOC;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    st = current_device(&d);
    if (st != EMU_OK) return st;
    if (K == 0) {                                        // G = U = 0, and act(0) * 0 = 0
        cudaError_t e = launch_scale(M, F, 0.0f, H, ldh, stream);
        if (e == cudaSuccess && G) e = launch_scale(M, F, 0.0f, G, ldg, stream);
        if (e == cudaSuccess && U) e = launch_scale(M, F, 0.0f, U, ldg, stream);
        return from_cuda(e);
    }
    return gated_forward(act, M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, Wp, ldwp, H, ldh, G, U, ldg, d, stream);
}

emu_status_t emu_gated_bwd(int act, int64_t M, int64_t F, int64_t K, const float* dH, int64_t lddh,
                           const float* X, int64_t ldx, const void* Wp, int64_t ldwp,
                           const float* G, const float* U, int64_t ldg, float* dX, int64_t lddx,
                           float* dW, int64_t lddw, emu_stream_t stream_) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    emu_status_t st = check_sizes(act, M, F, K);
    if (st != EMU_OK) return st;
    if (lddh < 1 || lddh < F || ldx < 1 || ldx < K || ldg < 1 || ldg < F ||
        (dX && (lddx < 1 || lddx < K)) || (dW && (lddw < 1 || lddw < K)))
        return EMU_ERR_INVALID_VALUE;
    if (K == 0 || (!dX && !dW)) return EMU_OK;
    const bool some = M > 0 && F > 0;
    if (some && (!dH || !G || !U || (dW && !X) || (dX && !pieces_ok(Wp, ldwp, K))))
        return EMU_ERR_INVALID_VALUE;
    if (!small_enough(M, F, K)) return EMU_ERR_ALLOC;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    st = current_device(&d);
    if (st != EMU_OK) return st;
    const int64_t Fp = gated_rows(F);
    if (!some) {                                         // sums over nothing
        cudaError_t e = cudaSuccess;
        if (dX && M > 0) e = launch_scale(M, K, 0.0f, dX, lddx, stream);
        if (e == cudaSuccess && dW && F > 0) e = launch_scale(2 * Fp, K, 0.0f, dW, lddw, stream);
        return from_cuda(e);
    }
    // workspace: the pieces of [dG dU] (M rows of 2 Fp), then X's (M rows)
    const int64_t ldxp = mn_ld(K);
    const size_t gu_bytes = ((size_t)6 * M * 2 * Fp + 1023) / 1024 * 1024;
    st = ensure_buffer(&d->ws, &d->ws_bytes, gu_bytes + (dW ? (size_t)6 * M * ldxp : 0));
    if (st != EMU_OK) return st;
    uint16_t* gu = static_cast<uint16_t*>(d->ws);
    uint8_t* xp = static_cast<uint8_t*>(d->ws) + gu_bytes;
    const bool vec = aligned16(dH) && aligned16(G) && aligned16(U) && lddh % 4 == 0 && ldg % 4 == 0;
    const int64_t want = (M * (Fp / 8) + 255) / 256, most = (int64_t)d->sms * 16;
    with_act(act, [&](auto a) {
        gated_grad_split<decltype(a)::value><<<(unsigned)(want < most ? want : most), 256, 0, stream>>>(
            M, F, Fp, dH, lddh, G, U, ldg, vec, gu);
    });
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return from_cuda(e);
    if (dW) {                                            // independent: may run beside it
        e = launch_split_pieces(kModeBf16x9, X, M, K, ldx, 0, xp, ldxp, stream, true);
        if (e != cudaSuccess) return from_cuda(e);
    }
    if (dX) {
        st = gemm_on_pieces(kModeBf16x9, PieceSet{gu, 2 * Fp, 0, 0}, PieceSet{Wp, ldwp, 0, 1}, M, K,
                            2 * Fp, 1.0f, 0.0f, dX, lddx, d, stream);
        if (st != EMU_OK) return st;
    }
    if (dW)
        st = gemm_on_pieces(kModeBf16x9, PieceSet{gu, 2 * Fp, 0, 1}, PieceSet{xp, ldxp, 0, 1},
                            2 * Fp, K, M, 1.0f, 0.0f, dW, lddw, d, stream);
    return st;
}

}  // extern "C"
