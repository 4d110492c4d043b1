/*
 * emu_layers.h -- C ABI of libemusgemm: what a transformer block computes
 * beside its attention, on one GB300 GPU (sm_103a).
 *
 *   emu_gated, emu_gated_bwd         gated feed-forward, forward and backward
 *   emu_lora                         a projection with the low-rank adapters
 *                                    of many requests at once
 *   emu_qk_norm_rope, ..._bwd        norm of each query and key head with the
 *                                    position rotation, forward and backward
 *
 * The matrix products are emu_sgemm's BF16X9 (emu_sgemm.h): FP32 in and out,
 * at FP32 accuracy.  The conventions of emu_sgemm.h hold: row-major storage,
 * device pointers owned by the caller, work enqueued asynchronously on
 * `stream`, arguments checked on the host before anything is launched,
 * status codes, the library's workspace (calls on one device share it and
 * must be serialised; a call can be captured in a CUDA graph once a call of
 * the same shape has run outside capture).  Values on the device that have
 * to be in range (adapter indices, positions) are checked by the kernels: one
 * that is not records EMU_ERR_INVALID_VALUE in the device's sticky error word
 * (emu_get_last_device_error) and reads nothing out of bounds.  Infinities in
 * a product's operands usually give NaN, as in emu_sgemm; they and NaN stay in
 * the outputs that they enter.  The kernel
 * timing of emu_profile_enable counts the GEMMs that gated's backward and
 * lora run on emu_sgemm's kernel; the other kernels of this header are not
 * counted.
 */
#ifndef EMU_LAYERS_H
#define EMU_LAYERS_H

#include "emu_sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------- gated feed-forward --
 *
 * H = act(G) * U element by element, G = X Wg^T, U = X Wu^T; X is M x K, the
 * weights Wg (gate) and Wu (up) are F x K, H is M x F.  One kernel forms both
 * products and writes H.
 */
typedef enum {
    EMU_ACT_SILU = 0,       /* g / (1 + e^-g) */
    EMU_ACT_GELU = 1,       /* g (1 + erf(g / sqrt 2)) / 2 */
    EMU_ACT_GELU_TANH = 2,  /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
    EMU_ACT_RELU = 3,       /* max(g, 0) */
    EMU_ACT_SIGMOID = 4     /* 1 / (1 + e^-g) */
} emu_act_t;

/* Rows of one projection in the packed pieces: F rounded up to 32 (-1 for an
 * F out of range). */
int64_t emu_gated_rows(int64_t F);

/*
 * emu_gated_pack -- the weights' BF16 pieces in the layout that the other two
 * entry points read: three planes (emu_split_bf16x3's pieces 0, 1, 2) of
 * 2 * emu_gated_rows(F) rows x ldwp BF16 bit patterns, Wg's rows from row 0,
 * Wu's from row emu_gated_rows(F), zeros in the rows between.  Pack again
 * whenever the weights change.
 *
 *  Wp, ldwp   16-byte aligned; ldwp >= K, a multiple of 64.
 */
emu_status_t emu_gated_pack(int64_t F, int64_t K, const float* Wg, int64_t ldwg, const float* Wu,
                            int64_t ldwu, void* Wp, int64_t ldwp, emu_stream_t stream);

/*
 * emu_gated -- H = act(X Wg^T) * (X Wu^T).
 *
 *  act           an emu_act_t
 *  M, F, K       each >= 0.  M == 0 or F == 0 is a no-op; K == 0 gives zeros.
 *  Wp, ldwp      the packed pieces of Wg and Wu (emu_gated_pack)
 *  Wg, Wu        the weights themselves, or both NULL.  Where they are given
 *                with 16-byte aligned rows and there are few rows of X, the
 *                kernel streams them instead of the pieces (fewer bytes); Wp
 *                must hold the pieces of the same values.
 *  G, U, ldg     where the two products are stored as well, M x F each, for
 *                emu_gated_bwd; or both NULL.
 *
 * Every element of G and U meets emu_sgemm's BF16X9 bound; act and the
 * product are computed in FP32 from them.  No output may overlap an input.
 */
emu_status_t emu_gated(int act, int64_t M, int64_t F, int64_t K, const float* X, int64_t ldx,
                       const float* Wg, int64_t ldwg, const float* Wu, int64_t ldwu,
                       const void* Wp, int64_t ldwp, float* H, int64_t ldh, float* G, float* U,
                       int64_t ldg, emu_stream_t stream);

/*
 * emu_gated_bwd -- the gradients of a loss whose gradient in H is dH:
 *     dG = dH * U * act'(G),  dU = dH * act(G)    (element by element)
 *     dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X.
 *
 *  G, U, ldg     as emu_gated stored them
 *  dX, lddx      M x K, or NULL
 *  dW, lddw      2 * emu_gated_rows(F) rows x K, or NULL: dWg in the first F
 *                rows, dWu in F rows from row emu_gated_rows(F); the rows
 *                between are written too (zeros).
 *  act'(0) of EMU_ACT_RELU is 0.
 */
emu_status_t emu_gated_bwd(int act, int64_t M, int64_t F, int64_t K, const float* dH, int64_t lddh,
                           const float* X, int64_t ldx, const void* Wp, int64_t ldwp,
                           const float* G, const float* U, int64_t ldg, float* dX, int64_t lddx,
                           float* dW, int64_t lddw, emu_stream_t stream);

/* -------------------------------------------------- low-rank adapters --
 *
 * emu_lora -- Y[t] = X[t] W^T + bias + scale_i (X[t] A_i^T) B_i^T, i = index[t]:
 * one projection that all rows share, and for each row (token) the low-rank
 * adapter that its request asked for.
 *
 *  M, N, K       X is M x K, W is N x K, Y is M x N.  M == 0 or N == 0 is a
 *                no-op; K == 0 gives the bias.
 *  Wp, ldwp      W's pieces as emu_sgemm_bsplit's BF16X9 takes them: 3 planes
 *                of N rows x ldwp, ldwp >= K and a multiple of 8.
 *  W, ldw        W itself or NULL, as in emu_gated.
 *  bias          N values or NULL.
 *  R, adapters   rank and number of adapters, at most 8191 (an adapter of a lower rank has
 *                zeros in its last rows of A, columns of B); R == 0 or
 *                adapters == 0 runs the projection alone.
 *  A, B          adapters x R x K and adapters x N x R, contiguous.
 *  scale         `adapters` values, or NULL for ones.
 *  index         M values: the token's adapter, or -1 for none.  The tokens may
 *                be in any order.  Another value counts as none and records
 *                EMU_ERR_INVALID_VALUE in the device's error word.
 *
 * The projection meets emu_sgemm's BF16X9 bound with the adapter's term as
 * the C that it adds to; that term is computed in FP32.  Y may not overlap an
 * input.
 */
emu_status_t emu_lora(int64_t M, int64_t N, int64_t K, const float* X, int64_t ldx, const float* W,
                      int64_t ldw, const void* Wp, int64_t ldwp, const float* bias, int64_t R,
                      int64_t adapters, const float* A, const float* B, const float* scale,
                      const int32_t* index, float* Y, int64_t ldy, emu_stream_t stream);

/* ------------------------------ norm and rotation of queries and keys --
 *
 * For every token t and head h of the queries and of the keys, x the head's D
 * values, w its side's weight:
 *     n = w * x / sqrt(mean(x^2) + eps)
 *     y = n with the pairs (a, b) of its first `rot` values turned to
 *         (a c - b s, a s + b c),  c = cos[p, j], s = sin[p, j], p = positions[t]
 * where pair j is (n[j], n[j + rot/2]), or (n[2j], n[2j+1]) when interleaved.
 * Sums and products are in FP32; the result is rounded once to the type.
 */
typedef enum { EMU_F32 = 0, EMU_BF16 = 1, EMU_F16 = 2 } emu_dtype_t;

/* Heads of one tensor: element (t, h, d) at data[t * token_stride +
 * h * head_stride + d] (strides in elements).  A slice of a projection's
 * output can be given as it is. */
typedef struct {
    void* data;
    int64_t heads, token_stride, head_stride;
} emu_heads_t;

/*
 * emu_qk_norm_rope
 *
 *  heads         four of them: q, k, and the outputs q', k'.  Either side may
 *                have 0 heads.  An output may be its input (same data and
 *                strides), otherwise it may not overlap one.
 *  dtype         type of q, k and the outputs (an emu_dtype_t)
 *  T, D, rot     tokens (at most 2^25 - 1), values of a head (1..512), rotated values (even,
 *                0..D).  T == 0 is a no-op.
 *  wq, wk        D values each (FP32), or NULL for ones
 *  cos, sin      table_rows x rot/2 (FP32, contiguous); rot == 0 reads neither
 *  positions     T values in [0, table_rows); another value gives NaN in that
 *                token's rotated values (in the backward pass, in all its
 *                gradients) and records EMU_ERR_INVALID_VALUE in the device's
 *                error word
 */
emu_status_t emu_qk_norm_rope(int dtype, int64_t T, int64_t D, int64_t rot, int interleaved,
                              float eps, const emu_heads_t* heads, const float* wq,
                              const float* wk, const float* cos, const float* sin,
                              int64_t table_rows, const int32_t* positions, emu_stream_t stream);

/*
 * emu_qk_norm_rope_bwd -- heads: six, q and k as the forward had them, the
 * gradients dq, dk to write, and the gradients dq', dk' of the outputs.  dwq,
 * dwk: D FP32 values each, or NULL, summed over tokens and heads in a fixed
 * order: the same inputs give the same bits.
 */
emu_status_t emu_qk_norm_rope_bwd(int dtype, int64_t T, int64_t D, int64_t rot, int interleaved,
                                  float eps, const emu_heads_t* heads, const float* wq,
                                  const float* wk, const float* cos, const float* sin,
                                  int64_t table_rows, const int32_t* positions, float* dwq,
                                  float* dwk, emu_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EMU_LAYERS_H */
