// emu_host.h -- host-side state and helpers of libemusgemm that its entry
// points share: the per-device state, the workspace, tensor maps and the GEMM
// on pieces that are already in device memory.  Defined in emu_sgemm.cu.
// Everything here is used with g_mu held.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <mutex>

#include "emu_internal.h"
#include "emu_sgemm.h"

namespace emu {

constexpr int kMaxDevices = 64;
constexpr int kHostChunksMax = 8;        // row chunks of emu_sgemm_host's copy/compute pipeline

struct DeviceState {
    int checked = 0;           // 0 unknown, 1 supported, -1 unsupported
    int sms = 0;
    int* err = nullptr;        // device address of g_emu_error
    void* ws = nullptr;        // workspace for the split pieces
    size_t ws_bytes = 0;
    void* stage = nullptr;     // device staging for emu_sgemm_host
    size_t stage_bytes = 0;
    // emu_sgemm_host's pipeline: host->device and device->host copy streams
    // and per-chunk events (created on first use, kept until exit)
    cudaStream_t s_in = nullptr, s_out = nullptr;
    cudaEvent_t ev_in[kHostChunksMax] = {}, ev_done[kHostChunksMax] = {};
    cudaEvent_t ev_panel = nullptr;      // each column panel of op(B) landed
    // the GEMM's stream-K tail: one slot of partial sums per cluster (grown on
    // demand), flags (zeroed once) and the epoch that marks this call's flags
    void* part = nullptr;
    size_t part_bytes = 0;
    unsigned* flags = nullptr;
    unsigned epoch = 0;
};

extern std::mutex g_mu;

emu_status_t from_cuda(cudaError_t e);
// Current device state, checking the architecture once.
emu_status_t current_device(DeviceState** out, int* dev_out = nullptr);
emu_status_t ensure_buffer(void** buf, size_t* have, size_t need);

// Tensor map over `planes` row-major planes of rows x cols elements (row
// stride ld elements, plane stride plane_rows*ld, plane_rows 0 meaning
// rows), box of box_cols x box_rows, 128-byte swizzle, zero fill outside the
// matrix.
emu_status_t make_plane_map(CUtensorMap* map, const void* base, bool fp32, int64_t rows,
                            int64_t cols, int64_t ld, int planes, int box_cols, int box_rows,
                            int64_t plane_rows = 0);

// 2-D map over C for the bulk tensor stores of the GEMM epilogue (any beta;
// with beta != 0 the epilogue reads C itself first): box of 16 columns x 32
// rows, 64-byte swizzle.  The map covers the first N & ~3 columns only: a
// bulk store clips a box at the edge of the map in whole 16-byte units
// (measured on GB300: with N = 4k + 1..3 it wrote zeros up to column 4k + 3,
// past C), so the epilogue stores the last N % 4 columns of each row itself.
// Returns false (and the kernel stores C directly) when C's rows are not
// 16-byte aligned or C is narrower than 4 columns.
bool make_c_map(CUtensorMap* map, float* C, int64_t M, int64_t N, int64_t ldc);

// Plan the tail of the persistent GEMM (schedule.h) for the `clusters` of
// this GEMM variant that can be resident at once, and give it its
// workspace: one slot of bm x bn FP32 sums and 2 x 16 flags per cluster
// sharing the tail.  fix2: the planner's cost of a hand-over in half K
// blocks.  Sets p.tail_*, p.part_ws, p.flags and p.epoch.
emu_status_t plan_tail(TcGemmParams& p, int clusters, int fix2, int bm, int bn, DeviceState* d);

// Where one operand's pieces are: planes starting at p, ld elements per
// row, plane_rows rows apart (0: the planes' own row count).  mn = 0:
// K-major, a row per row of op(A) (or of op(B)^T), K elements long.  mn = 1
// (two-pass BF16 modes): M- or N-major, a row per K index, M (or N) elements
// long, ld a multiple of 64 (mn_ld) -- what a row-wise split writes from A
// stored K x M or B stored K x N.
struct PieceSet {
    const void* p;
    int64_t ld;
    int64_t plane_rows;
    int mn;
};

// Row length of M- or N-major pieces: whole 64-element chunks (the tensor
// copies read them a chunk at a time).
inline int64_t mn_ld(int64_t cols) { return (cols + 63) / 64 * 64; }

// Bytes of one operand's pieces: `rows` rows of op(A) (or of op(B)^T) over K.
inline size_t piece_bytes(int mode, bool mn, int64_t rows, int64_t K) {
    const size_t per = (size_t)mode_pieces(mode) * mode_piece_bytes(mode);
    return mn ? per * (size_t)K * mn_ld(rows) : per * (size_t)rows * plane_ld(K);
}

// The tensor-core GEMM on pieces already in device memory (op(A)'s and
// op(B)^T's, as PieceSet says).  Launched as a programmatic dependent of the
// split ahead of it in the stream.
emu_status_t gemm_on_pieces(int mode, const PieceSet& a, const PieceSet& b, int64_t M, int64_t N,
                            int64_t K, float alpha, float beta, float* C, int64_t ldc,
                            DeviceState* d, cudaStream_t stream);

// Few rows of X against FP32 weights (gemm_few.cu): whether the weights can be streamed (16-byte
// aligned rows, at most kFewRows rows of X), and the GEMM on X's pieces at
// `xp` (M rows of ldp).  W2 NULL: Y = alpha X W^T + beta Y, W N x K; else the
// gated form over N columns.  p carries the outputs (C, ldc, alpha, beta, act,
// G, U, ldg).  Launched as a programmatic dependent of the split of X, which
// must itself have been launched as an ordinary kernel: the weights are read
// before that split has ended.
constexpr int64_t kFewRows = 160;
bool few_rows_ok(int64_t M, const float* W, int64_t ldw);
// plane_rows: rows from one plane of X's pieces to the next (0: M).
emu_status_t gemm_few_rows(const float* W, int64_t ldw, const float* W2, int64_t ldw2, int64_t M,
                           int64_t N, int64_t K, const void* xp, int64_t ldp, int64_t plane_rows,
                           TcGemmParams p, DeviceState* d, cudaStream_t stream);

// The last M % 256 rows of M > 256, where streaming the FP32 weights (N rows in
// all, of K) for them costs less than one more row of 256-row tiles, mostly
// empty (0: run all rows in tiles).  Per 128 x 64 block of the weights a row of
// tiles takes 15.8 ns (a pair's 36 MMAs for two of them, shared by 76 pairs), the
// stream 4.8 ns up to 32 rows, 5.8 up to 64, 8.8 up to 128 and 10.5 up to 160
// (gemm_few's rate on 152 CTAs).  Start, end and uneven rounds take 10 to 20 us
// of that gain.  Measured, us, in tiles alone and with the last rows streamed:
// gated 777 x 2048 x (2 x 5504) 208 / 200, 356 x 4096 x (2 x 8192) 293 / 251, 612 x
// 2048 x (2 x 5504) 162 / 173, 300 x 1024 x (2 x 1024) 32.5 / 47; adapters 1040 x
// 2048 x 6144 119.5 / 118, 3117 x 1216 x 1152 94.5 / 114.
inline int64_t ragged_rows(int64_t M, int64_t N, int64_t K) {
    const int64_t rows = M % 256;
    if (M <= 256 || rows == 0 || rows > kFewRows) return 0;
    const double stream_ns = rows <= 32 ? 4.8 : rows <= 64 ? 5.8 : rows <= 128 ? 8.8 : 10.5;
    const double gain_ns = rows <= 32 ? 10000.0 : rows <= 64 ? 15000.0 : 20000.0;
    const double blocks = double((N + 127) / 128) * double((K + 63) / 64);
    return blocks * (15.8 - stream_ns) > gain_ns ? rows : 0;
}

}  // namespace emu
