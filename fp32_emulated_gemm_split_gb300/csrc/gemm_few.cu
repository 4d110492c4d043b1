// gemm_few.cu -- the emulated GEMM for few rows of X: Y = X W^T with at most
// 160 rows, where what counts is reading W once.  Used by the gated
// feed-forward and the projection with adapters (include/emu_layers.h).
//
// The method is BF16x9 (gemm_kblock.cu), with the operands' roles swapped: W
// is the tensor core's A operand, 128 rows of it per tile, read as FP32 (4
// bytes a value; its three pieces would be 6) and split on chip into tensor
// memory; X's pieces, which a split kernel has written, are the narrow B
// operand.  For each 64-element K block a TMA producer fetches 128 x 64 FP32
// values of W into a ring of staging buffers (two 128-byte-swizzled boxes),
// split warps turn them into pieces in tensor memory, and the MMAs' partial of
// that block is added to FP32 registers with round to nearest.
//
// Stacked form (BN <= 32): an MMA with its A operand in tensor memory takes
// 44 cycles however few columns it has up to 64 (measured; 48 at 96 columns,
// 64 at 128, then in proportion), so the nine products one by one would be
// bound by instructions.  The three pieces of X side by side are one operand of 3 BN columns: piece i of W
// times all of them is one MMA per K step, and column group j collects
//     a0 b_j + 2^-8 (a1 b_j + 2^-8 a2 b_j),
// largest i first with the scaling between; the accumulator warps add the
// groups times 2^-8j.  At BN = 64, 128 and 160 the nine products run band by
// band, over as many columns as there are rows (in 16s).
//
// Bound by HBM: every value of W is read once.  One CTA per SM, each on its
// own (no clusters: with CTA pairs the hand-offs between producer, split, MMA
// and accumulators crossed SMs and took longer than the work between them:
// 94 us against 39.5 us of HBM time at 24 x 4096 x (2 x 8192)).
//
// Work: tiles of 128 rows (gated: 64 rows of each weight), dealt to the CTAs
// with the tail's K blocks shared evenly (schedule.h); a CTA that holds a
// later part of a tile leaves its FP32 sums in global memory for the owner.
//
// Programmatic launch: W is read before the split of X, the kernel ahead, has
// ended; only X's pieces and the output wait for it.  (X's rows split in this
// kernel too, by a warp per pipeline, would save that launch, but beside the
// busy split warps such a warp took twice the time of the stream: 24 x 4096 x
// (2 x 8192) 146 us against 61 then.)
#include <mutex>

#include "emu_device.cuh"
#include "gated.cuh"
#include "schedule.h"

namespace emu {
namespace {

constexpr int kBox = 128 * 128;                       // 128 rows x 32 floats
constexpr int kABuf = 2 * kBox;                       // one K block of FP32 W
constexpr int kPieceCols = 32;                        // tensor-memory columns of a piece's K block
constexpr int kSmemMax = 232448;

template <int BN, bool GATED>
struct Cfg {
    static constexpr bool stacked = BN <= 32;
    static constexpr int d_cols = stacked ? 3 * BN : BN;
    // All split warps work on one K block after another, each of them on its
    // own (there is no barrier among them), into a ring of stages in tensor
    // memory.  Two threads issue the MMAs, of the even and of the odd blocks
    // (one would need about 2100 cycles for a block's waits, MMAs and commits
    // beside the busy split warps, the stream 1400); the rings that they wait on
    // have even counts, so each has stages of its own and meets every barrier's
    // phases in order.  At BN = 128 and 160 the nine products take 2300 or 2900
    // cycles of the tensor core anyway: one issuer, which waits for the next
    // block while this one's last MMAs are in the queue (131 rows x 4096 x 6144:
    // 60 us, 68 with the waits between the blocks, 62 with two issuers), and half
    // the split warps.  The issuers' code is run by whole warps: by one lane of
    // it, an MMA cost 70 to 80 cycles to issue, the operands' moves to uniform
    // registers among the split warps' work (24 x 4096 x (2 x 8192): 61 -> 56 us).
    static constexpr int issuers = BN >= 128 ? 1 : 2;
    static constexpr int split_warps = BN >= 128 ? 8 : 16;
    static constexpr bool early = issuers == 1;          // (needs two stages of each ring per issuer)
    // tensor memory: partials, then W's pieces (96 columns per K block)
    static constexpr int partials = 2;
    static constexpr int a_stages = BN == 16 || BN == 64 ? 4 : 2;
    static_assert(a_stages % issuers == 0 && partials % issuers == 0, "an issuer's own stages");
    static constexpr int a_base = partials * d_cols;
    static_assert(a_base + a_stages * 3 * kPieceCols <= 512, "tensor memory overflow");
    // shared memory: FP32 buffers (as many as fit: the stream's bytes in
    // flight), stages of X's pieces, the gated hand-over
    static constexpr int a_bufs = BN == 16 ? 6 : BN == 32 ? 5 : BN == 64 ? (GATED ? 3 : 4) : BN == 128 ? 3 : 2;
    static constexpr int b_tile = BN * kTcBKBytes;
    static constexpr int b_stages = BN <= 64 ? 4 : 2;
    static_assert(b_stages % issuers == 0, "an issuer's own stages");
    // (the gated hand-over in `passes` of BN / passes rows of X)
    static constexpr int acc_warps = BN == 16 ? 4 : BN == 160 ? 16 : 8;
    static constexpr int acc_cols = BN / (acc_warps / 4);
    static constexpr int passes = BN <= 64 ? 1 : acc_warps / 4;
    static constexpr int ex_bytes = GATED ? 128 * BN / passes * 4 : 0;
    static constexpr int smem = a_bufs * kABuf + b_stages * 3 * b_tile + ex_bytes + 2048;
    static_assert(smem <= kSmemMax, "shared memory overflow");
    // warps: 0 TMA of W and tensor-memory allocation, 1 TMA of X's pieces, 2
    // (and 3) MMA, then the accumulators, four per column group, and the split
    // warps
    static constexpr int acc0 = 4, split0 = acc0 + acc_warps;
    static constexpr int threads = 32 * (split0 + split_warps);
};

__device__ __forceinline__ unsigned load_acquire(const unsigned* a) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a) : "memory");
    return v;
}

// 16 elements (quarter kq of the K block's 64) of row r of the two swizzled 128
// x 32 FP32 boxes at `box`, the three pieces' 8 columns each at `col` (piece i
// at col + 32 i).  The 32 lanes read the same 16-byte chunk of 32 rows, which
// the swizzle spreads over the banks.  One test per 16 elements keeps
// infinities and NaNs off the packed path.
__device__ __forceinline__ void split_to_tmem(const uint8_t* box, uint32_t col, int r, int kq) {
    const uint8_t* row = box + (kq >> 1) * kBox + r * 128;
    float x[16];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(row + (((4 * (kq & 1) + c) ^ (r & 7)) << 4));
        x[4 * c] = v.x; x[4 * c + 1] = v.y; x[4 * c + 2] = v.z; x[4 * c + 3] = v.w;
    }
    float m = max_abs_nan(x[0], x[1]);
#pragma unroll
    for (int j = 2; j < 16; ++j) m = max_abs_nan(m, x[j]);
    uint32_t w0[8], w1[8], w2[8];
    if (m < __uint_as_float(0x7F800000u)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) split_finite_pair(x[2 * j], x[2 * j + 1], w0[j], w1[j], w2[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) split_bf16x3_pair(x[2 * j], x[2 * j + 1], w0[j], w1[j], w2[j]);
    }
    __syncwarp();
    tmem_st_32x32b_x8(col, w0);
    tmem_st_32x32b_x8(col + 32, w1);
    tmem_st_32x32b_x8(col + 64, w2);
}

// The gated form's second weight.
template <bool GATED>
struct Second {};
template <>
struct Second<true> {
    CUtensorMap map;
};

template <int BN, bool GATED>
__global__ void __launch_bounds__(Cfg<BN, GATED>::threads, 1)
gemm_few_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ Second<GATED> second,
                const __grid_constant__ CUtensorMap mapB, const TcGemmParams p) {
    using C = Cfg<BN, GATED>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* bst = smem + C::a_bufs * kABuf;              // X's pieces
    float* ex = reinterpret_cast<float*>(bst + C::b_stages * 3 * C::b_tile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ex) + C::ex_bytes);
    // FP32 buffer full / free, X's stage full / free, W's pieces ready / free,
    // partial full / free, an issuer's MMAs done (only where a wait gave up)
    constexpr int NF = C::a_bufs, NB = C::b_stages, NA = C::a_stages, ND = C::partials;
    const uint32_t afull0 = smem_u32(bars), afree0 = afull0 + 8 * NF;
    const uint32_t bfull0 = afree0 + 8 * NF, bfree0 = bfull0 + 8 * NB;
    const uint32_t pready0 = bfree0 + 8 * NB, pfree0 = pready0 + 8 * NA;
    const uint32_t dfull0 = pfree0 + 8 * NA, dfree0 = dfull0 + 8 * ND;
    const uint32_t drain0 = dfree0 + 8 * ND;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * (NF + NB + NA + ND) + C::issuers);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const TileSchedule sch = {p.tiles_m, p.num_kb, p.tail_tiles, p.tail_clusters, int(gridDim.x)};
    const int nunits = sched_units(sch, cta);
    uint32_t blocks = 0;                                  // K blocks of all units
    for (int i = 0; i < nunits; ++i) {
        const Unit u = sched_unit(sch, cta, i);
        blocks += uint32_t(u.kb1 - u.kb0);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NF; ++i) {
            mbar_init(afull0 + 8 * i, 1);
            mbar_init(afree0 + 8 * i, C::split_warps);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(bfull0 + 8 * i, 1);
            mbar_init(bfree0 + 8 * i, 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(pready0 + 8 * i, C::split_warps);
            mbar_init(pfree0 + 8 * i, 1);
        }
        for (int i = 0; i < ND; ++i) {
            mbar_init(dfull0 + 8 * i, 1);
            mbar_init(dfree0 + 8 * i, C::acc_warps);
        }
        for (int i = 0; i < C::issuers; ++i) mbar_init(drain0 + 8 * i, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&mapA);
            tma_prefetch_desc(&mapB);
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    // Block g's place in a ring of `count`, and the phase of its barriers there.
    auto slot_of = [](uint32_t g, int count) { return g % count; };
    auto phase_of = [](uint32_t g, int count) { return (g / count) & 1; };

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------ stream of W
            uint32_t g = 0;
            bool ok = true;
            for (int i = 0; i < nunits && ok; ++i) {
                const Unit w = sched_unit(sch, cta, i);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++g) {
                    const uint32_t f = slot_of(g, C::a_bufs);
                    if (!mbar_wait(afree0 + 8 * f, phase_of(g, C::a_bufs) ^ 1, p.err, kDevErrTimeout) || *abort_flag) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(smem + f * kABuf), bar = afull0 + 8 * f;
                    mbar_arrive_expect_tx(bar, kABuf);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int k = kb * 64 + 32 * x;
                        if constexpr (GATED) {
                            tma_load_3d(dst + x * kBox, &mapA, bar, k, w.tile * 64, 0);
                            tma_load_3d(dst + x * kBox + kBox / 2, &second.map, bar, k, w.tile * 64, 0);
                        } else {
                            tma_load_3d(dst + x * kBox, &mapA, bar, k, w.tile * 128, 0);
                        }
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            // no copy may land after this CTA is gone (they have, unless a wait gave up)
            for (uint32_t i = g > NF ? g - NF : 0; i < g; ++i)
                mbar_wait(afull0 + 8 * slot_of(i, NF), phase_of(i, NF), p.err, kDevErrTimeout);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------------ X's pieces
            griddep_wait();                               // the split ahead has written them
            uint32_t g = 0;
            bool ok = true;
            for (int i = 0; i < nunits && ok; ++i) {
                const Unit w = sched_unit(sch, cta, i);
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++g) {
                    const uint32_t s = slot_of(g, C::b_stages);
                    if (!mbar_wait(bfree0 + 8 * s, phase_of(g, C::b_stages) ^ 1, p.err, kDevErrTimeout) || *abort_flag) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = smem_u32(bst + s * 3 * C::b_tile), bar = bfull0 + 8 * s;
                    mbar_arrive_expect_tx(bar, 3 * C::b_tile);
#pragma unroll
                    for (int pc = 0; pc < 3; ++pc)
                        tma_load_3d(st + pc * C::b_tile, &mapB, bar, kb * 64, 0, pc);
                }
            }
            if (!ok) *abort_flag = 1;
            for (uint32_t i = g > NB ? g - NB : 0; i < g; ++i)
                mbar_wait(bfull0 + 8 * slot_of(i, NB), phase_of(i, NB), p.err, kDevErrTimeout);
        }
    } else if (warp < C::acc0) {
        if (warp - 2 < C::issuers) {
            // ----------------------------------------------------- MMA issuers
            const uint32_t leader = elect_one();
            // (not stacked: as many columns as there are rows of X, in 16s)
            const uint32_t idesc = make_idesc(1u, 128, C::stacked ? C::d_cols : (p.N + 15) / 16 * 16);
            // what block g's MMAs wait for: its partial, X's pieces, W's pieces
            auto drained = [&](uint32_t g) {
                return mbar_wait(dfree0 + 8 * slot_of(g, C::partials), phase_of(g, C::partials) ^ 1, p.err, kDevErrTimeout);
            };
            auto x_ready = [&](uint32_t g) {
                return mbar_wait(bfull0 + 8 * slot_of(g, C::b_stages), phase_of(g, C::b_stages), p.err, kDevErrTimeout);
            };
            auto w_ready = [&](uint32_t g) {
                return mbar_wait(pready0 + 8 * slot_of(g, C::a_stages), phase_of(g, C::a_stages), p.err, kDevErrTimeout);
            };
            bool ok = true;
            for (uint32_t g = warp - 2; g < blocks; g += C::issuers) {
                const uint32_t s = slot_of(g, C::b_stages), t = slot_of(g, C::a_stages);
                const uint32_t b = slot_of(g, C::partials);
                if (!C::early || g == 0) ok = drained(g) && x_ready(g) && w_ready(g);
                ok = ok && !*abort_flag;
                if (!__all_sync(0xffffffffu, ok)) {
                    // tensor memory is freed only behind the MMAs issued so far
                    *abort_flag = 1;
                    tc_commit(drain0 + 8 * (warp - 2), leader);
                    mbar_wait(drain0 + 8 * (warp - 2), 0, p.err, kDevErrTimeout);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + b * C::d_cols;
                const uint32_t a = tmem + C::a_base + t * 3 * kPieceCols;
                const uint32_t st = smem_u32(bst + s * 3 * C::b_tile);
                // piece i of W times the operand at `tile`: four K = 16 steps;
                // shift: times 2^-8 what the accumulator holds before them
                auto run = [&](int i, uint32_t tile, bool first, bool shift) {
                    const uint64_t desc = make_sw128_kmajor_desc(tile);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k == 0 && shift)
                            mma_cta1_ta_scaled<8>(d, a + kPieceCols * i, desc, idesc, leader);
                        else
                            mma_cta1_ta(d, a + kPieceCols * i + 8 * k, desc + 2 * k, idesc,
                                        (k == 0 && first) ? 0u : 1u, leader);
                    }
                };
                if constexpr (C::stacked) {
                    run(2, st, true, false);
                    run(1, st, false, true);
                    run(0, st, false, true);
                } else {
                    const uint32_t b0 = st, b1 = st + C::b_tile, b2 = st + 2 * C::b_tile;
                    run(2, b2, true, false);              // band 4
                    run(1, b2, false, true);              // band 3
                    run(2, b1, false, false);
                    run(0, b2, false, true);              // band 2
                    run(1, b1, false, false);
                    run(2, b0, false, false);
                    // the next block's waits, each behind MMAs that are in the queue
                    // (none of them waits for this block's MMAs)
                    const bool next = C::early && g + 1 < blocks;
                    if (next) ok = ok && drained(g + 1);
                    run(0, b1, false, true);              // band 1
                    if (next) ok = ok && x_ready(g + 1);
                    run(1, b0, false, false);
                    if (next) ok = ok && w_ready(g + 1);
                    run(0, b0, false, true);              // band 0
                }
                tc_commit(pfree0 + 8 * t, leader);
                tc_commit(dfull0 + 8 * b, leader);
                tc_commit(bfree0 + 8 * s, leader);
            }
        }
    } else if (warp >= C::split0) {
        // ---------------------------------------------------------- split warps
        const int w = warp - C::split0;
        const int r = 32 * (warp & 3) + lane;             // row: this warp's TMEM lanes
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        for (uint32_t g = 0; g < blocks; ++g) {
            const uint32_t f = slot_of(g, C::a_bufs), t = slot_of(g, C::a_stages);
            if (!mbar_wait(afull0 + 8 * f, phase_of(g, C::a_bufs), p.err, kDevErrTimeout) ||
                !mbar_wait(pfree0 + 8 * t, phase_of(g, C::a_stages) ^ 1, p.err, kDevErrTimeout) ||
                *abort_flag) {
                *abort_flag = 1;
                break;
            }
            __syncwarp();
            tc_fence_after();
            const uint32_t col = (tmem + C::a_base + t * 3 * kPieceCols) | lanes;
#pragma unroll
            for (int kq = w >> 2; kq < 4; kq += C::split_warps / 4)
                split_to_tmem(smem + f * kABuf, col + 8 * kq, r, kq);
            tmem_st_wait();
            tc_fence_before();                            // tensor-memory stores -> the MMA
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(pready0 + 8 * t);
                mbar_arrive(afree0 + 8 * f);
            }
        }
    } else if (warp >= C::acc0) {
        // ---------------------------------------------------- accumulator warps
        constexpr int AC = C::acc_cols;
        const int q = warp & 3, h = (warp - C::acc0) >> 2, aw = warp - C::acc0;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        auto slot = [&](int c) { return c * C::acc_warps + aw; };
        uint32_t g = 0;
        bool ok = true;
        griddep_wait();                                   // the kernel ahead may still read or write C
        for (int i = 0; i < nunits; ++i) {
            const Unit w = sched_unit(sch, cta, i);
            float acc[AC];
#pragma unroll
            for (int j = 0; j < AC; ++j) acc[j] = 0.0f;
            for (int kb = w.kb0; kb < w.kb1 && ok; ++kb, ++g) {
                const uint32_t b = slot_of(g, C::partials);
                if (!mbar_wait(dfull0 + 8 * b, phase_of(g, C::partials), p.err, kDevErrTimeout)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after();
                const uint32_t col = (tmem + b * C::d_cols + h * AC) | lanes;
#pragma unroll
                for (int c = 0; c < AC; c += 8) {
                    uint32_t r0[8], r1[8], r2[8];
                    tmem_ld_32x32b_x8(col + c, r0);
                    if constexpr (C::stacked) {
                        tmem_ld_32x32b_x8(col + BN + c, r1);
                        tmem_ld_32x32b_x8(col + 2 * BN + c, r2);
                    }
                    tmem_ld_wait();
                    if (c + 8 == AC) {
                        // all read: the buffer is free before the sums are formed
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(dfree0 + 8 * b);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v = __uint_as_float(r0[j]);
                        if constexpr (C::stacked)
                            v += fmaf(__uint_as_float(r2[j]), 0x1p-16f, __uint_as_float(r1[j]) * 0x1p-8f);
                        acc[c + j] += v;
                    }
                }
            }
            if (!GATED && (!ok || *abort_flag)) break;
            if (w.publish >= 0) {
                // a later part of a split tile: leave the sums for the owner
                if (!ok) continue;                        // (gated: on to the next meeting)
                float4* dst = reinterpret_cast<float4*>(p.part_ws) + (size_t)slot(cta) * (AC / 4 * 32) + lane;
#pragma unroll
                for (int j = 0; j < AC / 4; ++j)
                    __stcg(dst + j * 32, make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]));
                asm volatile("fence.acq_rel.gpu;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    asm volatile("st.release.gpu.global.u32 [%0], %1;"
                                 :: "l"(p.flags + slot(cta)), "r"(p.epoch) : "memory");
                continue;
            }
            // the owner adds the later parts in K order (bounded waits: those
            // CTAs leave theirs before they wait for anything).  The lanes look
            // at a flag each, then the parts are read four at a time where registers
            // allow it: flag and part after another took 0.7 us each.
            for (int o0 = 1; o0 <= w.others && ok; o0 += 32) {
                const int n = min(32, w.others - o0 + 1);
                unsigned* flag = p.flags + slot(cta + o0 + lane);
                const uint64_t t0 = global_timer_ns();
                while (!__all_sync(0xffffffffu, lane >= n || load_acquire(flag) == p.epoch)) {
                    __nanosleep(32);
                    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > EMU_WAIT_LIMIT_NS)) {
                        if (lane == 0) record_error(p.err, kDevErrTimeout);
                        ok = false;
                        break;
                    }
                }
                if (!ok) break;
                constexpr int kBatch = AC <= 16 ? 4 : 1;
                for (int o = 0; o < n; o += kBatch) {
                    float4 v[kBatch][AC / 4];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const float4* src = reinterpret_cast<const float4*>(p.part_ws) +
                                            (size_t)slot(cta + o0 + min(o + i, n - 1)) * (AC / 4 * 32) + lane;
#pragma unroll
                        for (int j = 0; j < AC / 4; ++j) v[i][j] = __ldcg(src + j * 32);
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        if (o + i >= n) break;
#pragma unroll
                        for (int j = 0; j < AC / 4; ++j) {
                            acc[4 * j] += v[i][j].x;
                            acc[4 * j + 1] += v[i][j].y;
                            acc[4 * j + 2] += v[i][j].z;
                            acc[4 * j + 3] += v[i][j].w;
                        }
                    }
                }
                // consumed: cleared, so that a replay of this launch waits afresh
                __syncwarp();
                if (lane < n) *const_cast<volatile unsigned*>(flag) = 0u;
            }
            const int col0 = h * AC;                      // rows of X
            if constexpr (GATED) {
                // rows 0..63 of the tile are the gate's, 64..127 the same rows
                // of the up projection: their sums meet in shared memory.  Every warp reaches the first barrier of a
                // tile, whether its waits held or not, and they leave together.
                // It also keeps the next tile's sums out until these are read.
                ok = bar_and(1, C::acc_warps * 32, ok && !*abort_flag);
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                constexpr int kRows = BN / C::passes;
                for (int pass = 0; pass < C::passes; ++pass) {
                    if (C::passes == 1 || h == pass) {
                        float* mine = ex + (C::passes == 1 ? h * AC * 128 : 0) + q * 32 + lane;
#pragma unroll
                        for (int j = 0; j < AC; ++j) mine[j * 128] = acc[j];
                    }
                    bar_and(1, C::acc_warps * 32, true);
                    few_gated_epilogue(p, ex, w.tile * 64, pass * kRows, min(kRows, p.N - pass * kRows),
                                       aw * 32 + lane, C::acc_warps * 32);
                    if (pass + 1 < C::passes) bar_and(1, C::acc_warps * 32, true);
                }
            } else {
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                few_epilogue<AC>(acc, p, w.tile * 128 + q * 32 + lane, col0);
            }
        }
        if (!ok) *abort_flag = 1;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "r"(512u) : "memory");
    }
}

// The dynamic shared-memory limit, raised once per device and variant.
constexpr int kMaxDev = 64;
template <int BN, bool GATED>
cudaError_t raise_smem() {
    static std::mutex mu;
    static bool done[kMaxDev] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < kMaxDev && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(gemm_few_kernel<BN, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<BN, GATED>::smem);
    if (e == cudaSuccess && dev < kMaxDev) done[dev] = true;
    return e;
}

template <int BN, bool GATED>
cudaError_t launch_few(const CUtensorMap& mapA, const Second<GATED>& second, const CUtensorMap& mapB,
                       const TcGemmParams& q, int ctas, cudaStream_t stream) {
    cudaError_t e = raise_smem<BN, GATED>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(Cfg<BN, GATED>::threads);
    cfg.dynamicSmemBytes = Cfg<BN, GATED>::smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemm_few_kernel<BN, GATED>, mapA, second, mapB, q);
}

template <bool GATED>
cudaError_t launch_bn(int bn, const CUtensorMap& mapA, const Second<GATED>& second,
                      const CUtensorMap& mapB, const TcGemmParams& q, int ctas, cudaStream_t stream) {
    switch (bn) {
        case 16: return launch_few<16, GATED>(mapA, second, mapB, q, ctas, stream);
        case 32: return launch_few<32, GATED>(mapA, second, mapB, q, ctas, stream);
        case 64: return launch_few<64, GATED>(mapA, second, mapB, q, ctas, stream);
        case 128: return launch_few<128, GATED>(mapA, second, mapB, q, ctas, stream);
        case 160: return launch_few<160, GATED>(mapA, second, mapB, q, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// One CTA per SM: each takes nearly all of an SM's shared memory and all of
// its tensor memory.
int gemm_few_ctas(int sms) { return sms; }

cudaError_t launch_gemm_few(int bn, const CUtensorMap& mapA, const CUtensorMap* mapA2,
                            const CUtensorMap& mapB, const TcGemmParams& p, int sms,
                            cudaStream_t stream) {
    if (p.tiles_m == 0 || p.num_kb == 0) return cudaSuccess;
    TcGemmParams q = p;
    const int resident = gemm_few_ctas(sms);
    const bool split = q.tail_tiles > 0 && q.tail_tiles <= q.tiles_m && q.part_ws && q.flags &&
                       q.tail_clusters >= 1 && q.tail_clusters <= resident &&
                       (q.tiles_m - q.tail_tiles) % resident == 0;
    if (!split) q.tail_tiles = q.tail_clusters = 0;
    const int ctas = sched_grid_clusters(q.tiles_m, q.tail_tiles, q.tail_clusters, resident);
    const cudaError_t e = mapA2 ? launch_bn<true>(bn, mapA, Second<true>{*mapA2}, mapB, q, ctas, stream)
                                : launch_bn<false>(bn, mapA, Second<false>{}, mapB, q, ctas, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace emu
