// kv_prompt.cu -- the attention over 8-bit keys and values for many rows of a
// sequence (prompts, drafts of many query heads); the mathematics is
// kv_attention.cu's.
//
// A segment is 128 or 256 rows (a key head's query heads, of one token after another), a
// unit 128 tokens of it.  Bound by the tensor cores and the exponentials, which
// take about as long: S = Q K^T and O = P V are tcgen05 MMAs of 128 x 128 (x D),
// S, P and O in tensor memory, P over the S that it came from.  Roles of a CTA, one per SM:
// one warp copies codes into a ring (bulk copies: as loads, 32 KB a unit waited for the
// L1's misses in flight), four write them as FP16 into swizzled tiles, and two groups of
// four turn S into P, a thread a row, each with a warp that issues its MMAs.  Each group
// has an O of its own (of its own rows, or of the units that it takes in turn with the
// other), so that one's exponentials run beside the other's products; sums of the same
// rows are joined at the segment's end, as are those of CTAs that share a segment
// (kv_join_kernel).  The CTAs take equal consecutive
// ranges of all units, of which a causal tile has as many as it needs.  Each role goes from
// a segment to the next by itself, through rings: the next one's codes and scores are under
// way while the outputs of the last are written.
//
// Measured: three prompts of 2000 tokens behind 1500 to 4500 kept, 32 heads over 8 of
// 128, BF16 (412 GFLOP), 600 us, 687 TFLOP/s.  A unit of 256 rows takes about 5000 cycles, its
// MMAs 2560 (scores of 64 tokens are bound by reading Q again: 512 of them), a group's weights
// 2500; codes, MMAs and weights wait for one another.  A segment costs 17,000 cycles
// besides: Q, units that some row does not see, outputs.  Barriers that let the groups compute by
// turns: 831 us for 709 before.
//
// FP32 rows: two pieces of Q and of P, twice the MMAs.  The scores' maximum is
// taken in a pass of its own over S (0.5 operations a value).  (1200 to 2500 tokens,
// window 1000, 12 heads over 4 of 96: 110 us.)
#include "kv_attention.cuh"

namespace emu {
namespace {

constexpr int kTile = 128;                           // rows of a segment, tokens of a unit
constexpr int kPanel = kTile * 128;                  // 128 rows of 64 FP16 values, swizzled
constexpr int kSoftWarps = 8, kCodeWarps = 4;
constexpr int kMmaWarp = kSoftWarps + kCodeWarps, kCopyWarp = kMmaWarp + 2;    // (an issuer for each group)
constexpr int kThreads = (kCopyWarp + 2) * 32;        // (the last warp fills the fourth group of warps)
enum { kCode, kMma, kCopy };
constexpr int kSegs = 4;                             // segments whose descriptions are held
// Registers of a thread: at launch, of the groups that turn scores into weights, of the others.
constexpr int kLaunchRegs = 128, kSoftRegs = 168, kOtherRegs = 88;
static_assert(kSoftWarps * kSoftRegs + (kThreads / 32 - kSoftWarps) * kOtherRegs <= kThreads / 32 * kLaunchRegs, "no more than there are");
constexpr int kHalf = kTile / 2;                     // tokens of a copied piece: keys, keys, values, values of a unit

// ------------------------------------------------- tiles of a sequence --

// Tile i of a sequence: its units from first(i) to end(i), in the order of tiles and, within one, heads.
// What a segment costs besides (its queries, its outputs, units that some row does not see)
// counts as SETUP units more, that come first, and of which nothing is done: CTAs with many
// short tiles took 1.6 times as long as the others without them.
template <int ROWS, int SETUP>
struct Tiles {
    static constexpr int kSlope = ROWS / kTile;      // units that a tile `group` tiles on lies further
    int n, pos0, window, count;
    uint32_t group;
    __device__ __forceinline__ Tiles(const AttnParams& p, const Seq& s)
        : n(s.n), pos0(max(s.len, 0) - s.n), window(p.window), count((int)(((int64_t)s.n * p.group + ROWS - 1) / ROWS)),
          group(p.group) {}
    static __device__ __forceinline__ int up(int token) { return (token >> 7) + ((token & 127) != 0); }
    __device__ __forceinline__ int end_token(uint32_t i) const {         // behind the last one that a row sees, any tile but the last
        return pos0 + (int)((ROWS * (i + 1) - 1) / group) + 1;
    }
    __device__ __forceinline__ int first_token(uint32_t i) const {       // negative: none before
        return window ? pos0 + (int)(ROWS * i / group) - window + 1 : -1;
    }
    __device__ __forceinline__ int first(int i) const { return max(first_token(i), 0) / kTile; }
    __device__ __forceinline__ int end(int i) const {                    // (a tile that sees nothing has a unit: it is written)
        return max(up(i == count - 1 ? pos0 + n : end_token(i)), 1);
    }
    __device__ __forceinline__ int units(int i) const { return end(i) - first(i); }
    __device__ __forceinline__ int cost(int i) const { return units(i) + SETUP; }
    // sum of max(low, a + kSlope k) over 0 <= k < c
    static __device__ __forceinline__ int64_t ramp(int a, int c, int low) {
        const int flat = min((max(low - a, 0) + kSlope - 1) / kSlope, c);
        return (int64_t)flat * low + (int64_t)(c - flat) * a + kSlope * ((int64_t)(c - 1 + flat) * (c - flat)) / 2;
    }
    // The costs of the first m tiles, m < count: a tile `group` tiles on lies ROWS tokens on.
    __device__ __forceinline__ int64_t before(uint32_t m) const {
        int64_t sum = (int64_t)SETUP * m;
        for (uint32_t r = 0; r < min(group, m); ++r) {
            const int c = (int)((m - r + group - 1) / group);
            sum += ramp(up(end_token(r)), c, 1);
            if (window) sum -= ramp(first_token(r) >> 7, c, 0);
        }
        return sum;
    }
    __device__ __forceinline__ int64_t all() const { return count ? before(count - 1) + cost(count - 1) : 0; }
};

// ------------------------------------------------------- tensor memory --

__device__ __forceinline__ void tmem_st_x16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
           "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
// D = A B (+ D), A and B in shared memory
__device__ __forceinline__ void mma_cta1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t leader) {
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader) : "memory");
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t two(float x) { return pack_f32x2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 8 values as they lie in memory (16 or 32 bytes; wide: from a 16-byte boundary), and as FP32.
template <typename T, int W>
__device__ __forceinline__ void load_words(const T* from, bool wide, uint32_t (&w)[W]) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(from) + i);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    } else {
        T x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = from[i];
        memcpy(w, x, sizeof(x));
    }
}
template <typename T, int W>
__device__ __forceinline__ void values_of(const uint32_t (&w)[W], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[2 * i] = __uint_as_float(w[2 * i]);
            x[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
        } else {
            kv_widen<T>(w[i], x[2 * i], x[2 * i + 1]);
        }
    }
}

// How a CTA's rows and shared memory are shared out.
//
// PAIR (16-bit rows, more than 128 of a sequence): a segment of 256 rows, a tile of 128 for
// each group, every unit for both: half the codes per row are copied and turned.  Otherwise 128
// rows, and the groups take units in turn (few rows; FP32 rows, whose two pieces of Q fill the place).
template <typename T, int NG, bool PAIR>
struct Plan {
    static constexpr bool TWO = sizeof(T) == 4;
    static constexpr int rows = PAIR ? 2 * kTile : kTile;
    static constexpr int q_tiles = PAIR || TWO ? 2 : 1;          // tiles of Q, or pieces
    // Two stages of V, so that they are written while products run; where the groups take units in turn two of K as well
    // (each issuer then meets every phase of its own).  Pairs: 594 us, two of K and one of V 630, two each 607 (three
    // slots are left for codes).
    static constexpr int k_stages = PAIR ? 1 : 2, v_stages = 2;
    // Parts of a unit whose scores and weights go by themselves: the scores of one are under way while the group looks at
    // the other's.  (16-bit pairs: 664 us, 630 in two; FP32 in two 123 us for 105)
    static constexpr int parts = PAIR ? 2 : 1;
    // Units of a group that are added up in tensor memory, a power of two.  An MMA rounds toward zero, 2^-25 of the sum lost on
    // the average as it grows, and a unit is 8 of them, 16 with two pieces: behind so many units O is added to a sum in
    // memory, to the nearest, where sequences are that long (LONG).  Values of one sign, 400,000 tokens: FP32 9e-7 off (1e-3
    // with one sum), FP16 3e-5 besides its roundings (2e-3; 6e-5 with 128 units).  Three FP32 prompts of 2000 behind 3000,
    // 16 heads over 4 of 128: 604 us, 550 with one sum.
    static constexpr uint32_t chain = TWO ? 4 : 64;
    static constexpr int piece = kHalf * NG * 64;                // bytes of a piece of codes
    static constexpr int tiles = (q_tiles + k_stages + v_stages) * NG * kPanel;
    static constexpr int slots = (216 * 1024 - tiles) / piece < 10 ? (216 * 1024 - tiles) / piece : 10;
    static constexpr int bytes = tiles + slots * piece;
    // (17,000 to 20,000 cycles, a unit 5000 to 6000.  Prompts in BF16 and window in FP32: 596 and 115 us; with one unit 625 and
    // 138, with 8 and 6 units 586 and 120.)
    static constexpr int setup = PAIR ? 4 : 3;
};

__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// ------------------------------------------------------------- kernel --

template <typename T, int NG, bool PAIR, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const __grid_constant__ AttnParams p) {
    constexpr bool TWO = sizeof(T) == 4;
    constexpr int PIECES = TWO ? 2 : 1;
    static_assert(!(PAIR && TWO), "one piece of each tile");
    using Pl = Plan<T, NG, PAIR>;
    using Ti = Tiles<Pl::rows, Pl::setup>;
    constexpr int SLOTS = Pl::slots, PARTS = Pl::parts, kPart = kTile / PARTS, KS = Pl::k_stages, VS = Pl::v_stages, kStageBytes = NG * kPanel;
    extern __shared__ __align__(1024) uint8_t smem[];
    // q: [tile or piece][64 values], k and v: [stage][64 values] panels; then the ring of codes as they are
    const uint32_t q_at = smem_u32(smem), k_at = q_at + Pl::q_tiles * kStageBytes, v_at = k_at + KS * kStageBytes,
                   raw_at = v_at + VS * kStageBytes;
    __shared__ __align__(8) uint64_t bars[39 + 2 * SLOTS];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int64_t warp_sum[kThreads / 32];
    // Segments, a ring that the copying warp fills: each role goes from one to the next by itself.  And whether a NaN
    // was taken out of a segment's values.
    __shared__ Work works[kSegs];
    __shared__ int nan_flags[kSegs];
    // of a unit's tiles of 16 tokens: keys, values (eight units: a group may still read a unit's while the copies
    // are four ahead)
    __shared__ float scales[8][2][8];
    __shared__ uint32_t present[SLOTS];              // of a piece's tiles of 16 tokens: those that were copied
    __shared__ float q_factor[2][kTile];
    __shared__ float row_stat[2][kTile][3];          // maximum, sum, reference of each group
    __shared__ float ref_moved[2][kTile];            // what its sums in memory are held against
    const uint32_t k_full = smem_u32(bars), k_free = k_full + 16, v_full = k_full + 32, v_free = k_full + 48,
                   s_full = k_full + 64, p_full = k_full + 96, o_done = k_full + 128,      // [group][part]
                   q_full = k_full + 160, drained = k_full + 176, c_full = k_full + 184, seg_full = k_full + 248,
                   seg_free = seg_full + 8 * kSegs,
                   raw_full = seg_free + 8 * kSegs, raw_free = raw_full + 8 * SLOTS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = p.D;
    volatile int* const aborted = &abort_flag;
    const float nan = __uint_as_float(0x7FC00000u);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + 8 * i, kCodeWarps * 32);
            mbar_init(k_free + 8 * i, PAIR ? 2 : 1);
            mbar_init(v_full + 8 * i, kCodeWarps * 32);
            mbar_init(v_free + 8 * i, PAIR ? 2 : 1);
            mbar_init(q_full + 8 * i, kSoftWarps * 32);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, kTile);
            mbar_init(o_done + 8 * i, 1);
        }
        mbar_init(drained, 2);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(seg_full + 8 * i, 1);
            mbar_init(seg_free + 8 * i, kCopyWarp);  // (a lane of each warp but the copying one and the last)
            nan_flags[i] = 0;
        }
        for (int i = 0; i < 8; ++i) mbar_init(c_full + 8 * i, 8);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_free + 8 * i, kCodeWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    // all units, and where this CTA's range of them begins: a run of sequences per thread
    const int per = (p.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, p.B); ++b) {
        const Seq s = seq_of(p, b);
        mine += Ti(p, s).all() * p.heads;
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    int64_t all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) sum += warp_sum[w];
        all += warp_sum[w];
    }
    griddep_launch_dependents();                     // (kv_join_kernel waits for this one's end)
    const int64_t ctas = min((int64_t)gridDim.x, all);
    bool ok = true;

    uint32_t last_seg = 0;                           // of thread 0: the segment that it had last
    if (blockIdx.x < ctas) {
        const int64_t begin = all * blockIdx.x / ctas;
        if (sum - mine <= begin && begin < sum) {    // (one thread)
            int64_t before = sum - mine;
            int b = tid * per;
            for (;; ++b) {
                const int64_t n = Ti(p, seq_of(p, b)).all() * p.heads;
                if (begin < before + n) break;
                before += n;
            }
            Work& work = works[0];
            work.all = all;
            work.ctas = ctas;
            work.at = begin;
            work.stop = all * (blockIdx.x + 1) / ctas;
            work.base = before;
            work.seq = b;
        }
        __syncthreads();
        {
            // the tile of the sequence: every thread tries some, twice where there are many
            Work& work = works[0];
            const Ti ti(p, seq_of(p, work.seq));
            const int64_t u = (work.at - work.base) / p.heads;
            __shared__ int found;
            int lo = 0, hi = ti.count;               // in [lo, hi)
            while (hi - lo > 1) {
                const int step = (hi - lo + kThreads - 1) / kThreads, i = lo + tid * step;
                __syncthreads();
                if (i < hi) {
                    const int64_t from = ti.before(i), to = i + step < hi ? ti.before(i + step) : INT64_MAX;
                    if (from <= u && u < to) found = i;
                }
                __syncthreads();
                lo = found;
                hi = min(hi, lo + step);
            }
            if (tid == 0) {
                work.begin = work.base + ti.before(lo) * p.heads;            // of the tile's first head
                const int cost = ti.cost(lo);
                work.head = (int)((work.at - work.begin) / cost);
                work.begin += (int64_t)work.head * cost;
                work.row0 = lo * Pl::rows;
            }
        }
        uint32_t j = 0, second = 0, pieces = 0;      // units, those of a second tile, copied pieces of this CTA so far
        uint32_t seg = 0;                            // segments so far
        // The rest of a segment's description, from its sequence, tile, head, first unit and the CTA's next unit.
        auto describe = [&](Work& w) {
            const Seq s = seq_of(p, w.seq);
            const Ti ti(p, s);
            const int i = w.row0 / Pl::rows, units = ti.units(i);
            w.bad = s.len < 0;
            w.start = s.start;
            w.len = max(s.len, 0);
            w.pos0 = w.len - s.n;
            w.end = w.begin + units + Pl::setup;
            // from unit a to unit b
            const int a = max((int)(w.at - w.begin) - Pl::setup, 0), b = max((int)(min(w.stop, w.end) - w.begin) - Pl::setup, 0);
            w.rows = (int)min((int64_t)s.n * p.group - w.row0, (int64_t)Pl::rows);
            w.token0 = (ti.first(i) + a) * kTile;
            w.units = b - a;
            w.starts = a == 0;
            w.whole = w.units == units;
        };
        // The segment behind it: the next head, tile or sequence.
        auto advance = [&](Work& w) {
            w.at = w.begin = w.end;
            if (++w.head == p.heads) {
                w.head = 0;
                Seq s = seq_of(p, w.seq);
                if (w.row0 + (int64_t)Pl::rows < (int64_t)s.n * p.group) {
                    w.row0 += Pl::rows;
                } else {
                    w.row0 = 0;
                    do s = seq_of(p, ++w.seq);
                    while (s.n == 0);
                }
            }
            describe(w);
        };
        if (tid == 0) describe(works[0]);
        __syncthreads();
        // Whether this CTA has a unit of the segment behind w.
        auto goes_on = [](const Work& w) { return w.end + Pl::setup < w.stop; };
        // whether a row (from position pos_a to pos_b) does not see some of the tokens
        auto hides = [&](int tok, int tokens, int pos_a, int pos_b, int len) {
            return tok + tokens > pos_a + 1 || tok + tokens > len || (p.window && tok <= pos_b - p.window);
        };
        // phases: of unit i's stages of keys and values, and of its scores in group t (of a segment from unit j0 on)
        auto k_phase = [](uint32_t i) { return i / KS & 1; };
        auto v_phase = [](uint32_t i) { return i / VS & 1; };
        auto s_phase = [&](uint32_t i, uint32_t t, uint32_t j0, uint32_t second) {
            return PAIR ? (t ? second + (i - j0) : i) & 1 : i >> 1 & 1;
        };
        // Segment seg's description is there (its warps agree).
        auto has_segment = [&]() {
            ok = ok && mbar_wait(seg_full + 8 * (seg % kSegs), seg / kSegs & 1, p.err, kDevErrTimeout) && !*aborted;
            return ok = __all_sync(0xffffffffu, ok);
        };
        // Segment seg is over for this warp; whether another one follows.
        auto leave_segment = [&](const Work& work) {
            const bool more = goes_on(work), both = PAIR && work.rows > kTile;
            if (both) second += work.units;
            j += work.units;
            pieces += 4 * work.units;
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_free + 8 * (seg % kSegs));
            ++seg;
            return more;
        };
        // One segment, as a warp of this role; whether another one follows.
        auto segment = [&](int role) __attribute__((always_inline)) {
            if (role != kCopy && !has_segment()) {
                *aborted = 1;
                return false;
            }
            const Work& work = works[seg % kSegs];
            const int units = work.units, token0 = work.token0, len = work.len, pos0 = work.pos0, head = work.head;
            const int row0 = work.row0, rows = work.rows;
            // tokens that some row of the segment sees
            const int pos_first = pos0 + row0 / p.group, pos_last = pos0 + (row0 + rows - 1) / p.group;
            const int sees_end = max(0, min(len, pos_last + 1));
            const int sees_begin = p.window ? max(0, pos_first - p.window + 1) : 0;
            const uint32_t j0 = j, j1 = j + units;
            const bool both = PAIR && rows > kTile;  // (a second tile)

            if (role == kMma) {
                // ------------------------------------------------- MMAs
                const uint32_t t = warp - kMmaWarp;  // the group
                const uint32_t leader = elect_one();
                const uint32_t idesc_s = make_idesc(0u, kTile, kPart), idesc_o = make_idesc(0u, kTile, D) | kIdescBMn;
                const uint64_t q_desc = make_sw128_kmajor_desc(q_at + (PAIR ? t : 0) * kStageBytes);
                const uint64_t k_desc = make_sw128_kmajor_desc(k_at), v_desc = make_sw128_mn_desc(v_at, kPanel);
                constexpr uint32_t kStage = kStageBytes >> 4;        // a stage (a piece of Q) in descriptors
                const uint32_t s_at = tmem + t * kTile, o_at = tmem + (2 + t) * kTile;
                const bool idle = PAIR && t && !both;
                // (two barriers: the rows may be a segment ahead of a group that had no unit in the one before)
                ok = ok && mbar_wait(q_full + 8 * (seg & 1), seg >> 1 & 1, p.err, kDevErrTimeout);
                ok = __all_sync(0xffffffffu, ok);
                // S = Q K^T, part h of unit i
                auto scores = [&](uint32_t i, int h) {
                    const uint64_t b = k_desc + i % KS * kStage + h * (kPart * 128 >> 4);
#pragma unroll
                    for (int piece = PIECES - 1; piece >= 0; --piece)
#pragma unroll
                        for (int k = 0; k < NG * 4; ++k)
                            if (k < D / 16) {
                                const uint32_t step = (k / 4) * (kPanel >> 4) + (k % 4) * 2;
                                mma_cta1(s_at + h * kPart, q_desc + piece * kStage + step, b + step, idesc_s,
                                         piece < PIECES - 1 || k > 0, leader);
                            }
                    tc_commit(s_full + 8 * (2 * t + h), leader);
                };
                // O += P V
                auto products = [&](uint32_t i, int h, bool go_on) {
                    const uint64_t b = v_desc + i % VS * kStage;
#pragma unroll
                    for (int x = 0; x < kPart / 16; ++x) {
                        // (2048 bytes of V a step; P's pieces beside one another, 32 tokens at a time)
                        const int k = h * (kPart / 16) + x;
                        const uint32_t at = s_at + 32 * (k / 2) + 8 * (k % 2);
                        if constexpr (TWO) mma_cta1_ta(o_at, at + 16, b + k * (2048 >> 4), idesc_o, x > 0 || go_on, leader);
                        mma_cta1_ta(o_at, at, b + k * (2048 >> 4), idesc_o, TWO || x > 0 || go_on, leader);
                    }
                    tc_commit(o_done + 8 * (2 * t + h), leader);
                };
                auto wait = [&](uint32_t bar, uint32_t phase) {
                    ok = ok && mbar_wait(bar, phase, p.err, kDevErrTimeout) && !*aborted;
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    return ok;
                };
                // MMAs of one warp run in the order of their issue, so P is read before the next S is written over it:
                // part 0 of the next unit is on the way while the group looks at part 1.
                const uint32_t by = PAIR ? 1 : 2, from = PAIR ? j0 : j0 + ((j0 ^ t) & 1);
                if (from < j1 && wait(k_full + 8 * (from % KS), k_phase(from))) {
                    if (!idle)
#pragma unroll
                        for (int h = 0; h < PARTS; ++h) scores(from, h);
                    tc_commit(k_free + 8 * (from % KS), leader);
                }
                for (uint32_t i = from; i < j1 && ok; i += by) {
                    const uint32_t next = i + by, phase = s_phase(i, t, j0, second);
                    const bool go_on = LONG ? (i - from) / by % Pl::chain != 0 : i > from;
                    if (!wait(v_full + 8 * (i % VS), v_phase(i))) break;
#pragma unroll
                    for (int h = 0; h < PARTS; ++h) {
                        if (!idle) {
                            if (!wait(p_full + 8 * (2 * t + h), phase)) break;
                            products(i, h, h > 0 || go_on);
                        }
                        if (h == PARTS - 1) tc_commit(v_free + 8 * (i % VS), leader);
                        if (next < j1) {
                            if (h == 0 && !wait(k_full + 8 * (next % KS), k_phase(next))) break;
                            if (!idle) scores(next, h);
                            if (h == PARTS - 1) tc_commit(k_free + 8 * (next % KS), leader);
                        }
                    }
                }
                if (!ok) *aborted = 1;
            } else if (role == kCopy) {
                // ----------------------------------------------- copies
                const int32_t* pages = p.table + (int64_t)work.seq * p.width;
                const int P = 1 << p.page_log, run = min(P, kHalf);          // tokens of a copy
                // lane L < 8 looks after tile L of 16 tokens of a unit: its page (-1: bad, -2: no row sees it)
                auto page_of = [&](uint32_t i) {
                    const int tok = token0 + (int)(i - j0) * kTile + 16 * (lane & 7);
                    if (i >= j1 || tok >= sees_end || tok + 16 <= sees_begin) return -2;
                    const int page = pages[tok >> p.page_log];
                    return page >= 0 && page < p.pages ? page : -1;
                };
                // pages two units ahead, scales one
                int page = -2, page_next = page_of(j0), page_after = page_of(j0 + 1);
                auto scale_of = [&](const float* from) {
                    return page_next >= 0 ? __ldg(from + (int64_t)page_next * p.heads + head) : page_next == -1 ? nan : 0.0f;
                };
                float ks_next = scale_of(p.ks), vs_next = scale_of(p.vs);
                uint32_t g = pieces;
                for (uint32_t i = j0; i < j1 && ok; ++i) {
                    const int tok = token0 + (int)(i - j0) * kTile + 16 * (lane & 7);
                    const float ks = ks_next, vs = vs_next;
                    page = page_next;
                    page_next = page_after;
                    page_after = page_of(i + 2);
                    ks_next = scale_of(p.ks);
                    vs_next = scale_of(p.vs);
                    const int64_t place = (int64_t)max(page, 0) * p.heads + head;
                    if (page == -1) record_error(p.err, kDevErrValue);
                    // A copy brings what it covers of a page, seen or not: a page of 64 tokens and more has one for
                    // a piece, by the lane of its first tile that is seen.
                    const uint32_t seen = __ballot_sync(0xffffffffu, page >= 0) & 0xFF;
                    const int first = (lane & 7) & ~(run / 16 - 1);          // of the tiles of this lane's copy
                    const uint32_t of_copy = ((1u << run / 16) - 1) << first;
                    const bool copies = lane < 8 && (seen & of_copy) && (31 - __clz((seen & of_copy) & -(seen & of_copy))) == lane;
                    const int from = (tok - 16 * ((lane & 7) - first)) & (P - 1);
                    const int64_t offset = ((place << p.page_log) + from) * D;
                    const uint32_t who = __ballot_sync(0xffffffffu, copies);
#pragma unroll
                    for (int piece = 0; piece < 4; ++piece, ++g) {
                        const uint32_t slot = g % SLOTS, bar = raw_full + 8 * slot;
                        ok = ok && mbar_wait(raw_free + 8 * slot, (g / SLOTS & 1) ^ 1, p.err, kDevErrTimeout) && !*aborted;
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        const uint32_t mine = 0xFu << 4 * (piece & 1);
                        if (lane == 0) {
                            present[slot] = (seen & mine) >> 4 * (piece & 1);
                            mbar_arrive_expect_tx(bar, __popc(who & mine) * run * D);
                        }
                        __syncwarp();
                        if (copies && (1u << lane & mine))
                            copy_bytes(raw_at + slot * Pl::piece + (first & 3) * 16 * D, (piece < 2 ? p.k : p.v) + offset,
                                       run * D, bar);
                    }
                    if (lane < 8) {
                        scales[i & 7][0][lane] = ks;
                        scales[i & 7][1][lane] = vs;
                        mbar_arrive(c_full + 8 * (i & 7));
                    }
                }
                // the next segment: as soon as the one that had its place is over
                if (ok && goes_on(work)) {
                    const uint32_t x = seg + 1;
                    ok = mbar_wait(seg_free + 8 * (x % kSegs), (x / kSegs & 1) ^ 1, p.err, kDevErrTimeout) && !*aborted;
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && lane == 0) {
                        Work next = work;
                        advance(next);
                        works[x % kSegs] = next;
                        nan_flags[x % kSegs] = 0;
                        mbar_arrive(seg_full + 8 * (x % kSegs));
                    }
                }
                if (!ok) {
                    // no copy may land after this CTA is gone
                    *aborted = 1;
                    for (uint32_t x = g > SLOTS ? g - SLOTS : 0; x < g; ++x)
                        mbar_wait(raw_full + 8 * (x % SLOTS), x / SLOTS & 1, p.err, kDevErrTimeout);
                }
            } else if (role == kCode) {
                // ------------------------------------------------ codes
                // A thread has 16 values of rows r and r + 32 of a piece (64 tokens) and panel: two rows' quarters by eight
                // lanes, whose stores meet all banks.
                const int ct = tid - kSoftWarps * 32, r = ct >> 2, quarter = ct & 3;
                const uint32_t load_at = r * D + quarter * 16, store_at = r * 128 + (quarter * 32 ^ (r & 7) << 4);
                auto halves = [&](const uint4& v, uint32_t to) {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = kv_half2((uint16_t)w[e]);
                        h[2 * e + 1] = kv_half2((uint16_t)(w[e] >> 16));
                    }
                    sts128(to, h[0], h[1], h[2], h[3]);
                    sts128(to ^ 16, h[4], h[5], h[6], h[7]);
                };
                uint32_t g = pieces;
                // A unit's keys or values, two pieces, as FP16 into a tile.
                auto turn = [&](uint32_t to, int tok, bool clean) {
                    uint4 v[2][NG * 2];
                    uint32_t there[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t slot = (g + x) % SLOTS;
                        ok = ok && mbar_wait(raw_full + 8 * slot, (g + x) / SLOTS & 1, p.err, kDevErrTimeout) && !*aborted;
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) return;
                        const uint32_t from = raw_at + slot * Pl::piece + load_at;
                        there[x] = present[slot];
#pragma unroll
                        for (int n = 0; n < NG; ++n)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint4& w = v[x][2 * n + h];
                                if (n * 64 + quarter * 16 < D)
                                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                                 : "r"(from + n * 64 + h * 32 * D) : "memory");
                            }
                    }
                    if (clean || (there[0] & there[1]) != 0xF || tok < sees_begin || tok + kTile > sees_end) {
                        uint32_t nans = 0;
#pragma unroll
                        for (int n = 0; n < NG * 4; ++n) {
                            uint4& w4 = v[n / (NG * 2)][n % (NG * 2)];
                            const int half = n / (NG * 2), row = r + 32 * (n & 1), at = tok + half * kHalf + row;
                            if (!(there[half] >> (row >> 4) & 1) || at < sees_begin || at >= sees_end) w4 = make_uint4(0, 0, 0, 0);
                            if (clean && n % (NG * 2) / 2 * 64 + quarter * 16 < D) {
                                // a NaN counts in the rows that see its token only: 0 times NaN is NaN, so it is taken
                                // out here and put into those rows at the end
                                uint32_t* const w[4] = {&w4.x, &w4.y, &w4.z, &w4.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t x = nan_bytes(*w[e]);
                                    *w[e] &= ~x;
                                    nans |= x;
                                }
                            }
                        }
                        if (nans) nan_flags[seg % kSegs] = 1;
                    }
#pragma unroll
                    for (int n = 0; n < NG * 4; ++n)
                        if (n % (NG * 2) / 2 * 64 + quarter * 16 < D)
                            halves(v[n / (NG * 2)][n % (NG * 2)],
                                   to + store_at + n % (NG * 2) / 2 * kPanel + (n & 1) * 32 * 128 + n / (NG * 2) * kHalf * 128);
                    __syncwarp();
                    if (lane < 2) mbar_arrive(raw_free + 8 * ((g + lane) % SLOTS));
                    g += 2;
                };
                for (uint32_t i = j0; i < j1 && ok; ++i) {
                    const int tok = token0 + (int)(i - j0) * kTile;
                    const bool edge = hides(tok, kTile, pos_first, pos_last, len);
#pragma unroll 1
                    for (int side = 0; side < 2 && ok; ++side) {
                        const uint32_t s = side ? i % VS : i % KS, to = (side ? v_at : k_at) + s * kStageBytes;
                        ok = mbar_wait((side ? v_free : k_free) + 8 * s, (side ? v_phase(i) : k_phase(i)) ^ 1, p.err, kDevErrTimeout) &&
                             !*aborted;
                        ok = __all_sync(0xffffffffu, ok);
                        turn(to, tok, edge && side);
                        if (!ok) break;
                        fence_async_smem();
                        mbar_arrive((side ? v_full : k_full) + 8 * s);
                    }
                }
                if (!ok) *aborted = 1;
            }
            if (role == kCopy) {                     // (no part in seg_free)
                const bool more = goes_on(work);
                pieces += 4 * units;
                j = j1;
                ++seg;
                __syncwarp();
                return ok && more;
            }
            return leave_segment(work) && ok;
        };
        // Scores to weights, a thread a row; and around them Q of the next segment and the outputs of this one.
        auto scores_to_weights = [&]() __attribute__((always_inline)) {
            const int half = warp >> 2, r = tid & (kTile - 1);           // group, row of its tile
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t s_at = (tmem + half * kTile) | lanes, o_at = (tmem + (2 + half) * kTile) | lanes;
            // O and x times the sums in memory, added up there or, at the end, in O.
            auto move_sums = [&](bool start, bool end, float x) {
                float4* const sums = p.moved + (size_t)(blockIdx.x * 2 + half) * (D >> 2) * kTile + r;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    float4 old[4];
                    tmem_ld_32x32b_x16(o_at + c, o);
#pragma unroll
                    for (int e = 0; e < 4; ++e) old[e] = start ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : sums[(c / 4 + e) * kTile];
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float4 y = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                               __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                        add_to(y, x, old[e]);
                        if (!end) sums[(c / 4 + e) * kTile] = y;
                        o[4 * e] = __float_as_uint(y.x);
                        o[4 * e + 1] = __float_as_uint(y.y);
                        o[4 * e + 2] = __float_as_uint(y.z);
                        o[4 * e + 3] = __float_as_uint(y.w);
                    }
                    if (end) tmem_st_x16(o_at + c, o);
                }
                tmem_st_wait();
                tc_fence_before();
            };
            float m = -INFINITY, l = 0.0f, ref = -INFINITY;
            bool more = true;                        // segment seg follows; segment seg - 1 waits for its last products
            for (;;) {
                row_stat[half][r][0] = m;
                row_stat[half][r][1] = l;
                row_stat[half][r][2] = ref;
                // (behind the barrier all scores of segment seg - 1 have been read, and so has its Q)
                if (more) ok = has_segment();
                ok = bar_and(1, kSoftWarps * 32, ok);
                if (!ok) break;
                // Q: 16 lanes a row, eight values each, 16 rows at a time (all loads before the first use); a group has its
                // tile's rows, or half of the one tile's
                if (more) {
                    const Work& work = works[seg % kSegs];
                    const int row0 = work.row0, rows = work.rows, head = work.head, tile_row = PAIR ? half * kTile : 0;
                    constexpr int ROWS = PAIR ? 32 : 16, LOADS = 8;      // of a warp, at once (16: 709 -> 735 us)
                    const int r0 = (PAIR ? 0 : half * 64) + (warp & 3) * ROWS, d = (lane & 15) * 8;
                    const uint32_t to = q_at + (PAIR ? half * kStageBytes : 0) + (d / 64) * kPanel;
#pragma unroll 1
                    for (int b = 0; b < ROWS; b += 2 * LOADS) {
                        constexpr int W = TWO ? 8 : 4;
                        uint32_t raw[LOADS][W];
#pragma unroll
                        for (int n = 0; n < LOADS; ++n) {
                            const int at = row0 + min(tile_row + r0 + b + 2 * n + (lane >> 4), rows - 1), i = at / p.group;
                            const T* from = static_cast<const T*>(p.q) + (work.start + i) * p.q_t +
                                            (head * p.group + at - i * p.group) * p.q_h + d;
                            if (d < D) load_words(from, p.wide, raw[n]);
                            else
#pragma unroll
                                for (int e = 0; e < W; ++e) raw[n][e] = 0;
                        }
#pragma unroll
                        for (int n = 0; n < LOADS; ++n) {
                            const int rr = r0 + b + 2 * n + (lane >> 4);
                            float x[8], top = 0.0f;
                            values_of<T>(raw[n], x);
#pragma unroll
                            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
                            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            // 2^(14 - E), top = m 2^E; a negative scale turns q
                            const int E = max((int)(__float_as_uint(top) >> 23) - 127, -112);
                            const float up = copysignf(__uint_as_float((uint32_t)(14 - E + 127) << 23), p.scale);
                            if ((lane & 15) == 0)
                                q_factor[PAIR ? half : 0][rr] = score_factor(top, E, fabsf(p.scale));
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float a = x[2 * e] * up, c = x[2 * e + 1] * up;
                                hi[e] = half2_bits(a, c);
                                lo[e] = TWO ? half2_rest(a, c, hi[e]) : 0u;
                            }
                            if (d < D) {
                                const uint32_t line = to + rr * 128 + ((d % 64 * 2) ^ ((rr & 7) << 4));
                                sts128(line, hi[0], hi[1], hi[2], hi[3]);
                                if (TWO) sts128(line + kStageBytes, lo[0], lo[1], lo[2], lo[3]);
                            }
                        }
                    }
                    fence_async_smem();
                    mbar_arrive(q_full + 8 * (seg & 1));
                }
                if (seg > 0) {
                    // --------------------------------------------- the end of segment seg - 1
                    // the last products: of this group's tile, of both groups' units
                    const Work& work = works[(seg - 1) % kSegs];
                    const int units = work.units, token0 = work.token0, len = work.len, pos0 = work.pos0, head = work.head;
                    const int row0 = work.row0, rows = work.rows;
                    const uint32_t j1 = j, j0 = j - units;
                    const bool both = PAIR && rows > kTile, idle = PAIR && half && !both, two_units = !PAIR && units > 1;
                    const int tile_row = PAIR ? half * kTile : 0;
                    const int row = row0 + min(tile_row + r, rows - 1), token = row / p.group, pos = pos0 + token;
                    const int pos_first = pos0 + row0 / p.group, pos_last = pos0 + (row0 + rows - 1) / p.group;
                    auto done = [&](uint32_t i, uint32_t t) {
                        return mbar_wait(o_done + 8 * (2 * t + PARTS - 1), s_phase(i, t, j0, second - (both ? units : 0)), p.err, kDevErrTimeout);
                    };
                    if (!idle) ok = done(j1 - 1, PAIR ? half : (j1 - 1) & 1) && (!two_units || done(j1 - 2, (j1 - 2) & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && !idle) {
                        tc_fence_after();
                        const uint32_t s0 = PAIR ? half : j0 & 1;    // the group that had the first unit
                        const float m_a = row_stat[s0][r][0], l_a = row_stat[s0][r][1], ref_a = row_stat[s0][r][2];
                        float m_all = m_a, ref_all = ref_a, l_all = l_a, x_a = 1.0f, x_b = 0.0f;
                        if (two_units) {
                            const float m_b = row_stat[s0 ^ 1][r][0], l_b = row_stat[s0 ^ 1][r][1], ref_b = row_stat[s0 ^ 1][r][2];
                            m_all = fmaxf(m_a, m_b);
                            ref_all = fmaxf(ref_a, ref_b);
                            l_all = l_a * weight_of(m_a, l_a, m_all) + l_b * weight_of(m_b, l_b, m_all);
                            x_a = share_of(ref_a, ref_all);
                            x_b = share_of(ref_b, ref_all);
                        }
                        const bool live = tile_row + r < rows;
                        float* const slot = p.partial + ((2 * (int64_t)blockIdx.x + work.starts) * p.slot_rows + tile_row + r) * (D + 4);
                        if (!work.whole && live && (PAIR || half == 0))
                            *reinterpret_cast<float4*>(slot) = make_float4(m_all, l_all, ref_all, 0.0f);
                        const bool nan_seen = nan_flags[(seg - 1) % kSegs] != 0;
                        const float f_all = row_factor(work.bad, m_all, l_all, ref_all);
                        T* const to = static_cast<T*>(p.out) + (work.start + token) * p.out_t +
                                      (head * p.group + row - token * p.group) * p.out_h;
                        // eight values of the row from column c
                        auto put = [&](int c, float (&y)[8]) {
                            if (!live) return;
                            if (nan_seen)
                                for (int u = 0; u < units; ++u) {
                                    const int tok = token0 + u * kTile;
                                    if (!hides(tok, kTile, pos_first, pos_last, len)) continue;
                                    const int lo = max(tok, p.window ? pos - p.window + 1 : 0), hi = min(tok + kTile, min(pos, len - 1) + 1);
                                    for (int t = max(lo, 0); t < hi; ++t) {
                                        const int page = p.table[(int64_t)work.seq * p.width + (t >> p.page_log)];
                                        if (page < 0 || page >= p.pages) continue;
                                        const uint8_t* v = p.v + (((((int64_t)page * p.heads + head) << p.page_log) +
                                                                   (t & ((1 << p.page_log) - 1))) * D + c);
                                        for (int e = 0; e < 8; ++e)
                                            if ((v[e] & 0x7F) == 0x7F) y[e] = nan;
                                    }
                                }
                            if (work.whole) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] *= f_all;
                                kv_store8(to + c, p.wide_out, y);
                            } else {
                                *reinterpret_cast<float4*>(slot + 4 + c) = make_float4(y[0], y[1], y[2], y[3]);
                                *reinterpret_cast<float4*>(slot + 8 + c) = make_float4(y[4], y[5], y[6], y[7]);
                            }
                        };
                        if constexpr (PAIR) {
                            // (the next columns on the way while these are written: 830 us for 700, registers of the units' loop)
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t a[16];
                                tmem_ld_32x32b_x16((tmem + (2 + s0) * kTile + c) | lanes, a);
                                tmem_ld_wait();
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float y[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(a[8 * h + e]);
                                    put(c + 8 * h, y);
                                }
                            }
                        } else {
#pragma unroll 1
                            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 8) {
                                uint32_t a[8], b[8];
                                tmem_ld_32x32b_x8((tmem + (2 + s0) * kTile + c) | lanes, a);
                                if (two_units) tmem_ld_32x32b_x8((tmem + (2 + (s0 ^ 1)) * kTile + c) | lanes, b);
                                tmem_ld_wait();
                                float y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    y[e] = __uint_as_float(a[e]) * x_a;
                                    if (two_units) y[e] = fmaf(__uint_as_float(b[e]), x_b, y[e]);
                                }
                                put(c, y);
                            }
                        }
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(seg_free + 8 * ((seg - 1) % kSegs));
                }
                if (!more) break;
                // Q's factors; and the products of segment seg go over what was read here
                ok = bar_and(1, kSoftWarps * 32, ok);
                if (!ok) break;
                const Work& work = works[seg % kSegs];
                const int units = work.units, token0 = work.token0, len = work.len, rows = work.rows, row0 = work.row0;
                const int tile_row = PAIR ? half * kTile : 0;    // the tile's first row of the segment
                const bool both = PAIR && rows > kTile, idle = PAIR && half && !both;    // a second tile; no row in this one
                const int pos = work.pos0 + (row0 + min(tile_row + r, rows - 1)) / p.group;
                const int pos_a = work.pos0 + (row0 + min(tile_row, rows - 1)) / p.group;
                const int pos_b = work.pos0 + (row0 + min(tile_row + kTile, rows) - 1) / p.group;
                const uint32_t j0 = j, j1 = j + units;
                const float factor = q_factor[PAIR ? half : 0][r];
                m = ref = -INFINITY;
                l = 0.0f;
                bool first = true;                       // O's sum is about to begin
                const uint32_t by = PAIR ? 1 : 2, i0 = PAIR ? (idle ? j1 : j0) : j0 + ((j0 ^ half) & 1);
                for (uint32_t i = i0; ok; i += by) {
                    const uint32_t phase = s_phase(i, half, j0, second), at = (i - i0) / by;
                    if (LONG && at >= Pl::chain && (at % Pl::chain == 0 || i >= j1)) {
                        ok = mbar_wait(o_done + 8 * (2 * half + PARTS - 1), phase ^ 1, p.err, kDevErrTimeout) && !*aborted;
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const bool start = at == Pl::chain;
                        if (i < j1 || !start) move_sums(start, i >= j1, start ? 0.0f : share_of(ref_moved[half][r], ref));
                        ref_moved[half][r] = ref;
                        first = true;
                    }
                    if (i >= j1) break;
#pragma unroll 1
                    for (int h = 0; h < PARTS; ++h) {
                        ok = mbar_wait(s_full + 8 * (2 * half + h), phase, p.err, kDevErrTimeout) &&
                             mbar_wait(c_full + 8 * (i & 7), i >> 3 & 1, p.err, kDevErrTimeout) && !*aborted;
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int tok = token0 + (int)(i - j0) * kTile + h * kPart;
                        const uint32_t s_part = s_at + h * kPart;
                        const bool edge = hides(tok, kPart, pos_a, pos_b, len);
                        const int last = min(pos, len - 1), from = p.window ? pos - p.window : -1;
                        const float* const ks = scales[i & 7][0] + h * (kPart / 16);
                        const float* const vs = scales[i & 7][1] + h * (kPart / 16);
                        if constexpr (!TWO) {
                            // Most units: the maximum and the reference as they are, and P held back until it is known
                            // that none of it passed FP16's range.
                            if (!edge && !first) {
                                uint32_t w[kPart / 2], sc[2][16];
                                __half2 most = __float2half2_rn(0.0f);
                                uint64_t sums = 0;
                                const uint64_t m2 = two(-m);
                                const float up = exp2_of(m - ref);
                                float f_most = 0.0f;
                                tmem_ld_32x32b_x16(s_part, sc[0]);
#pragma unroll
                                for (int g = 0; g < kPart / 16; ++g) {
                                    tmem_ld_wait();
                                    if (g + 1 < kPart / 16) tmem_ld_32x32b_x16(s_part + 16 * (g + 1), sc[(g + 1) & 1]);
                                    const float f = vs[g] * up;
                                    const uint64_t k2 = two(factor * ks[g]), f2 = two(f);
                                    f_most = fmaxf(f_most, f);
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const uint64_t x = fma_f32x2(pack_f32x2(sc[g & 1][e], sc[g & 1][e + 1]), k2, m2);
                                        const uint64_t pp = pack_f32x2(__float_as_uint(exp2_of(lo_of(x))), __float_as_uint(exp2_of(hi_of(x))));
                                        sums = add_f32x2(sums, pp);
                                        const uint64_t ww = mul_f32x2(pp, f2);
                                        const uint32_t h = half2_bits(lo_of(ww), hi_of(ww));
                                        most = __hmax2(most, *reinterpret_cast<const __half2*>(&h));
                                        w[8 * g + e / 2] = h;
                                    }
                                }
                                const float more = lo_of(sums) + hi_of(sums);
                                const bool fits = !__hisinf(__low2half(most)) && !__hisinf(__high2half(most)) && !(more > 1e37f) &&
                                                  f_most < kFarScale && m > -INFINITY;
                                if (__all_sync(0xffffffffu, fits)) {
                                    l += more;
#pragma unroll
                                    for (int c = 0; c < kPart / 32; ++c)
                                        tmem_st_x16(s_part + 32 * c, *reinterpret_cast<const uint32_t(*)[16]>(w + 16 * c));
                                    tmem_st_wait();
                                    tc_fence_before();
                                    mbar_arrive(p_full + 8 * (2 * half + h));
                                    continue;
                                }
                            }
                        }
                        // the largest score, and the largest with its page's bound
                        float top = -INFINITY, over = -INFINITY;
                        uint32_t sc[2][16];              // (16 scores on the way while those before are looked at)
                        tmem_ld_32x32b_x16(s_part, sc[0]);
#pragma unroll 1
                        for (int c = 0; c < kPart; c += 32)
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                tmem_ld_wait();
                                if (g == 0) tmem_ld_32x32b_x16(s_part + c + 16, sc[1]);
                                else if (c + 32 < kPart) tmem_ld_32x32b_x16(s_part + c + 32, sc[0]);
                                if (edge) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const int t = tok + c + 16 * g + e;
                                        if (t > last || t <= from) sc[g][e] = 0xFF800000u;
                                    }
                                }
                                float x[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[e] = fmaxf(fmaxf(__uint_as_float(sc[g][e]), __uint_as_float(sc[g][4 + e])),
                                                 fmaxf(__uint_as_float(sc[g][8 + e]), __uint_as_float(sc[g][12 + e])));
                                float y = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                                // (what no row sees has scale 0)
                                if (y > -INFINITY) {
                                    y *= factor * ks[c / 16 + g];
                                    top = fmaxf(top, y);
                                    over = fmaxf(over, y + (float)scale_bound(vs[c / 16 + g]));
                                }
                            }
                        if (top > m) {
                            l *= exp2_of(m - top);
                            m = top;
                        }
                        // o's reference: p s_v is 2^13 to 2^14 at its largest (scale_bound is 14 below), so that its two pieces end at
                        // 2^-38 of it.  16-bit rows: 2^7 to 2^8 at first, and the reference moves where it would pass 2^14, so
                        // O is rescaled less often (three prompts of 2000: 595 to 611 us over five sets of values, 595 to 606
                        // with 2^3 at first, 617 with 2^9).
                        const bool move = over > ref;
                        if (__any_sync(0xffffffffu, move)) {
                            const float now = move ? over + (TWO ? 0.0f : 6.0f) : ref;
                            if (!first) {
                                // (O is whole once the products of the group's part before are)
                                ok = mbar_wait(o_done + 8 * (2 * half + (h ^ (PARTS - 1))), phase ^ (h == 0), p.err, kDevErrTimeout);
                                if (!__all_sync(0xffffffffu, ok)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                const float f = move ? exp2_of(ref - now) : 1.0f;
#pragma unroll 1
                                for (int c = 0; c < D; c += 8) {
                                    uint32_t o[8];
                                    tmem_ld_32x32b_x8(o_at + c, o);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st_32x32b_x8(o_at + c, o);
                                }
                                tmem_st_wait();
                            }
                            ref = now;
                        }
                        first = false;
                        float m0 = m == -INFINITY ? 0.0f : m, up = m == -INFINITY ? 0.0f : exp2_of(m - ref), back = 1.0f;
                        {
                            float most = 0.0f;
#pragma unroll
                            for (int c = 0; c < kPart / 16; ++c) most = fmaxf(most, vs[c]);
                            if (most * up > kFarScale && m > ref) {
                                m0 = ref;
                                up = 1.0f;
                                back = exp2_of(ref - m);
                            }
                        }
                        uint64_t sums = 0;
                        tmem_ld_32x32b_x16(s_part, sc[0]);
#pragma unroll 1
                        for (int c = 0; c < kPart; c += 32) {
                            uint32_t w[16], rest[16];
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                tmem_ld_wait();
                                if (g == 0) tmem_ld_32x32b_x16(s_part + c + 16, sc[1]);
                                else if (c + 32 < kPart) tmem_ld_32x32b_x16(s_part + c + 32, sc[0]);
                                const uint64_t k2 = two(factor * ks[c / 16 + g]), m2 = two(-m0), f2 = two(vs[c / 16 + g] * up);
#pragma unroll
                                for (int e = 0; e < 16; e += 2) {
                                    const uint64_t x = fma_f32x2(pack_f32x2(sc[g][e], sc[g][e + 1]), k2, m2);
                                    float p0 = exp2_of(lo_of(x)), p1 = exp2_of(hi_of(x));
                                    if (edge) {
                                        const int t0 = tok + c + 16 * g + e;
                                        if (t0 > last || t0 <= from) p0 = 0.0f;
                                        if (t0 + 1 > last || t0 + 1 <= from) p1 = 0.0f;
                                    }
                                    const uint64_t pp = pack_f32x2(__float_as_uint(p0), __float_as_uint(p1));
                                    sums = add_f32x2(sums, pp);
                                    const uint64_t ww = mul_f32x2(pp, f2);
                                    float w0 = lo_of(ww), w1 = hi_of(ww);
                                    if (edge) {          // (a page that is not there has no scale)
                                        if (p0 == 0.0f) w0 = 0.0f;
                                        if (p1 == 0.0f) w1 = 0.0f;
                                    }
                                    w[8 * g + e / 2] = half2_bits(w0, w1);
                                    if constexpr (TWO) rest[8 * g + e / 2] = half2_rest(w0, w1, w[8 * g + e / 2]);
                                }
                            }
                            // over the scores just read
                            tmem_st_x16(s_part + c, w);
                            if constexpr (TWO) tmem_st_x16(s_part + c + 16, rest);
                        }
                        l = fmaf(lo_of(sums) + hi_of(sums), back, l);
                        tmem_st_wait();
                        tc_fence_before();
                        mbar_arrive(p_full + 8 * (2 * half + h));
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                more = goes_on(work);
                j = j1;
                if (both) second += units;
                ++seg;
            }
            if (!ok) *aborted = 1;
            last_seg = seg ? seg - 1 : 0;
        };
        // (a unit's P waits in registers: with 128 for all, spilled, prompts took 700 us)
        if (works[0].units == 0) {                   // (nothing but a segment's setup: the next CTA does it)
        } else if (warp < kSoftWarps) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftRegs));
            scores_to_weights();
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
            if (warp < kMmaWarp) while (segment(kCode)) {}
            else if (warp < kCopyWarp) while (segment(kMma)) {}
            else if (warp == kCopyWarp) {
                if (lane == 0) mbar_arrive(seg_full);            // (the first segment)
                while (segment(kCopy)) {}
            }
        }
        // (tensor memory is freed behind the MMAs issued; they are done unless a wait gave up)
        if ((warp == kMmaWarp || warp == kMmaWarp + 1) && (!ok || *aborted)) {
            const uint32_t leader = elect_one();
            tc_commit(drained, leader);
            mbar_wait(drained, 0, p.err, kDevErrTimeout);
        }
    }
    if (tid == 0) {
        Work w = works[last_seg % kSegs];
        if (blockIdx.x >= ctas || w.whole || !w.starts) w.units = 0;     // (or 0 as it is)
        p.shared[blockIdx.x] = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u));
}

template <typename T, int NG, bool PAIR, bool LONG>
cudaError_t launch(AttnParams p, int dtype, int sms, cudaStream_t stream) {
    using Pl = Plan<T, NG, PAIR>;
    auto kern = kv_prompt_kernel<T, NG, PAIR, LONG>;
    static bool done[kMaxDevices] = {};              // (g_mu is held)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        // (the warps' shares of registers add up to what the block is launched with, or they would wait for ever)
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, kern);
        if (e == cudaSuccess && a.numRegs != kLaunchRegs) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Pl::bytes);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    p.slot_rows = Pl::rows;
    kern<<<(unsigned)sms, kThreads, Pl::bytes, stream>>>(p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(dtype, p, (unsigned)sms, Pl::rows / 16, stream);
}

// Whether a group may have more units of a segment than one sum takes: by what a table's row holds, or a window and the
// tokens of a segment.  (Without the moves' code 16-bit prompts take 605 us for 630: registers of the units' loop.)
template <typename Pl>
bool is_long(const AttnParams& p) {
    const int64_t kept = (int64_t)p.width << p.page_log, seen = p.window ? (int64_t)p.window + Pl::rows / p.group + 1 : kept;
    return (kept < seen ? kept : seen) > (int64_t)Pl::chain * kTile;
}

template <typename T, int NG>
cudaError_t launch_rows(const AttnParams& p, int dtype, int64_t max_rows, int sms, cudaStream_t stream) {
    if constexpr (sizeof(T) == 2) {
        if (max_rows > kTile)
            return is_long<Plan<T, NG, true>>(p) ? launch<T, NG, true, true>(p, dtype, sms, stream)
                                                 : launch<T, NG, true, false>(p, dtype, sms, stream);
        if (!is_long<Plan<T, NG, false>>(p)) return launch<T, NG, false, false>(p, dtype, sms, stream);
    }
    return launch<T, NG, false, true>(p, dtype, sms, stream);
}

template <typename T>
cudaError_t launch_typed(const AttnParams& p, int dtype, int64_t max_rows, int sms, cudaStream_t stream) {
    return p.D <= 64 ? launch_rows<T, 1>(p, dtype, max_rows, sms, stream) : launch_rows<T, 2>(p, dtype, max_rows, sms, stream);
}

}  // namespace

cudaError_t launch_prompt(int dtype, const AttnParams& p, int64_t max_rows, int sms, cudaStream_t stream) {
    if (dtype == EMU_F32) return launch_typed<float>(p, dtype, max_rows, sms, stream);
    if (dtype == EMU_BF16) return launch_typed<__nv_bfloat16>(p, dtype, max_rows, sms, stream);
    return launch_typed<__half>(p, dtype, max_rows, sms, stream);
}

}  // namespace emu
