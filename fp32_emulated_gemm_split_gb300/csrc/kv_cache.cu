// kv_cache.cu -- the pages of keys and values kept in 8 bits: which pages a
// batch's requests get and where its new tokens go (emu_kv_tables), and the
// store that rounds keys and values into their slots (emu_kv_store);
// include/emu_layers.h.  kv_attention.cu reads them.
#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"
#include "kv_cache.cuh"

#include <type_traits>

namespace emu {
namespace {

// ---------------------------------------------------- tables and slots --
//
//   held = ceil(kept / P), need = ceil((kept + new) / P)
//   page j of a sequence, held <= j < need:  free[taken + sum of (need - held)
//   over the sequences before it + j - held]
//
// Bound by latency: one launch.  Every block sums new and need - held over all
// sequences up to the last one of its rows by itself, so that no block waits for
// another.  Measured: 24 sequences 3.1 us, 1500 with 45,000 tokens 5.9.  A new page's first token is always a new one, and its thread writes
// the table's entry.
constexpr int kTabThreads = 256, kTabSeqs = 4;       // sequences per thread and round
constexpr int kTabRound = kTabThreads * kTabSeqs;
constexpr int kTabRows = 512;                        // rows per block

struct TableParams {
    int B, T, width, page_log;
    int64_t pages, n_free;
    const int32_t *kept, *fresh, *free_pages, *taken;
    int32_t *table, *starts, *lengths, *slots, *positions, *taken_out;
    int* err;
};

__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const TableParams p) {
    __shared__ int first_row[kTabRound], held_at[kTabRound];   // of a round's sequences: first row, tokens held
    __shared__ int64_t first_page[kTabRound];                  // pages given before it, less those it holds
    __shared__ int64_t warp_rows[kTabThreads / 32], warp_pages[kTabThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << p.page_log;
    const int row0 = blockIdx.x * kTabRows, row1 = min(row0 + kTabRows, p.T);
    const int64_t taken = p.taken ? *p.taken : 0;
    int64_t rows = 0, given = 0;                     // of the rounds before this one
    const int rounds = (p.B + kTabRound - 1) / kTabRound;
    const int last_mine = rounds - 1 - (int)(((unsigned)(rounds - 1) + gridDim.x - blockIdx.x % gridDim.x) % gridDim.x);
    for (int r = 0; r < rounds; ++r) {
        if (rows >= row1 && r > last_mine) break;    // neither rows nor sequences of this block are left
        const bool mine = r % (int)gridDim.x == (int)blockIdx.x;
        int kept[kTabSeqs], fresh[kTabSeqs];
        int64_t gets[kTabSeqs], my_rows = 0, my_pages = 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kTabSeqs; ++i) {
            const int b = r * kTabRound + tid * kTabSeqs + i;
            kept[i] = b < p.B ? p.kept[b] : 0;
            fresh[i] = b < p.B ? p.fresh[b] : 0;
            if (kept[i] < 0 || fresh[i] < 0 || (int64_t)kept[i] + fresh[i] > (int64_t)p.width << p.page_log) {
                bad = true;
                kept[i] = fresh[i] = 0;
            }
            gets[i] = (((int64_t)kept[i] + fresh[i] + P - 1) >> p.page_log) - (((int64_t)kept[i] + P - 1) >> p.page_log);
            my_rows += fresh[i];
            my_pages += gets[i];
        }
        // sums over the threads before this one
        int64_t a = my_rows, g = my_pages;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ua = __shfl_up_sync(0xffffffffu, a, o), ug = __shfl_up_sync(0xffffffffu, g, o);
            if (lane >= o) { a += ua; g += ug; }
        }
        if (lane == 31) { warp_rows[warp] = a; warp_pages[warp] = g; }
        __syncthreads();
        int64_t round_rows = 0, round_pages = 0;
#pragma unroll
        for (int w = 0; w < kTabThreads / 32; ++w) {
            if (w < warp) { a += warp_rows[w]; g += warp_pages[w]; }
            round_rows += warp_rows[w];
            round_pages += warp_pages[w];
        }
        a += rows - my_rows;
        g += given - my_pages;
#pragma unroll
        for (int i = 0; i < kTabSeqs; ++i) {
            const int j = tid * kTabSeqs + i, b = r * kTabRound + j;
            const int start = (int)min(a, (int64_t)p.T);
            first_row[j] = b < p.B ? start : INT32_MAX;
            held_at[j] = kept[i];
            first_page[j] = taken + g - (((int64_t)kept[i] + P - 1) >> p.page_log);
            if (mine && b < p.B) {
                // (a sequence whose rows do not all fit ends with those that do)
                const int end = (int)min(a + fresh[i], (int64_t)p.T);
                if (b == 0) p.starts[0] = 0;
                p.starts[b + 1] = end;
                p.lengths[b] = kept[i] + (end - start);
                if (a + fresh[i] > p.T) {
                    bad = true;
                    // (the one that rows run out in: no page is given behind its last row)
                    if (a <= p.T)
                        *p.taken_out = (int)min(taken + g + (((int64_t)kept[i] + (p.T - a) + P - 1) >> p.page_log) -
                                                    (((int64_t)kept[i] + P - 1) >> p.page_log), (int64_t)INT32_MAX);
                }
            }
            a += fresh[i];
            g += gets[i];
        }
        if (bad && mine) record_error(p.err, kDevErrValue);
        __syncthreads();
        // the block's rows that belong to this round's sequences
        const int begin = (int)min(max(rows, (int64_t)row0), (int64_t)row1);
        const int end = (int)min(rows + round_rows, (int64_t)row1);
        for (int t = begin + tid; t < end; t += kTabThreads) {
            int lo = 0, hi = kTabRound;              // the last sequence that starts at t or before it
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (first_row[m] <= t) lo = m; else hi = m;
            }
            const int b = r * kTabRound + lo, pos = held_at[lo] + (t - first_row[lo]), j = pos >> p.page_log;
            int32_t* entry = p.table + (int64_t)b * p.width + j;
            int page;
            if (j < (held_at[lo] + P - 1) >> p.page_log) {
                page = *entry;                       // the page that the tokens held end in
            } else {
                const int64_t at = first_page[lo] + j;
                page = at >= 0 && at < p.n_free ? p.free_pages[at] : -1;
                if (page < 0 || page >= p.pages) page = -1;
                if ((pos & (P - 1)) == 0) *entry = page;
            }
            const bool ok = page >= 0 && page < p.pages;
            if (!ok) record_error(p.err, kDevErrValue);
            p.slots[t] = ok ? (page << p.page_log) + (pos & (P - 1)) : -1;
            p.positions[t] = pos;
        }
        rows += round_rows;
        given += round_pages;
        if (r == rounds - 1 && mine && tid == 0 && rows <= p.T) *p.taken_out = (int)min(taken + given, (int64_t)INT32_MAX);
        __syncthreads();
    }
    if (p.B == 0 && blockIdx.x == 0 && tid == 0) {
        p.starts[0] = 0;
        *p.taken_out = (int)taken;
    }
    // rows behind the last sequence
    for (int t = max(row0, (int)min(rows, (int64_t)p.T)) + tid; t < row1; t += kTabThreads) {
        p.slots[t] = -1;
        p.positions[t] = 0;
    }
}

// ---------------------------------------------------------- the store --
//
//   s = 2^e, the least with max |x| <= 448 s over the page's and head's finite values
//   code = e4m3(x / s)
//
// A power of two costs e4m3 nothing but range (its error is relative), and makes
// the growth of a page's scale nearly free of error: codes divided by a power of
// two stay exact down to the type's subnormal values.  Bound by HBM: the values
// are read once and the codes written once.
//
// A unit of work is what a window of tokens has of runs of new rows that follow each
// other in one page, for one head and side; a run's first token leads, and the
// window that it is in does the run.  For a few tokens a window is one token and a
// warp's (the warps of tokens that do not lead see that and leave); otherwise it is a
// block's, whose warps share long runs and take short ones in turn.  Measured:
// prompts of 17,600 tokens, 8 heads of 128 (118 MB), 38 us, instructions issued in 63 %
// of the cycles; a warp for each run 86 us, magnitudes compared as FP32 values 54.
constexpr int kStoreWarps = 8, kStoreThreads = kStoreWarps * 32;
constexpr int kStoreKeep = 4;                        // chunks of 8 values that a lane keeps from the first look to the second

struct StoreParams {
    const void* in[2];                               // keys, values
    int64_t in_t[2], in_h[2];
    uint8_t* codes[2];
    float* scales[2];
    const int32_t* slots;
    int T, heads, D, page_log, window;               // window: tokens per unit
    uint32_t per_row_inverse;                        // 2^32 / chunks of a row, rounded up
    int wide;                                        // every row of a head starts on 16 bytes
    int64_t slots_all;                               // pages * P
    int64_t units;
    int* err;
};

// 8 neighbouring values as they lie in memory.
template <typename T>
struct Chunk8 {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T* at, bool wide) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(at)[i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else {
            T x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = at[i];
            memcpy(w, x, sizeof(x));
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
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
};

// The scale of values whose largest finite magnitude has these bits.
__device__ __forceinline__ float scale_of(uint32_t top) {
    // top = m 2^E, 1 <= m < 2: top <= 448 2^(E-8) where m <= 1.75
    const int E = (int)(top >> 23) - 127;
    const int e = max(E - 8 + ((top & 0x7FFFFFu) > 0x600000u), -126);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Stores the run of n rows at token t and slot `slot`: by a warp (THREADS 32), or by
// the block (tops: shared memory for its warps' maxima).
template <typename T, int THREADS>
__device__ __forceinline__ void store_run(const StoreParams& p, int side, int head, int t, int slot, int n, uint32_t* tops) {
    const int me = threadIdx.x % THREADS, P = 1 << p.page_log, per_row = p.D >> 3;
    const int64_t in_t = side ? p.in_t[1] : p.in_t[0];
    const T* rows = static_cast<const T*>(side ? p.in[1] : p.in[0]) + head * (side ? p.in_h[1] : p.in_h[0]) + t * in_t;
    const int page = slot >> p.page_log, r0 = slot & (P - 1), chunks = n * per_row;
    const int64_t unit = (int64_t)page * p.heads + head;
    float* const scale = (side ? p.scales[1] : p.scales[0]) + unit;
    uint8_t* const codes = (side ? p.codes[1] : p.codes[0]) + unit * P * p.D;
    const float old = r0 > 0 ? *scale : 0.0f;
    auto from = [&](int c) {                         // chunk c of the run
        const int row = (int)__umulhi((uint32_t)c, p.per_row_inverse);
        return rows + row * in_t + (c - row * per_row) * 8;
    };
    Chunk8<T> kept[kStoreKeep];
    // the largest magnitude as its bits (16-bit types: of the two halves of a word at once)
    constexpr uint32_t kMagnitude = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    constexpr uint32_t kInfinite = sizeof(T) == 4 ? 0x7F800000u : std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    uint32_t bits = 0;
    auto look = [&](const Chunk8<T>& v) {
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i)
            bits = sizeof(T) == 4 ? max(bits, v.w[i] & kMagnitude) : __vmaxu2(bits, v.w[i] & kMagnitude);
    };
    // over the warp, the block
    auto all = [&](uint32_t x) {
        x = __reduce_max_sync(0xffffffffu, x);
        if constexpr (THREADS > 32) {
            if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = x;
            __syncthreads();                         // (all have read the old scale, too)
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) x = max(x, tops[w]);
        }
        return x;
    };
    auto each = [&](auto&& f) {                      // over the run's chunks, those kept and then the others again
#pragma unroll
        for (int i = 0; i < kStoreKeep; ++i)
            if (i * THREADS + me < chunks) f(i * THREADS + me, kept[i]);
#pragma unroll 1
        for (int c = kStoreKeep * THREADS + me; c < chunks; c += THREADS) {
            Chunk8<T> v;
            v.load(from(c), p.wide);
            f(c, v);
        }
    };
#pragma unroll
    for (int i = 0; i < kStoreKeep; ++i)
        if (i * THREADS + me < chunks) kept[i].load(from(i * THREADS + me), p.wide);
    each([&](int, const Chunk8<T>& v) { look(v); });
    bits = all(sizeof(T) == 4 ? bits : max(bits & 0xFFFFu, bits >> 16));
    const bool finite = bits < kInfinite;
    uint32_t top;
    if (finite) {
        if constexpr (sizeof(T) == 4) top = bits;
        else top = __float_as_uint(std::is_same<T, __half>::value ? __half2float(__ushort_as_half((unsigned short)bits))
                                                                  : __uint_as_float(bits << 16));
    } else {
        // infinities and NaN do not count
        top = 0;
        each([&](int, const Chunk8<T>& v) {
            float x[8];
            v.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = __float_as_uint(x[e]) & 0x7FFFFFFFu;
                top = max(top, m < 0x7F800000u ? m : 0u);
            }
        });
        if constexpr (THREADS > 32) __syncthreads();
        top = all(top);
    }
    const float now = fmaxf(old, scale_of(top));
    if (r0 > 0 && now > old) {
        // the page's other rows, rounded again
        const float ratio = old / now;
#pragma unroll 1
        for (int c = me; c < P * per_row; c += THREADS) {
            const int row = (int)__umulhi((uint32_t)c, p.per_row_inverse);
            if (row >= r0 && row < r0 + n) continue;
            uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)c * 8);
            const uint2 w = *at;
            *at = make_uint2(kv_rescale(w.x, ratio), kv_rescale(w.y, ratio));
        }
    }
    if constexpr (THREADS == 32) __syncwarp();
    if (me == 0) *scale = now;
    // a power of two's inverse is exact
    const bool exact = (__float_as_uint(now) & 0x7FFFFFu) == 0 && now >= 1.1754944e-38f && now < 8.5e37f;
    const float inverse = exact ? 1.0f / now : 0.0f;
    auto put = [&](int c, const float (&x)[8]) {
        *reinterpret_cast<uint2*>(codes + ((int64_t)r0 * per_row + c) * 8) =
            make_uint2(kv_codes(x[0], x[1], x[2], x[3]), kv_codes(x[4], x[5], x[6], x[7]));
    };
    if (finite && exact)
        each([&](int c, const Chunk8<T>& v) {
            float x[8];
            v.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inverse;
            put(c, x);
        });
    else
        each([&](int c, const Chunk8<T>& v) {
            float x[8];
            v.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = (__float_as_uint(x[e]) & 0x7F800000u) == 0x7F800000u ? __uint_as_float(0x7FC00000u) : x[e] / now;
            put(c, x);
        });
}

template <typename T, bool BLOCK>
__global__ void __launch_bounds__(kStoreThreads, sizeof(T) == 4 ? 3 : 4) kv_store_kernel(const __grid_constant__ StoreParams p) {
    __shared__ uint32_t tops[2][kStoreWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kStoreWarps + warp;
    if (unit >= p.units) return;
    const int side = (int)(unit & 1), P = 1 << p.page_log;
    const int64_t v = unit >> 1;
    const int head = (int)(v % p.heads), t0 = (int)(v / p.heads) * p.window;

    // Where runs begin or there are none, 32 tokens at a time from t0 on: the slots of the window and of
    // the 64 tokens behind it are loaded at once.
    auto slot_at = [&](int t) { return t < p.T ? p.slots[t] : -1; };
    auto breaks = [&](int slot, int before) {
        return __ballot_sync(0xffffffffu, slot < 0 || slot >= p.slots_all || before < 0 || before != slot - 1 || (slot & (P - 1)) == 0);
    };
    const int t_lane = t0 + lane;
    const int slot_lane = slot_at(t_lane), slot_1 = slot_at(t_lane + 32), slot_2 = slot_at(t_lane + 64);
    const int before_0 = t_lane > 0 ? slot_at(t_lane - 1) : -1;
    if (slot_lane < -1 || slot_lane >= p.slots_all) record_error(p.err, kDevErrValue);
    int up = __shfl_up_sync(0xffffffffu, slot_1, 1), last = __shfl_sync(0xffffffffu, slot_lane, 31);
    const uint32_t break_0 = breaks(slot_lane, before_0), break_1 = breaks(slot_1, lane ? up : last);
    up = __shfl_up_sync(0xffffffffu, slot_2, 1);
    last = __shfl_sync(0xffffffffu, slot_1, 31);
    const uint32_t break_2 = breaks(slot_2, lane ? up : last);
    const bool valid = slot_lane >= 0 && slot_lane < p.slots_all;
    int turn = 0, shared = 0;
    for (uint32_t todo = break_0 & __ballot_sync(0xffffffffu, valid && lane < p.window); todo; todo &= todo - 1) {
        const int which = __ffs(todo) - 1, t = t0 + which;
        const int slot = __shfl_sync(0xffffffffu, slot_lane, which);
        // the next break ends the run
        const uint32_t rest = which == 31 ? 0u : break_0 >> (which + 1);
        int n;
        if (rest) n = __ffs(rest);
        else if (break_1) n = 32 - which + __ffs(break_1) - 1;
        else if (break_2) n = 64 - which + __ffs(break_2) - 1;
        else {
            n = 96 - which;                          // (pages of 128 and 256)
            for (int most = min(P - (slot & (P - 1)), p.T - t); n < most;) {
                const int i = n + lane;
                const uint32_t ends = __ballot_sync(0xffffffffu, i >= most || p.slots[t + i] != slot + i);
                if (ends) {
                    n += __ffs(ends) - 1;
                    break;
                }
                n += 32;
            }
        }
        if constexpr (BLOCK) {
            // (all warps see the same runs)
            if (n * (p.D >> 3) > kStoreKeep * 32) store_run<T, kStoreThreads>(p, side, head, t, slot, n, tops[shared++ & 1]);
            else if (turn++ % kStoreWarps == warp) store_run<T, 32>(p, side, head, t, slot, n, nullptr);
        } else {
            store_run<T, 32>(p, side, head, t, slot, n, nullptr);
        }
    }
}

bool heads_fit(const emu_heads_t& h, int64_t T) {
    constexpr int64_t most = int64_t(1) << 40;
    return h.token_stride >= -most && h.token_stride <= most && h.head_stride >= -most && h.head_stride <= most &&
           (T == 0 || h.data != nullptr);
}

}  // namespace

bool kv_cache_ok(const emu_kv_cache_t& c) {
    if (c.page < 16 || c.page > 256 || (c.page & (c.page - 1)) != 0) return false;
    if (c.D < 16 || c.D > 256 || c.D % 16 != 0 || c.heads < 1 || c.heads > 1024) return false;
    if (c.pages < 0 || c.pages > INT32_MAX / c.page) return false;
    if (c.pages == 0) return true;
    auto on16 = [](const void* q) { return q && reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    auto on4 = [](const void* q) { return q && reinterpret_cast<uintptr_t>(q) % 4 == 0; };
    return on16(c.k) && on16(c.v) && on4(c.k_scale) && on4(c.v_scale);
}

}  // namespace emu

using namespace emu;

extern "C" {

emu_status_t emu_kv_tables(int64_t B, const int32_t* kept, const int32_t* fresh, int64_t pages, int64_t page,
                           const int32_t* free_pages, int64_t n_free, const int32_t* taken, int32_t* table,
                           int64_t width, int64_t T, int32_t* starts, int32_t* lengths, int32_t* slots,
                           int32_t* positions, int32_t* taken_out, emu_stream_t stream) {
    if (B < 0 || B > 1 << 20 || T < 0 || T > kKvMaxRows || width < 0 || width > INT32_MAX || pages < 0 || n_free < 0 ||
        n_free > INT32_MAX)
        return EMU_ERR_INVALID_VALUE;
    if (page < 16 || page > 256 || (page & (page - 1)) != 0 || pages > INT32_MAX / page || width > INT32_MAX / page)
        return EMU_ERR_INVALID_VALUE;
    if (!starts || !taken_out || (n_free > 0 && !free_pages)) return EMU_ERR_INVALID_VALUE;
    if (B > 0 && (!kept || !fresh || !lengths || (width > 0 && !table))) return EMU_ERR_INVALID_VALUE;
    if (T > 0 && (!slots || !positions)) return EMU_ERR_INVALID_VALUE;
    // Every block reads the inputs for itself, and none waits for another: what one writes no other may read.
    const struct { const int32_t* at; int64_t n; } ranges[] = {{starts, B + 1}, {lengths, B}, {slots, T}, {positions, T},
        {taken_out, 1}, {table, B * width}, {kept, B}, {fresh, B}, {free_pages, n_free}, {taken, taken ? 1 : 0}};
    for (int i = 0; i < 6; ++i)                      // (the written ones are first)
        for (int j = i + 1; j < 10; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(ranges[i].at), b = reinterpret_cast<uintptr_t>(ranges[j].at);
            if (ranges[i].n && ranges[j].n && a < b + 4 * (uintptr_t)ranges[j].n && b < a + 4 * (uintptr_t)ranges[i].n)
                return EMU_ERR_INVALID_VALUE;
        }
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    const emu_status_t st = current_device(&d);
    if (st != EMU_OK) return st;
    TableParams p = {};
    p.B = (int)B; p.T = (int)T; p.width = (int)width;
    p.page_log = kv_log2(page);
    p.pages = pages; p.n_free = n_free;
    p.kept = kept; p.fresh = fresh; p.free_pages = free_pages; p.taken = taken;
    p.table = table; p.starts = starts; p.lengths = lengths; p.slots = slots; p.positions = positions;
    p.taken_out = taken_out;
    p.err = d->err;
    const unsigned blocks = (unsigned)(T > kTabRows ? (T + kTabRows - 1) / kTabRows : 1);
    kv_tables_kernel<<<blocks, kTabThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return from_cuda(cudaGetLastError());
}

emu_status_t emu_kv_store(int dtype, int64_t T, const emu_heads_t* k, const emu_heads_t* v, const int32_t* slots,
                          const emu_kv_cache_t* cache, emu_stream_t stream_) {
    if (dtype < EMU_F32 || dtype > EMU_F16 || !k || !v || !cache || T < 0 || T > kKvMaxRows || !kv_cache_ok(*cache) ||
        k->heads != cache->heads || v->heads != cache->heads || !heads_fit(*k, T) || !heads_fit(*v, T) ||
        (T > 0 && !slots))
        return EMU_ERR_INVALID_VALUE;
    if (T == 0) return EMU_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState* d = nullptr;
    const emu_status_t st = current_device(&d);
    if (st != EMU_OK) return st;
    StoreParams p = {};
    const emu_heads_t* in[2] = {k, v};
    const int size = dtype == EMU_F32 ? 4 : 2;
    p.wide = 1;
    for (int s = 0; s < 2; ++s) {
        p.in[s] = in[s]->data;
        p.in_t[s] = in[s]->token_stride;
        p.in_h[s] = in[s]->head_stride;
        if (reinterpret_cast<uintptr_t>(in[s]->data) % 16 || in[s]->token_stride * size % 16 ||
            in[s]->head_stride * size % 16)
            p.wide = 0;
    }
    p.codes[0] = static_cast<uint8_t*>(cache->k);
    p.codes[1] = static_cast<uint8_t*>(cache->v);
    p.scales[0] = cache->k_scale;
    p.scales[1] = cache->v_scale;
    p.slots = slots;
    p.T = (int)T; p.heads = (int)cache->heads; p.D = (int)cache->D;
    p.page_log = kv_log2(cache->page);
    p.slots_all = cache->pages * cache->page;
    p.err = d->err;
    p.per_row_inverse = (uint32_t)(((uint64_t(1) << 32) + p.D / 8 - 1) / (p.D / 8));
    // A warp for each of a few tokens; else a block for each window, up to 32 tokens, of which there are eight or more an SM.
    // Blocks are for runs that a warp alone takes long over: 8 heads of 128 in BF16, runs of 100 tokens, 200 rows 4.5 us (a warp
    // a run 12.3), 4000 rows 9.3 (26.5).  Single tokens are better off with a warp each beyond 32 too: 32 rows 2.9 (2.5), 96
    // rows 5.7 (2.7), 256 rows 8.3 (3.5), 4096 rows 48 (27); runs of 4: 96 rows 4.3 (2.8), 4096 rows 16.0 (16.9).
    const bool block = T > 32;
    p.window = 1;
    while (block && p.window < 32 && (T + 2 * p.window - 1) / (2 * p.window) * cache->heads * 2 >= (int64_t)d->sms * 8) p.window *= 2;
    p.units = (T + p.window - 1) / p.window * cache->heads * 2;
    const unsigned blocks = (unsigned)(block ? p.units : (p.units + kStoreWarps - 1) / kStoreWarps);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    auto go = [&](auto t) {
        using V = decltype(t);
        if (block) kv_store_kernel<V, true><<<blocks, kStoreThreads, 0, stream>>>(p);
        else kv_store_kernel<V, false><<<blocks, kStoreThreads, 0, stream>>>(p);
    };
    if (dtype == EMU_F32) go(float{});
    else if (dtype == EMU_BF16) go(__nv_bfloat16{});
    else go(__half{});
    return from_cuda(cudaGetLastError());
}

}  // extern "C"
