// kv_cache.cu -- the pages of keys and values kept in 8 bits: which pages a
// batch's requests get and where its new tokens go (emu_kv_tables), and the
// store that rounds keys and values into their slots (emu_kv_store);
// include/emu_layers.h.  kv_attention.cu reads them.
#include "emu_device.cuh"
#include "emu_host.h"
#include "emu_layers.h"
#include "kv_cache.cuh"

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
// another.  A new page's first token is always a new one, and its thread writes
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
                if (a + fresh[i] > p.T) bad = true;
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
        if (r == rounds - 1 && mine && tid == 0) *p.taken_out = (int)min(taken + given, (int64_t)INT32_MAX);
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
// A unit of work is a run of new rows that follow each other in one page, for one
// head and side; a warp does it.  The run's first token leads: the warps of the
// others see that and leave.
constexpr int kStoreWarps = 4;
constexpr int kStoreKeep = 8;                        // chunks of 8 values that a lane keeps from the first look to the second

struct StoreParams {
    const void* in[2];                               // keys, values
    int64_t in_t[2], in_h[2];
    uint8_t* codes[2];
    float* scales[2];
    const int32_t* slots;
    int T, heads, D, page_log, window;               // window: tokens per unit
    int wide;                                        // every row of a head starts on 16 bytes
    int64_t slots_all;                               // pages * P
    int64_t units;
    int* err;
};

// The scale of values whose largest finite magnitude has these bits.
__device__ __forceinline__ float scale_of(uint32_t top) {
    // top = m 2^E, 1 <= m < 2: top <= 448 2^(E-8) where m <= 1.75
    const int E = (int)(top >> 23) - 127;
    const int e = max(E - 8 + ((top & 0x7FFFFFu) > 0x600000u), -126);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <typename T>
__global__ void __launch_bounds__(kStoreWarps * 32) kv_store_kernel(const StoreParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kStoreWarps + (threadIdx.x >> 5);
    if (unit >= p.units) return;
    const int side = (int)(unit & 1), P = 1 << p.page_log;
    const int64_t v = unit >> 1;
    const int head = (int)(v % p.heads), t0 = (int)(v / p.heads) * p.window;
    const int per_row = p.D >> 3;                    // chunks
    const T* in = static_cast<const T*>(side ? p.in[1] : p.in[0]) + head * (side ? p.in_h[1] : p.in_h[0]);
    const int64_t in_t = side ? p.in_t[1] : p.in_t[0];
    uint8_t* const all_codes = side ? p.codes[1] : p.codes[0];
    float* const all_scales = side ? p.scales[1] : p.scales[0];

    // the window's tokens that lead a run
    bool leads = false;
    const int t_lane = t0 + lane;
    int slot_lane = -1;
    if (lane < p.window && t_lane < p.T) {
        slot_lane = p.slots[t_lane];
        const int before = t_lane > 0 ? p.slots[t_lane - 1] : -1;
        leads = slot_lane >= 0 && slot_lane < p.slots_all &&
                (before < 0 || before != slot_lane - 1 || (slot_lane & (P - 1)) == 0);
        if (slot_lane < -1 || slot_lane >= p.slots_all) record_error(p.err, kDevErrValue);
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, leads); todo; todo &= todo - 1) {
        const int which = __ffs(todo) - 1, t = t0 + which;
        const int slot = __shfl_sync(0xffffffffu, slot_lane, which);
        const int page = slot >> p.page_log, r0 = slot & (P - 1);
        int n = 1;                                   // rows of the run
        for (int most = min(P - r0, p.T - t); n < most;) {
            const int i = n + lane;
            const uint32_t ends = __ballot_sync(0xffffffffu, i >= most || p.slots[t + i] != slot + i);
            if (ends) {
                n += __ffs(ends) - 1;
                break;
            }
            n += 32;
        }
        const int chunks = n * per_row;
        const T* rows = in + t * in_t;
        float kept[kStoreKeep][8];
        uint32_t top = 0;
        auto look = [&](const float (&x)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t a = __float_as_uint(x[e]) & 0x7FFFFFFFu;
                top = max(top, a < 0x7F800000u ? a : 0u);
            }
        };
        auto from = [&](int c) {                     // chunk c of the run
            const int row = c / per_row;
            return rows + row * in_t + (c - row * per_row) * 8;
        };
#pragma unroll
        for (int i = 0; i < kStoreKeep; ++i) {
            const int c = i * 32 + lane;
            if (c < chunks) kv_load8(from(c), p.wide, kept[i]);
        }
#pragma unroll
        for (int i = 0; i < kStoreKeep; ++i)
            if (i * 32 + lane < chunks) look(kept[i]);
        for (int c = kStoreKeep * 32 + lane; c < chunks; c += 32) {
            float x[8];
            kv_load8(from(c), p.wide, x);
            look(x);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        float* scale = all_scales + (int64_t)page * p.heads + head;
        uint8_t* codes = all_codes + ((int64_t)page * p.heads + head) * (int64_t)P * p.D;
        float now = scale_of(top);
        if (r0 > 0) {
            const float old = *scale;
            now = fmaxf(old, now);
            if (now > old) {
                // the page's other rows, rounded again
                const float ratio = old / now;
                for (int c = lane; c < P * per_row; c += 32) {
                    const int row = c / per_row;
                    if (row >= r0 && row < r0 + n) continue;
                    uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)c * 8);
                    const uint2 w = *at;
                    *at = make_uint2(kv_rescale(w.x, ratio), kv_rescale(w.y, ratio));
                }
            }
        }
        __syncwarp();
        if (lane == 0) *scale = now;
        // a power of two's inverse is exact
        const bool exact = (__float_as_uint(now) & 0x7FFFFFu) == 0 && now >= 1.1754944e-38f && now < 8.5e37f;
        const float inverse = exact ? 1.0f / now : 0.0f;
        auto write = [&](int c, const float (&x)[8]) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = x[4 * i + e];
                    const bool finite = (__float_as_uint(z) & 0x7F800000u) != 0x7F800000u;
                    y[e] = !finite ? __uint_as_float(0x7FC00000u) : exact ? z * inverse : z / now;
                }
                w[i] = kv_codes(y[0], y[1], y[2], y[3]);
            }
            *reinterpret_cast<uint2*>(codes + ((int64_t)r0 * per_row + c) * 8) = make_uint2(w[0], w[1]);
        };
#pragma unroll
        for (int i = 0; i < kStoreKeep; ++i)
            if (i * 32 + lane < chunks) write(i * 32 + lane, kept[i]);
        for (int c = kStoreKeep * 32 + lane; c < chunks; c += 32) {
            float x[8];
            kv_load8(from(c), p.wide, x);
            write(c, x);
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
    if (!starts || !taken_out || taken_out == taken || (n_free > 0 && !free_pages)) return EMU_ERR_INVALID_VALUE;
    if (B > 0 && (!kept || !fresh || !lengths || (width > 0 && !table))) return EMU_ERR_INVALID_VALUE;
    if (T > 0 && (!slots || !positions)) return EMU_ERR_INVALID_VALUE;
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
    // a token per unit until they fill the GPU's warps, up to 32
    p.window = 1;
    while (p.window < 32 && (T + p.window - 1) / p.window * cache->heads * 2 > (int64_t)d->sms * 64) p.window *= 2;
    p.units = (T + p.window - 1) / p.window * cache->heads * 2;
    const unsigned blocks = (unsigned)((p.units + kStoreWarps - 1) / kStoreWarps);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (dtype == EMU_F32) kv_store_kernel<float><<<blocks, kStoreWarps * 32, 0, stream>>>(p);
    else if (dtype == EMU_BF16) kv_store_kernel<__nv_bfloat16><<<blocks, kStoreWarps * 32, 0, stream>>>(p);
    else kv_store_kernel<__half><<<blocks, kStoreWarps * 32, 0, stream>>>(p);
    return from_cuda(cudaGetLastError());
}

}  // extern "C"
