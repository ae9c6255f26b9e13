// latent_keep.hip -- trees of drafted tokens, and which rows of a paged latent cache stay.
//
// Tree masks: from each token's parent to the set of tokens above it. Select: of a request's
// keys the first, the last, and those with the largest weights. Keep: the rows that stay move together in
// place. Few bytes a request: what bounds them is said at each.
#include <algorithm>

#include "latent_line.hpp"

namespace skinny {
namespace {

using namespace latent;

// ---- tree masks ---------------------------------------------------------------------------
// One workgroup a request, one thread a token, whose set of 512 bits at most is 16 registers. Paths
// double: after r rounds a token has its 2^r nearest ancestors' bits and knows the one above them. The
// launch and the rounds bound it (64 trees of 24 tokens 4.0 us, 8 of 64 4.4, 32 of 512 13.5).
constexpr int MOST_TOKENS = 512, MOST_WORDS = MOST_TOKENS / 32;

__global__ __launch_bounds__(MOST_TOKENS) void latent_tree_mask_kernel(const int32_t *parents, int32_t *mask, int32_t *depth,
                                                                      int tokens, int words) {
    __shared__ uint32_t sets[MOST_WORDS][MOST_TOKENS];
    __shared__ int above[MOST_TOKENS];
    const int j = threadIdx.x;
    const int64_t at = (int64_t)blockIdx.x * tokens + j;
    uint32_t set[MOST_WORDS] = {};
    int up = -1;
    if (j < tokens) {
        const int p = parents[at];
        up = p >= 0 && p < j ? p : -1;
#pragma unroll
        for (int w = 0; w < MOST_WORDS; ++w) set[w] = w == j / 32 ? 1u << (j & 31) : 0u;
    }
    for (int far = 1; far < tokens; far *= 2) {
        above[j] = up;
#pragma unroll
        for (int w = 0; w < MOST_WORDS; ++w)
            if (w < words) sets[w][j] = set[w];
        __syncthreads();
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < MOST_WORDS; ++w)
                if (w < words) set[w] |= sets[w][up];
            up = above[up];
        }
        __syncthreads();
    }
    if (j >= tokens) return;
    int count = 0;
#pragma unroll
    for (int w = 0; w < MOST_WORDS; ++w)
        if (w < words) {
            mask[at * words + w] = (int32_t)set[w];
            count += __popc(set[w]);
        }
    depth[at] = count - 1;
}

// ---- select -------------------------------------------------------------------------------
// One workgroup a request. The weights' bits are turned into whole numbers of the same order and counted by
// their upper 13 bits, which names the bin of the smallest one that stays: all above it stay, none below. Of its
// numbers, a few dozen of thousands where weights are spread like sums of softmax weights, each is ranked
// against each, equal ones by their places; the last one to stay is the border. Where they are too many, two more
// rounds of counts, by 10 and 9 bits, find it. Then each wave, whose keys are a piece of the
// request's, writes its own behind the waves' before it: the list rises. Up to 65536 keys are held in
// registers between the passes; more are read again each time. Chains of dependent steps bound it, and with long
// requests what one CU loads and counts (64 requests of 4200 keys 8.2 us, 4 of 33000 .. 42000 24; keys in LDS
// instead of registers 61 where those took 29, rounds of counts instead of ranks 28 where it is 24).
constexpr int SELECT_THREADS = 1024, SELECT_WAVES = SELECT_THREADS / 64;
constexpr int ROUND_BITS[3] = {13, 10, 9};
constexpr int BINS = 1 << ROUND_BITS[0], PER_BIN = BINS / SELECT_THREADS;
constexpr int RANKED = 256;                  // most numbers that are ranked one by one
constexpr int HELD = 64, BATCH = 8;          // keys a lane holds; loads that go out together

struct SelectArgs {
    const float *weights;
    int64_t w_row;
    const int32_t *lens;
    int32_t *kept, *counts;
    int columns, budget, sinks, recent;
};

// whole numbers that order as the weights do: a NaN above all, both zeros the same
constexpr uint32_t ZERO = 0x80000000u;
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w);
    if (w != w) return ~0u;
    if (w == 0.0f) return ZERO;
    return u >> 31 ? ~u : u | 0x80000000u;
}

// A wave's keys: w[0 .. count), 64 at a time. each(f) calls f(i, number) for whole waves, in rising
// order, with key i + lane's number, or 0, which is no weight's, where there is none.
struct HeldKeys {
    uint32_t x[HELD];
    int count;
    __device__ __forceinline__ HeldKeys(const float *w, int n) : count(n) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int u = 0; u < HELD; u += BATCH)
            if (u * 64 < count) {
#pragma unroll
                for (int b = u; b < u + BATCH; ++b) x[b] = __float_as_uint(w[min(b * 64 + lane, count - 1)]);
            }
#pragma unroll
        for (int u = 0; u < HELD; u += BATCH)
            if (u * 64 < count) {
#pragma unroll
                for (int b = u; b < u + BATCH; ++b) x[b] = b * 64 + lane < count ? order_of(__uint_as_float(x[b])) : 0u;
            }
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll
        for (int u = 0; u < HELD; u += BATCH)
            if (u * 64 < count) {
#pragma unroll
                for (int b = u; b < u + BATCH; ++b) {
                    uint32_t y = x[b];
                    asm volatile("" : "+v"(y));          // what a pass makes of it is not kept for the next
                    f(b * 64, y);
                }
            }
    }
};
struct ReadKeys {
    const float *w;
    int count;
    __device__ __forceinline__ ReadKeys(const float *p, int n) : w(p), count(n) {}
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        const int lane = threadIdx.x & 63;
        for (int u = 0; u < count; u += 64 * BATCH) {
            float v[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) v[b] = w[min(u + b * 64 + lane, count - 1)];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) f(u + b * 64, u + b * 64 + lane < count ? order_of(v[b]) : 0u);
        }
    }
};

template <typename Keys>
__global__ __launch_bounds__(SELECT_THREADS) void latent_select_kernel(SelectArgs a) {
    __shared__ __attribute__((aligned(16))) int bins[BINS];
    __shared__ int sh[SELECT_WAVES], waves_kept[SELECT_WAVES], found[3], ranked;
    __shared__ uint2 near_border[RANKED];                // number, place
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), req = blockIdx.x;
    const int n = min(max(a.lens[req], 0), 1 << 30);
    int32_t *kept = a.kept + (int64_t)req * a.budget;
    const int count = min(n, a.budget);
    if (tid == 0) a.counts[req] = count;
    for (int i = tid + count; i < a.budget; i += SELECT_THREADS) kept[i] = -1;
    if (n <= a.budget) {
        for (int i = tid; i < n; i += SELECT_THREADS) kept[i] = i;
        return;
    }
    // Of m + bare keys between, want stay: 0 <= want < m + bare. The last `bare` have no column, and so the weight 0: they are
    // counted, not read
    const int between = n - a.recent - a.sinks, want = a.budget - a.recent - a.sinks;
    const int m = max(0, min(between, a.columns - a.sinks)), bare = between - m;
    const int piece = (m + SELECT_THREADS - 1) / SELECT_THREADS * 64, i0 = min(m, wave * piece);
    const Keys keys(a.weights + req * a.w_row + a.sinks + i0, min(m, i0 + piece) - i0);
    auto clear = [&]() {
        for (int i = tid; i < BINS / 4; i += SELECT_THREADS) reinterpret_cast<int4 *>(bins)[i] = make_int4(0, 0, 0, 0);
    };
    clear();
    if (tid == 0) ranked = 0;
    if (tid < SELECT_WAVES) waves_kept[tid] = 0;
    for (int i = tid; i < a.sinks; i += SELECT_THREADS) kept[i] = i;
    for (int i = tid; i < a.recent; i += SELECT_THREADS) kept[a.budget - a.recent + i] = n - a.recent + i;
    if (want == 0) return;
    // what the waves before this one counted
    auto before = [&](const int (&of)[SELECT_WAVES]) {
        int s = 0;
#pragma unroll
        for (int v = 0; v < SELECT_WAVES; ++v) s += v < wave ? of[v] : 0;
        return s;
    };
    __syncthreads();

    uint32_t border = 0, known = 0;                      // the border's upper bits, which bits those are
    int still = want, same = 0;                          // to be found among the numbers with these bits; those
    // One more round of counts: of the numbers with the known bits, by the next ones.
    auto round = [&](int shift, int bits, bool first) __attribute__((always_inline)) {
        keys.each([&](int, uint32_t x) {
            if (first ? x != 0 : x - border <= ~known) atomicAdd(&bins[x >> shift & ((1u << bits) - 1)], 1);
        });
        if (bare && tid == 0 && (first || ZERO - border <= ~known)) atomicAdd(&bins[ZERO >> shift & ((1u << bits) - 1)], bare);
        __syncthreads();
        // numbers in the bins above this thread's (threads count down from the topmost)
        int own[PER_BIN], sum = 0;
#pragma unroll
        for (int b = 0; b < PER_BIN; ++b) sum += own[b] = bins[PER_BIN * (SELECT_THREADS - 1 - tid) + b];
        int above = wave_scan(sum);
        if (lane == 63) sh[wave] = above;
        __syncthreads();
        above += before(sh) - sum;
#pragma unroll
        for (int b = PER_BIN - 1; b >= 0; --b) {
            if (above < still && still <= above + own[b]) {
                found[0] = PER_BIN * (SELECT_THREADS - 1 - tid) + b;
                found[1] = still - above;
                found[2] = own[b];
            }
            above += own[b];
        }
        __syncthreads();
        border |= (uint32_t)found[0] << shift;
        known |= ((1u << bits) - 1) << shift;
        still = found[1];
        same = found[2];
    };
    round(32 - ROUND_BITS[0], ROUND_BITS[0], true);

    // The border: numbers above it stay, and of those equal to it the ones up to place `last`.
    int last = 0, mine = 0;                              // mine: the wave's that stay
    int rest = 0;                                        // of the keys without a column, those that stay: the first ones
    if (same <= RANKED && !(bare && ZERO - border <= ~known)) {
        if (ZERO > border) rest = bare;
        keys.each([&](int i, uint32_t x) {
            const uint32_t over = x - border;            // numbers with these bits: 0 .. ~known
            mine += x > border && over > ~known;
            const uint64_t near = __ballot(over <= ~known);
            if (near) {                                  // the same in all lanes
                int at = 0;
                if (lane == 0) at = atomicAdd(&ranked, __popcll(near));
                at = uniform(at) + __popcll(near & ((1ull << lane) - 1));
                if (near >> lane & 1) near_border[at] = make_uint2(x, i0 + i + lane);
            }
        });
        mine = wave_scan(mine);                          // in lane 63
        __syncthreads();
        // a wave ranks every 16th, against four in a lane
        uint2 other[RANKED / 64];
#pragma unroll
        for (int u = 0; u < RANKED / 64; ++u) other[u] = u * 64 + lane < same ? near_border[u * 64 + lane] : make_uint2(0, 0);
        for (int c = wave; c < same; c += SELECT_WAVES) {
            const uint2 own = near_border[c];
            int rank = 0;
#pragma unroll
            for (int u = 0; u < RANKED / 64; ++u)
                rank += __popcll(__ballot(other[u].x > own.x || (other[u].x == own.x && other[u].y < own.y)));
            if (rank < still && lane == 0) atomicAdd(&waves_kept[own.y / (uint32_t)piece], 1);
            if (rank == still - 1 && lane == 0) {
                found[0] = (int)own.x;
                found[1] = (int)own.y;
            }
        }
        __syncthreads();
        border = (uint32_t)found[0];
        last = found[1];
        if (lane == 63) sh[wave] = mine + waves_kept[wave];
    } else {
        clear();
        __syncthreads();
        round(32 - ROUND_BITS[0] - ROUND_BITS[1], ROUND_BITS[1], false);
        clear();
        __syncthreads();
        round(0, ROUND_BITS[2], false);
        int equal = 0;
        keys.each([&](int, uint32_t x) {
            mine += __popcll(__ballot(x > border));
            equal += __popcll(__ballot(x == border));
        });
        if (lane == 0) waves_kept[wave] = equal;
        __syncthreads();
        const int first = before(waves_kept);            // of the equal ones, those of waves before
        int columned = 0;                                // all of them that have a column
#pragma unroll
        for (int v = 0; v < SELECT_WAVES; ++v) columned += waves_kept[v];
        if (ZERO >= border) rest = ZERO > border ? bare : max(0, still - columned);
        if (first < still && still <= first + equal) {   // the last that stays is one of this wave's
            int left = still - first;
            keys.each([&](int i, uint32_t x) {
                const uint64_t here = __ballot(x == border);
                if (left > 0 && left <= __popcll(here)) {
                    if ((here >> lane & 1) && __popcll(here & ((1ull << lane) - 1)) == left - 1) found[1] = i0 + i + lane;
                }
                left -= __popcll(here);
            });
        }
        if (lane == 0) sh[wave] = mine + max(0, min(equal, still - first));
        __syncthreads();
        last = still > columned ? INT_MAX : found[1];
    }
    __syncthreads();
    for (int i = tid; i < rest; i += SELECT_THREADS) kept[a.budget - a.recent - rest + i] = a.sinks + m + i;
    int at = a.sinks + before(sh);
    keys.each([&](int i, uint32_t x) {
        const bool stays = x > border || (x == border && i0 + i + lane <= last);
        const uint64_t all = __ballot(stays);
        if (stays) kept[at + __popcll(all & ((1ull << lane) - 1))] = a.sinks + i0 + i + lane;
        at += __popcll(all);
    });
}

// ---- keep ---------------------------------------------------------------------------------
// Rows move to places that are not behind their own, in place. Columns of a row do not touch each other: a workgroup
// takes one piece of all of a request's rows, in chunks in the order of their places, of which it reads
// all rows before it writes one. Places rise and no row lies before its place, so what a chunk writes no
// later one reads. Pieces of 384 bytes, and 512 rows a chunk (196 KB on its way a workgroup), where there are
// requests enough to fill the chip with them; otherwise 128 bytes and 2048 rows, 262 KB, half of a CU's registers
// (one call after another: 64 requests, of 4096 of 4200 rows each 118 and 122 us, of 500 of 1000 12.7 and 15.7; 16 requests 63
// and 31, 7.5 and 5.7; with 1024 rows a chunk 4 requests of 2048 of 32768 11.2 us where it is 10.6). Many requests the bytes
// bound, which are not read again soon (past the caches: 94 us where it was 100; 64 requests of which most drop some 110 of 4200
// rows 86 us, 390 MB read and written, 4.5 TB/s), few of them the chain of a chunk's loads: list, page ids, rows, stores
// (13 us where the rows come from memory).
constexpr int DIM = 576;
constexpr int KEEP_TURNS = 16;               // rows that a lane has on their way
constexpr int KEEP_WEIGHTS = 2048;           // weights a workgroup

struct KeepArgs {
    uint16_t *cache;
    int64_t c_page, c_row;
    const int32_t *table;
    int64_t t_row;
    const int32_t *lens, *kept, *counts;
    int64_t k_row;
    int32_t *new_lens;
    const float *weights;
    float *new_weights;
    int64_t w_row, nw_row;
    int tokens, most, pages, page, max_pages, columns;
    uint32_t page_mul;                       // see quotient
    int page_shift;
};

// Of a request: its length, the first place that may change, how many rows are kept from there on.
struct Kept {
    int len, base, count, first;             // first: what kept's numbers count from
    __device__ __forceinline__ Kept(const KeepArgs &a, int req) {
        len = min(max(a.lens[req], 0), a.max_pages * a.page);
        first = a.tokens ? len - a.tokens : 0;
        base = max(0, first);
        count = min(max(a.counts[req], 0), min(a.most, len - base));
    }
    // the row that place base + j gets
    __device__ __forceinline__ int source(const KeepArgs &a, int req, int j) const {
        const int64_t r = (int64_t)first + a.kept[req * a.k_row + j];
        return r >= base + j && r < len ? (int)r : base + j;
    }
};

// LANES: of 16 bytes that a workgroup takes of a row.
template <int LANES, int THREADS>
__global__ __launch_bounds__(THREADS) void latent_keep_kernel(KeepArgs a) {
    constexpr int KEEP_ROWS = THREADS / LANES * KEEP_TURNS, SEGS = DIM / 8 / LANES;
    __shared__ int64_t from[KEEP_ROWS], to[KEEP_ROWS];   // elements of the cache; to -1: the row stays
    const int tid = threadIdx.x, seg = blockIdx.x, req = blockIdx.y;
    const Kept k(a, req);
    if (seg >= SEGS) {                                   // weights, which go to an array of their own
        for (int u = 0; u < KEEP_WEIGHTS; u += THREADS) {
            const int place = (seg - SEGS) * KEEP_WEIGHTS + u + tid;
            if (place >= a.columns) return;
            float w = 0.0f;
            if (place < k.base + k.count) {
                const int row = place < k.base ? place : k.source(a, req, place - k.base);
                if (row < a.columns) w = a.weights[req * a.w_row + row];
            }
            a.new_weights[req * a.nw_row + place] = w;
        }
        return;
    }
    if (seg == 0 && tid == 0) a.new_lens[req] = k.base + k.count;
    auto place = [&](int row) {                          // ids outside the pool are clamped
        const int page = page_of(a, row), id = min(max(a.table[req * a.t_row + page], 0), a.pages - 1);
        return id * a.c_page + (row - page * a.page) * a.c_row;
    };
    uint16_t *piece = a.cache + (seg * LANES + tid % LANES) * 8;
    for (int j0 = 0; j0 < k.count; j0 += KEEP_ROWS) {
        int moves = 0;
        for (int j = j0 + tid; j < min(k.count, j0 + KEEP_ROWS); j += THREADS) {
            const int row = k.source(a, req, j);
            const bool move = row != k.base + j;
            if (move) from[j - j0] = place(row);
            to[j - j0] = move ? place(k.base + j) : -1;
            moves |= move;
        }
        if (!__syncthreads_or(moves)) continue;
        u32x4_t x[KEEP_TURNS];
#pragma unroll
        for (int u = 0; u < KEEP_TURNS; ++u) {
            const int j = u * (THREADS / LANES) + tid / LANES;
            x[u] = u32x4_t{0, 0, 0, 0};
            if (j0 + j < k.count && to[j] >= 0)
                x[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(piece + from[j]));
        }
        in_vgpr(x);                                      // all are there
        __syncthreads();
#pragma unroll
        for (int u = 0; u < KEEP_TURNS; ++u) {
            const int j = u * (THREADS / LANES) + tid / LANES;
            if (j0 + j < k.count && to[j] >= 0)
                __builtin_nontemporal_store(x[u], reinterpret_cast<u32x4_t *>(piece + to[j]));
        }
        __syncthreads();                                 // from and to are read
    }
}

}  // namespace

hipError_t launch_latent_tree_mask(const int32_t *parents, int32_t *mask, int32_t *depth, int64_t batch, int64_t tokens,
                                   hipStream_t stream) {
    const unsigned threads = (unsigned)((tokens + 63) / 64 * 64);
    hipLaunchKernelGGL(latent_tree_mask_kernel, dim3((unsigned)batch), dim3(threads), 0, stream, parents, mask, depth,
                       (int)tokens, (int)((tokens + 31) / 32));
    return hipGetLastError();
}

hipError_t launch_latent_select(const skinny_latent_select_args &p, hipStream_t stream) {
    SelectArgs a;
    a.weights = p.weights;
    a.w_row = p.weights_stride;
    a.lens = p.lens;
    a.kept = p.kept;
    a.counts = p.counts;
    a.columns = (int)p.columns;
    a.budget = (int)p.budget;
    a.sinks = (int)p.sinks;
    a.recent = (int)p.recent;
    if (a.columns <= HELD * SELECT_THREADS)
        hipLaunchKernelGGL(latent_select_kernel<HeldKeys>, dim3((unsigned)p.batch), dim3(SELECT_THREADS), 0, stream, a);
    else
        hipLaunchKernelGGL(latent_select_kernel<ReadKeys>, dim3((unsigned)p.batch), dim3(SELECT_THREADS), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_latent_keep(const skinny_latent_keep_args &p, hipStream_t stream) {
    KeepArgs a;
    a.cache = static_cast<uint16_t *>(p.cache);
    a.c_page = p.cache_page_stride;
    a.c_row = p.cache_row_stride;
    a.table = p.table;
    a.t_row = p.table_stride;
    a.lens = p.lens;
    a.kept = p.kept;
    a.counts = p.counts;
    a.k_row = p.kept_stride;
    a.new_lens = p.new_lens;
    a.weights = p.weights;
    a.new_weights = p.new_weights;
    a.w_row = p.weights_stride;
    a.nw_row = p.new_weights_stride;
    a.tokens = (int)p.tokens;
    a.most = (int)p.most;
    a.pages = (int)p.pages;
    a.page = (int)p.page;
    a.max_pages = (int)p.max_pages;
    a.columns = (int)p.columns;
    reciprocal(a.page, a.page_mul, a.page_shift);
    const int64_t wblocks = a.new_weights ? (p.columns + KEEP_WEIGHTS - 1) / KEEP_WEIGHTS : 0;
    // few rows a request, as of a tree's path: few workgroups (64 requests of 5 rows 3.9 us, 8.0 otherwise)
    if (p.batch >= 64 || p.most <= 64)
        hipLaunchKernelGGL((latent_keep_kernel<24, 768>), dim3((unsigned)(DIM / 8 / 24 + wblocks), (unsigned)p.batch),
                           dim3(768), 0, stream, a);
    else
        hipLaunchKernelGGL((latent_keep_kernel<8, 1024>), dim3((unsigned)(DIM / 8 / 8 + wblocks), (unsigned)p.batch),
                           dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace skinny
