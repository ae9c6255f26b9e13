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
// launch bounds it.
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
// One workgroup a request. The weights' bits, turned into whole numbers of the same order, are searched from the
// top for the smallest one that stays: three rounds of counts by 11, 11 and 10 bits. Then each wave
// takes a piece of the keys, counts those above that number and equal to it, and writes its own behind the
// waves' before it, so that the list rises and of equal ones the first stay. The weights (4 bytes a key) are
// read once where they fit LDS, and from L2 five times where not. Chains of dependent steps
// bound it.
constexpr int SELECT_THREADS = 1024, SELECT_WAVES = SELECT_THREADS / 64;
constexpr int BINS = 2048, PER_BIN = BINS / SELECT_THREADS;
constexpr int CACHED = 36864;                // keys in LDS, 144 KB

struct SelectArgs {
    const float *weights;
    int64_t w_row;
    const int32_t *lens;
    int32_t *kept, *counts;
    int columns, budget, sinks, recent;
};

// whole numbers that order as the weights do: a NaN above all, both zeros the same
__device__ __forceinline__ uint32_t order_of(float w) {
    const uint32_t u = __float_as_uint(w);
    if (w != w) return ~0u;
    if (w == 0.0f) return 0x80000000u;
    return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ __launch_bounds__(SELECT_THREADS) void latent_select_kernel(SelectArgs a) {
    __shared__ uint32_t cache[CACHED];
    __shared__ int bins[BINS];
    __shared__ int sh[2 * SELECT_WAVES], found[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, req = blockIdx.x;
    const int n = min(max(a.lens[req], 0), a.columns);
    int32_t *kept = a.kept + (int64_t)req * a.budget;
    const int count = min(n, a.budget);
    if (tid == 0) a.counts[req] = count;
    for (int i = tid + count; i < a.budget; i += SELECT_THREADS) kept[i] = -1;
    if (n <= a.budget) {
        for (int i = tid; i < n; i += SELECT_THREADS) kept[i] = i;
        return;
    }
    for (int i = tid; i < a.sinks; i += SELECT_THREADS) kept[i] = i;
    for (int i = tid; i < a.recent; i += SELECT_THREADS) kept[a.budget - a.recent + i] = n - a.recent + i;
    // of m keys between, want stay: 0 <= want < m
    const int m = n - a.recent - a.sinks, want = a.budget - a.recent - a.sinks;
    if (want == 0) return;
    const float *w = a.weights + req * a.w_row + a.sinks;
    const bool cached = m <= CACHED;
    if (cached) {
        constexpr int U = 8;
        for (int i0 = tid; i0 < m; i0 += U * SELECT_THREADS) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = i0 + u * SELECT_THREADS < m ? w[i0 + u * SELECT_THREADS] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * SELECT_THREADS < m) cache[i0 + u * SELECT_THREADS] = order_of(x[u]);
        }
    }
    auto number = [&](int i) { return cached ? cache[i] : order_of(w[i]); };

    uint32_t border = 0, known = 0;                      // the border's upper bits, which bits those are
    int still = want;                                    // to be found among those with these upper bits
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, mine = PER_BIN * (SELECT_THREADS - 1 - tid);
        const uint32_t low = round == 2 ? BINS / 2 - 1 : BINS - 1;
        for (int i = tid; i < BINS; i += SELECT_THREADS) bins[i] = 0;
        __syncthreads();
        for (int i = tid; i < m; i += SELECT_THREADS) {
            const uint32_t x = number(i);
            if ((x & known) == border) atomicAdd(&bins[x >> shift & low], 1);
        }
        __syncthreads();
        // numbers in the bins above this thread's (threads count down from the topmost)
        int own = 0;
#pragma unroll
        for (int b = 0; b < PER_BIN; ++b) own += bins[mine + b];
        int sum = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 63) sh[wave] = sum;
        __syncthreads();
        int above = sum - own;
        for (int v = 0; v < wave; ++v) above += sh[v];
#pragma unroll
        for (int b = PER_BIN - 1; b >= 0; --b) {
            const int here = bins[mine + b];
            if (above < still && still <= above + here) {
                found[0] = mine + b;
                found[1] = still - above;
            }
            above += here;
        }
        __syncthreads();
        border |= (uint32_t)found[0] << shift;
        known |= low << shift;
        still = found[1];
    }

    // above the border all, of those equal to it the first `still`
    const int piece = (m + SELECT_THREADS - 1) / SELECT_THREADS * 64, i0 = min(m, wave * piece), i1 = min(m, i0 + piece);
    int more = 0, equal = 0;
    for (int i = i0 + lane; i < i1; i += 64) {
        const uint32_t x = number(i);
        more += x > border;
        equal += x == border;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        more += __shfl_xor(more, d);
        equal += __shfl_xor(equal, d);
    }
    __syncthreads();
    if (lane == 0) {
        sh[wave] = more;
        sh[SELECT_WAVES + wave] = equal;
    }
    __syncthreads();
    more = equal = 0;
    for (int v = 0; v < wave; ++v) {
        more += sh[v];
        equal += sh[SELECT_WAVES + v];
    }
    for (int i = i0; i < i1; i += 64) {                  // whole waves
        const uint32_t x = i + lane < i1 ? number(i + lane) : 0u;
        const uint64_t up = __ballot(i + lane < i1 && x > border), same = __ballot(i + lane < i1 && x == border);
        const uint64_t before = (1ull << lane) - 1;
        const int g = more + __popcll(up & before), e = equal + __popcll(same & before);
        if ((up >> lane & 1) || ((same >> lane & 1) && e < still)) kept[a.sinks + g + min(e, still)] = a.sinks + i + lane;
        more += __popcll(up);
        equal += __popcll(same);
    }
}

// ---- keep ---------------------------------------------------------------------------------
// Rows move to places that are not behind their own, in place. Columns of a row do not touch each other: a workgroup
// takes one 128-byte piece of all of a request's rows, in chunks in the order of their places, of which it
// reads all rows before it writes one. Places rise and no row lies before its place, so what a chunk writes
// no later one reads. A chunk is 1024 rows, 128 KB on its way a workgroup, since a request has
// only 9 of them.
constexpr int DIM = 576, SEGS = DIM * 2 / 128;
constexpr int KEEP_THREADS = 512, KEEP_TURNS = 16, KEEP_ROWS = KEEP_THREADS / 8 * KEEP_TURNS;
constexpr int KEEP_WEIGHTS = 4 * KEEP_THREADS;           // weights a workgroup

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
    uint32_t page_mul;                       // see page_of
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

__global__ __launch_bounds__(KEEP_THREADS) void latent_keep_kernel(KeepArgs a) {
    __shared__ int64_t from[KEEP_ROWS], to[KEEP_ROWS];   // elements of the cache; to -1: the row stays
    const int tid = threadIdx.x, seg = blockIdx.x, req = blockIdx.y;
    const Kept k(a, req);
    if (seg >= SEGS) {                                   // weights, which go to an array of their own
        for (int u = 0; u < KEEP_WEIGHTS; u += KEEP_THREADS) {
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
    uint16_t *piece = a.cache + seg * 64 + (tid & 7) * 8;
    for (int j0 = 0; j0 < k.count; j0 += KEEP_ROWS) {
        int moves = 0;
        for (int j = j0 + tid; j < min(k.count, j0 + KEEP_ROWS); j += KEEP_THREADS) {
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
            const int j = u * (KEEP_THREADS / 8) + (tid >> 3);
            x[u] = u32x4_t{0, 0, 0, 0};
            if (j0 + j < k.count && to[j] >= 0) x[u] = *reinterpret_cast<const u32x4_t *>(piece + from[j]);
        }
        in_vgpr(x);                                      // all are there
        __syncthreads();
#pragma unroll
        for (int u = 0; u < KEEP_TURNS; ++u) {
            const int j = u * (KEEP_THREADS / 8) + (tid >> 3);
            if (j0 + j < k.count && to[j] >= 0) *reinterpret_cast<u32x4_t *>(piece + to[j]) = x[u];
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
    hipLaunchKernelGGL(latent_select_kernel, dim3((unsigned)p.batch), dim3(SELECT_THREADS), 0, stream, a);
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
    page_reciprocal(a.page, a.page_mul, a.page_shift);
    const int64_t wblocks = a.new_weights ? (p.columns + KEEP_WEIGHTS - 1) / KEEP_WEIGHTS : 0;
    hipLaunchKernelGGL(latent_keep_kernel, dim3((unsigned)(SEGS + wblocks), (unsigned)p.batch), dim3(KEEP_THREADS), 0, stream,
                       a);
    return hipGetLastError();
}

}  // namespace skinny
