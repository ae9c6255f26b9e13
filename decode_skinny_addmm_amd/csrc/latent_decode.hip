// latent_decode.hip -- absorbed latent attention of new tokens over a paged latent cache.
//
// For request i with n = lens[i] cached rows c_k = [z_k, r_k] (512 latents, 64 rotated numbers)
// and its `tokens` newest positions, query (j, h) attends to keys k < n - tokens + j + 1:
//     s_k = scale * q . c_k,   out = sum_k softmax(s)_k z_k,   lse = log sum_k exp(s_k).
//
// What bounds it: each cached row is 1152 bytes and serves tokens * heads queries at 2 * 1088
// operations each: up to 64 query rows a request the cache's bytes bound it (beyond, see below).
//   * A workgroup holds all query rows of a request (up to 128; more go in groups) and reads a
//     contiguous run of its keys once, in tiles of 32 keys through a ring of 4 LDS stages (two
//     stages, 74 KB, are in flight behind the one computed on; three with 128 rows, whose value
//     product does not run a tile behind). Keys and values are the same staged rows.
//   * One workgroup a CU; the tiles of all requests are one line, cut into equal runs, one a
//     workgroup, whatever the lengths (which only the device knows). A request cut between
//     workgroups leaves fp32 partial sums in the workspace, joined by a second kernel.
//   * 4 waves as WR row groups x WD groups of latent dims: each wave computes the whole scores
//     of its rows (repeated by the WD waves: matrix time is spare, and no scores cross waves)
//     and its dims of the output, so the only barrier is the ring's.
// With a window the line holds only the tiles that a request's rows see between them; with a tree of new tokens
// the tiles that hold them are masked by the tokens' words, which lie in LDS (see seen_keys).
// Measured: one request of 131071 keys x 32 heads 34 us (151 MB, 4.4 TB/s; its inner loop 6 TB/s) and 7
// for the join; 96 requests of about 4000 keys x 128 heads 119 us (484 MB read, 89 MB of partials
// written) and 22 for the join; 64 requests of 3000 keys x 64 heads 55 us (240 MB read) and 7.6 for the
// join; windows of 4096 of 64 requests x 16 heads 59 us (311 MB read, 5.3 TB/s) and 4.8; trees of 24 tokens x 8
// heads over 32 requests of 4096 keys 84 and 14, of 64 x 16 over 8 of 8000 138 and 16; a tree of 7 x 8 over 500
// keys 10 and 4. With 128 rows the matrix instructions take 40% of a wave's time (36% of the kernel's, with its
// start and end), and neither they nor memory bound it alone: in this layout of one wave a
// SIMD, registers full of sums and queries leave no room to run a tile's softmax beside the next one's
// products.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "latent_line.hpp"

namespace skinny {
namespace {

using namespace latent;

constexpr int L = 512, DIM = 576;            // latents, numbers of a cached row
constexpr int KT = 32;                       // keys a tile
constexpr int SEGS = DIM * 2 / 128;          // 128-byte pieces of a row
constexpr int STAGES = 4;
constexpr int STAGE_BYTES = KT * DIM * 2;
constexpr int THREADS = 256;

struct DecodeArgs {
    const uint16_t *q;
    int64_t q_row, q_head;                   // strides in elements
    const uint16_t *cache;
    int64_t c_page, c_row;
    const int32_t *table;
    int64_t t_row;
    const int32_t *lens;
    uint16_t *out;
    int64_t o_row, o_head;
    float *lse;
    float *work;                             // partial sums: see part_floats
    int2 *cuts;                              // a unit (request and row group): its first partial, its last workgroup
    int batch, tokens, heads, pages, page, max_pages;
    int rows, all_groups, grid;              // rows a request, row groups a request, workgroups
    int groups, side;                        // row groups of a request in the line, and side by side: see shared_run
    int lead;                                // see request_tiles
    uint32_t page_mul, head_mul;             // see quotient
    int page_shift, head_shift;
    float c;                                 // scale * log2(e)
};

// What a row sees of the context is bounded, or the new tokens are a tree: see skinny_latent_mask.
struct MaskedArgs : DecodeArgs {
    const int32_t *tree, *depth;             // NULL: a chain
    int64_t tree_row, depth_row;             // strides of a request
    int words;                               // of a token in tree
    int window, sinks;                       // window 0: the whole context, sinks 0
};
constexpr int MOST_WORDS = 16;               // trees of 512 tokens

// One partial: MB rows x 512 sums in the waves' own register order, then MB maxima, MB sums.
template <int MB>
__host__ __device__ constexpr int64_t part_floats() { return (int64_t)MB * (L + 2); }

__device__ __forceinline__ int clamp_len(const DecodeArgs &a, int n) {
    return min(max(n, 0), a.max_pages * a.page);         // at most 2^30: checked by the caller
}
__device__ __forceinline__ int request_len(const DecodeArgs &a, int i) { return clamp_len(a, a.lens[i]); }
// the same for a request that is the same in all lanes, as a scalar load: waiting for a vector
// load would wait for the ring's loads too
__device__ __forceinline__ int uniform_len(const DecodeArgs &a, int i) {
    typedef const __attribute__((address_space(4))) int32_t *constant_ptr;
    return clamp_len(a, ((constant_ptr)(uintptr_t)a.lens)[i]);
}
// The key tiles that a request's rows see between them, in the order in which they are taken: one at
// least, so that an empty request's outputs are written too. With a window they are those of the
// first keys and, `skip` further on, those from the first row's window on. (Positions rise by one a step of
// the chain or tree, the first row's is the lowest, and windows do not begin past it.)
struct Tiles {
    int count, head, skip;
    __device__ __forceinline__ int at(int t) const { return t < head ? t : t + skip; }
};
__device__ __forceinline__ Tiles tiles_of(const DecodeArgs &, int len) { return {max(1, (len + KT - 1) / KT), INT_MAX, 0}; }
__device__ __forceinline__ Tiles tiles_of(const MaskedArgs &a, int len) {
    Tiles s{max(1, (len + KT - 1) / KT), INT_MAX, 0};
    if (a.window) {
        const int head = (min(a.sinks, len) + KT - 1) / KT, from = max(0, len - a.tokens + 1 - a.window) / KT;
        if (from > head) {
            s.head = head;
            s.skip = from - head;
            s.count -= s.skip;
        }
    }
    return s;
}
// What a unit (request and row group) takes of the line: its tiles, and ahead of them `lead` places of no work, so
// that a run that ends one unit and begins the next, which loads queries and leaves partials twice, is given
// fewer tiles. (8 requests x 1024 rows x 8000 keys: runs of 57 tiles in one unit took 121 to 129 us, in two 132
// to 141.)
template <typename A>
__device__ __forceinline__ int request_tiles(const A &a, int i) { return tiles_of(a, request_len(a, i)).count + a.lead; }

// Bits b of a tile of keys that starts at k0 with k0 + b < x.
__device__ __forceinline__ uint32_t keys_below(int x, int k0) {
    const int n = x - k0;
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
}

// Runs that the line is cut into: at most one a CU, and with many rows fewer where that leaves less
// work. A run of r tiles takes r t, and the total / r runs leave partials of b bytes each, written and
// read at rate w: r t + 2 b total / (r w) is least at r = sqrt(2 b total / (w t)), so that there are
// sqrt(total) sqrt(w t / 2 b) runs. With the measured t = 1.7 us for 64 rows and 2.4 for 128 (64 requests
// of 3000, 6000 and 12000 keys give 1.8 to 1.9 and 2.2 to 2.6, which moves the factors by 6% at most)
// and w = 4.5 TB/s (128 heads: 32 requests x 1000 keys 57 -> 50 us, one of 10000 37 -> 34; 64 heads:
// 2 x 3000 26 -> 25; of 16 and 32 rows the partials are too small to matter).
// A line of so few tiles that this gives each a run of its own gives them with the places of no work, too, which are
// `total`'s others (in us where pairs of tiles shared runs, and so: 8 requests x 40 keys x 64 heads 13.9 and 11.0, 3 x 80 x 128
// heads 17.3 and 14.2).
template <int MB>
__device__ __forceinline__ int runs(int most, int64_t total, int64_t tiles) {
    const int grid = (int)min((int64_t)most, total);
    if constexpr (MB < 64) return grid;
    constexpr float FACTOR = MB == 64 ? 5.4f : 4.5f;
    if (tiles <= (int)(FACTOR * FACTOR)) return grid;
    return min(grid, max(1, (int)(FACTOR * sqrtf((float)total))));
}

// Row groups of a request read the same keys. Where they divide the chip well they are not behind each other in
// the line but side by side: the line holds a request's tiles once, and each of its runs is taken by `side`
// workgroups, one a group, at the same time and on one XCD, whose L2 serves all but the first. (Workgroups go to
// the XCDs in turn.) 8 groups read 90 MB where it was 575, 2 groups 162 where it was 330, which takes them from 91 to
// 88 us; 8 groups as long as before. Runs are counted in whole `side`s, which costs 2 or 3 groups of a short request
// most. One request, in us behind each other and side by side: 2 groups x 640 keys 18.9 and 20.7, x 4000 26.6 and 27.3;
// 8 x 1000 25.5 and 26.2, x 4000 37.2 and 36.8; 29 x 96 23.6 and 17.6, x 4000 65.6 and 62.8; 60 x 256 38.9 and 30.2, x 4000
// 95.6 and 94.5; 128 x 96 28.2 and 21.6, x 4000 152 and 150. 16 requests of 5 groups x 1000 56.4 and 52.4, of 28 164 and 159.
struct SharedRun {
    int run, own;                            // the run, the row group (of those side by side); run -1: none
};
__device__ __forceinline__ SharedRun shared_run(int block, int grid, int side) {
    if (side == 1) return {block < grid ? block : -1, 0};
    const int all = grid * side, per = (all + 7) / 8, p = (block & 7) * per + (block >> 3);
    if (block >> 3 >= per || p >= all) return {-1, 0};
    return {p / side, p % side};
}

template <typename T, int WR, int WD>
struct Shape {
    static constexpr int MB = T::ROWS * WR;              // rows a workgroup
    static constexpr int ND = L / T::DIMS / WD;          // dim tiles a wave
    static constexpr int KS = DIM / T::KSTEP;            // K steps of the score product
    static constexpr int NO4 = T::NO / 4;                // 4-register groups of a dim tile
    // softmax of a tile beside the score product of the next: takes registers that 128 rows x 512
    // sums leave no room for
    static constexpr bool FLOW = MB < 128;
    // Fragments read ahead of the matrix instructions (they need about 130 cycles; a 32 x 32 instruction
    // takes 32 of them, a 16 x 16 one 16): of keys, and of values.
    static constexpr int KAHEAD = MB == 128 ? 7 : 11, VAHEAD = 3;
};

// What a workgroup stages, in order: for each unit (request and row group) of its run, the unit's
// query rows as QT tiles of 32 rows, then its tiles of keys. One stream through the ring, so that
// a unit's first tiles are loaded while the last one's outputs are written.
struct Cursor {
    int req, g, len, t, t0, end;             // unit; next item: query tile t + QT if t < 0, else key tile t
    Tiles tiles;
    int taken;                               // places of the run in this unit
    int64_t left;                            // places of the run from this unit on
    bool more;
    // from place `first` of the unit on
    template <typename A>
    __device__ __forceinline__ void enter(const A &a, int first, int qt) {
        len = uniform_len(a, req);
        tiles = tiles_of(a, len);
        t = -qt;
        taken = (int)min((int64_t)(tiles.count + a.lead - first), left);
        t0 = max(0, first - a.lead);
        end = first + taken - a.lead;
        more = end > 0;                      // a run may end with places of no work
    }
};
// An item whose load is due: this lane's row (of the request's queries, or of its cache page).
struct Due {
    int row, req;
    int kind;                                // 0: none, 1: queries, 2: keys
};
// The same where a wave's 8 rows of keys lie in one page: all of it the same in all lanes.
struct BlockDue {
    int row;                                 // the wave's first row
    int kind;                                // 0: none, 1: queries, 2 + r: keys, of which rows up to r are the request's
    int id;                                  // of its page
};
// Where an item's pieces come from (base and each lane's own bytes, or its address) and go to.
struct Source {
    const uint16_t *base;
    uint32_t own;
    int kind;                                // that `own` is of
    int to;
    uint64_t lanes;                          // all if there is an item, else none
};

// of a row's pieces, those that go out with group `at` of `of` (both known when compiled)
template <bool BLOCKS, int I = 0>
__device__ __forceinline__ void pieces_at(int at, int of, const Source &p) {
    if constexpr (I < SEGS) {
        if (I * of / SEGS == at) {
            if constexpr (BLOCKS) load_lds_piece_in<I>(p.lanes, p.base, p.own, p.to);
            else load_lds_piece_in<I>(p.lanes, p.base, p.to);
        }
        pieces_at<BLOCKS, I + 1>(at, of, p);
    }
}

// MASKED: of the keys before its own, a row sees those of a mask, held a tile as 32 bits.
// BLOCKS: pages are whole groups of 8 rows, so that the 8 keys that a wave stages of a tile lie in one page, whose
// id and address are worked out once a wave, by the scalar unit. A step's cursor and addresses take the wave
// some 970 cycles otherwise, and 775 so, of a tile of 128 rows' 4300 (8 requests of 8000 keys x 1024 rows: 157 and 148
// us). Not with 16 rows: their short tiles gain nothing, and where the caches hold the rows they lose (reads of LDS wait
// for the page id's scalar load with them, which may be why; 64 requests of 2100 keys x 16 heads: 32 us by lanes, 34 by blocks; of 3000 40.5 and
// 43.5; 32 heads the same either way).
template <typename T, int WR, int WD, bool MASKED, bool BLOCKS>
__global__ __launch_bounds__(THREADS) void latent_decode_kernel(std::conditional_t<MASKED, MaskedArgs, DecodeArgs> a) {
    typedef Shape<T, WR, WD> S;
    typedef typename T::acc_t acc_t;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE_BYTES + 4 * STAGES * 256];
    __shared__ int64_t sh[8];
    // of each wave's rows, the tree's words and behind them where a row's window begins
    __shared__ uint32_t masks[MASKED ? THREADS / 64 * T::ROWS * (MOST_WORDS + 1) : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int row = T::row(lane), grp = T::grp(lane);
    const int wr = wave % WR, d0 = (wave / WR) * (L / WD);
    constexpr int QT = (S::MB + KT - 1) / KT;            // query tiles a unit
    constexpr int PW = BLOCKS ? SEGS : SEGS + 1;         // loads a wave issues a stage: pieces, and a word of page ids

    Line<decltype(a), THREADS> line;
    line.measure(a, (int64_t)a.batch * a.groups * (max(1, (a.max_pages * a.page + KT - 1) / KT) + a.lead), sh);
    const int grid = uniform(max(1, runs<S::MB>(a.grid, line.total * a.side,
                                                (line.total - (int64_t)a.batch * a.groups * a.lead) * a.side) / a.side));
    const SharedRun mine = shared_run(blockIdx.x, grid, a.side);
    if (mine.run < 0) return;
    // me: the number of its partials
    const int own_group = uniform(mine.own), run0 = own_group * grid, me = uniform(run0 + mine.run);
    int64_t lo = run_start(line.total, grid, mine.run);
    const int64_t hi = run_start(line.total, grid, mine.run + 1);
    int req;
    int64_t base;
    line.find(a, lo, sh, req, base);

    // ---- the stream of staged tiles
    lds_u8 *ring = (lds_u8 *)lds;
    lds_u8 *ids = ring + STAGES * STAGE_BYTES + wave * (STAGES * 256);
    // Wave w takes rows 8w .. 8w + 7 of a tile, lane l row l / 8. What follows from the lane is worked
    // out where it is used: registers are short where 128 rows' sums are held
    auto own_lane = [&]() __attribute__((always_inline)) {
        int x = lane;
        asm volatile("" : "+v"(x));
        return x;
    };
    Cursor c;
    c.req = req;
    c.left = hi - lo;
    {
        const int places = tiles_of(a, uniform_len(a, req)).count + a.lead;
        c.g = (int)((lo - base) / places);
        c.enter(a, (int)((lo - base) % places), QT);
    }
    if (!c.more) return;
    // past the unit's query tiles, its key tiles, or into the next unit
    auto advance = [&]() __attribute__((always_inline)) {
        if (c.t < 0) {
            if (++c.t == 0) c.t = c.t0;
        } else if (++c.t == c.end) {
            c.left -= c.taken;
            c.more = c.left > 0;
            if (c.more) {
                if (++c.g == a.groups) {
                    c.g = 0;
                    ++c.req;
                }
                c.enter(a, 0, QT);
            }
        }
    };
    Source src{a.cache, 0, 0, 0, ~0ull};
    auto stage_address = [&](int slot) __attribute__((always_inline)) {
        return lds_address(ring + (uint32_t)slot % STAGES * STAGE_BYTES + wave * (SEGS * 1024));
    };
    auto chunk_of = [&](int x) __attribute__((always_inline)) { return ((x & 7) ^ swz(8 * wave + (x >> 3))) * 8; };
    // Item n is staged after step n, and the pieces of item n + LOOK go out between the matrix instructions that
    // follow, one at a time (ten loads in a row hold a wave up for 1100 cycles). The stage that they fill is
    // free: the value product is done with item n - 1, or, where it runs one step behind the score
    // product, with item n - 2. plan() takes the next item, aim() works out where a due one comes from. With
    // page ids by lane, step n takes those of item n + 2 LOOK, by way of LDS, and aims at item n + LOOK; by block,
    // it plans item n + LOOK + 1, whose id is there when the next step aims at it.
    constexpr int LOOK = S::FLOW ? 2 : 3;
    static_assert(LOOK <= QT + 1, "the items issued before the first step exist");
    // Of the unit that is staged: its row of the table, its last key; of the next tile: the wave's first key.
    typedef const __attribute__((address_space(4))) int32_t *constant_ptr;
    int64_t ids_row = 0;
    int last_key = 0, next_key = 0, of_req = 0;
    auto enter_block = [&]() __attribute__((always_inline)) {
        ids_row = c.req * a.t_row;
        last_key = max(0, c.len - 1);
        next_key = c.tiles.at(c.t0) * KT + 8 * wave;
        of_req = c.req;
    };
    auto plan_block = [&]() __attribute__((always_inline)) {
        BlockDue d{0, 0, 0};
        int page = 0;
        if (c.more) {
            bool same = false;                           // the next item is this unit's next tile of keys
            if (c.t >= 0) {                              // blocks past the end repeat the last one: masked
                const int k = min(next_key, last_key & ~7);
                page = page_of(a, k);
                d.row = k - page * a.page;
                d.kind = 2 + min(last_key - k, 7);
                next_key += KT;
                if (MASKED && c.t + 1 == c.tiles.head) next_key += c.tiles.skip * KT;
                same = c.t + 1 < c.end;
            } else {
                if (c.t == -QT) enter_block();
                d.row = (own_group + c.g) * S::MB + (c.t + QT) * KT + 8 * wave;
                d.kind = 1;
            }
            if (same) ++c.t;
            else advance();
        }
        // loaded in any case, so that nothing waits for it here
        d.id = ((constant_ptr)(uintptr_t)(a.table + uniform((int64_t)(ids_row + page))))[0];
        return d;
    };
    auto aim_block = [&](const BlockDue &d, int slot) __attribute__((always_inline)) {
        if (d.kind >= 2) {                               // ids outside the pool are clamped
            src.base = a.cache + (uint64_t)(uint32_t)min(max(d.id, 0), a.pages - 1) * (uint32_t)a.c_page +
                       (uint32_t)d.row * (uint32_t)a.c_row;
            // Rows past the request's last repeat it: what the pool holds behind it, which may not be finite, would
            // make the last tile go the way of add_values_carefully (64 requests x 33 keys x 64 heads: 16 us, and 28 with
            // NaN there).
            if (src.kind != d.kind) {
                const int x = own_lane();
                src.own = ((uint32_t)min(x >> 3, d.kind - 2) * (uint32_t)a.c_row + chunk_of(x)) * 2;
                src.kind = d.kind;
            }
        } else {                                         // rows past the last repeat it
            const int x = own_lane();
            const int r = min(d.row + (x >> 3), a.rows - 1), j = quotient(r, a.head_mul, a.head_shift), h = r - j * a.heads;
            src.base = a.q + (int64_t)of_req * a.tokens * a.q_row;
            src.own = ((uint32_t)j * (uint32_t)a.q_row + (uint32_t)h * (uint32_t)a.q_head + chunk_of(x)) * 2;
            src.kind = 1;
        }
        src.to = stage_address(slot);
    };
    // takes the next item; its page ids go to place `slot` of the ids' ring
    auto plan = [&](int slot) __attribute__((always_inline)) {
        Due d{0, c.req, 0};
        const int32_t *id = a.table;
        if (c.more) {
            const int kl = 8 * wave + (own_lane() >> 3);
            if (c.t < 0) {                               // rows past the last repeat it
                d.row = min((own_group + c.g) * S::MB + (c.t + QT) * KT + kl, a.rows - 1);
                d.kind = 1;
            } else {                                     // keys past the end repeat the last one: masked
                const int k = max(0, min(c.tiles.at(c.t) * KT + kl, c.len - 1));
                const int page = page_of(a, k);
                id = a.table + c.req * a.t_row + page;
                d.row = k - page * a.page;
                d.kind = 2;
            }
            advance();
        }
        load_lds_word(id, lds_address(ids + slot % STAGES * 256));
        return d;
    };
    auto aim = [&](const Due &d, int slot) __attribute__((always_inline)) {
        const int x = own_lane(), chunk = chunk_of(x);
        if (d.kind == 2) {                               // ids outside the pool are clamped
            const int id = *(__attribute__((address_space(3))) const int32_t *)(ids + slot % STAGES * 256 + x * 4);
            src.base = a.cache + (int64_t)min(max(id, 0), a.pages - 1) * a.c_page + (int64_t)d.row * a.c_row + chunk;
        } else {
            const int j = quotient(d.row, a.head_mul, a.head_shift), h = d.row - j * a.heads;
            src.base = a.q + ((int64_t)d.req * a.tokens + j) * a.q_row + h * a.q_head + chunk;
        }
        src.to = stage_address(slot);
    };
    int n = -1;
    Due due[LOOK];                                       // the next items to be issued
    BlockDue due_block;                                  // the next one
    if constexpr (BLOCKS) {
#pragma unroll
        for (int x = 0; x < LOOK; ++x) {
            aim_block(plan_block(), x);
            pieces_at<BLOCKS>(0, 1, src);
        }
        due_block = plan_block();
    } else {
        Due early[LOOK];
#pragma unroll
        for (int x = 0; x < LOOK; ++x) early[x] = plan(x);
        due[0] = plan(LOOK);
        aim(early[0], 0);                                // queries: their ids are not needed
        pieces_at<BLOCKS>(0, 1, src);
        wait_vmcnt<SEGS>();
#pragma unroll
        for (int x = 1; x < LOOK; ++x) {
            due[x] = plan(LOOK + x);
            aim(early[x], x);
            pieces_at<BLOCKS>(0, 1, src);
        }
    }
    lds_u8 *st = ring, *st_before = ring;
    auto step = [&]() __attribute__((always_inline)) {
        ++n;
        wait_vmcnt<PW *(LOOK - 1)>();
        lds_barrier();
        if constexpr (BLOCKS) {
            const bool there = due_block.kind != 0;
            if (there) aim_block(due_block, n + LOOK);
            due_block = plan_block();
            src.base = (const uint16_t *)uniform((int64_t)src.base);     // in scalar registers from here on
            src.to = uniform(src.to);
            src.lanes = lanes_if(there);
        } else {
            const bool there = due[0].kind != 0;
            const Due d = plan(n + 2 * LOOK);
            if (there) aim(due[0], n + LOOK);
            src.to = uniform(src.to);
            src.lanes = lanes_if(there);
#pragma unroll
            for (int x = 0; x + 1 < LOOK; ++x) due[x] = due[x + 1];
            due[LOOK - 1] = d;
        }
        st_before = st;
        st = ring + (uint32_t)n % STAGES * STAGE_BYTES;
    };
    // ---- fragment places within a stage. Score product: key row `row` of each subtile (subtiles
    // start at multiples of 16 rows: the same swizzle), K step k reads 16-byte chunk
    // k * KSTEP / 8 + grp of the row. The swizzle is an exclusive or of chunks, so the KA places of a
    // 128-byte piece differ by one too; they are worked out for each tile from one register.
    constexpr int KA = 64 / T::KSTEP;
    const int kbase = (row >> 3) * (SEGS * 1024) + (row & 7) * 128 + ((grp ^ swz(row)) << 4);
    auto place_of = [&](lds_u8 *from, int off) __attribute__((always_inline)) {
        int at = (int)(uintptr_t)from + off;
        asm volatile("" : "+v"(at));                     // one register, the rest is in the instruction
        return (lds_u8 *)(uintptr_t)(uint32_t)at;
    };
    auto find_keys = [&](lds_u8 *from, lds_u8 *(&at)[KA]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < KA; ++j) at[j] = place_of(from, kbase ^ (j * T::KSTEP * 2));
    };
    // Value product: 16-lane group reads keys kv + 0 .. 3 at dims dv + 0 .. 15; likewise for the dim
    // tile's place in its 128-byte piece and for the half of the key step
    constexpr int VA = 64 / T::DIMS;
    const int kv = T::place(0, grp) + ((lane & 15) >> 2);
    const int dv = (T::ROWS == 32 ? ((lane >> 4) & 1) * 16 : 0) + (lane & 3) * 4;
    const int vbase = (kv >> 3) * (SEGS * 1024) + (d0 >> 6) * 1024 + (kv & 7) * 128 + (((dv >> 3) ^ swz(kv)) << 4) + (dv & 4) * 2;
    auto find_values = [&](lds_u8 *from, lds_u8 *(&at)[VA][2]) __attribute__((always_inline)) {
        constexpr int HALF = T::place(4, 0);             // keys between the halves: 8 (another swizzle) or 16
#pragma unroll
        for (int j = 0; j < VA; ++j)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
                at[j][hh] = place_of(from, (vbase ^ (j * T::DIMS * 2) ^ (HALF == 8 ? hh * 16 : 0)) +
                                               hh * (HALF / 8) * (SEGS * 1024));
    };

    constexpr int NT = KT / T::ROWS;                     // key subtiles: 1 or 2
    constexpr int XS = T::NS / 8;                        // key steps of the value product
    constexpr int NK = S::KS * NT, NV = S::ND * XS;      // fragments of the score product, of the value product
    // places between matrix instructions where pieces go out: all of a step's, if a value product
    // follows each score product
    constexpr int ISSUES = S::FLOW ? NK : NK + NV;
    u32x4_t qf[S::KS], pf[XS];
    acc_t o[S::ND], s[NT], next[NT];
    float m, l;

    // S^T = K Q^T of the staged tile into `sum`, and beside it, in slices between the matrix
    // instructions, the softmax weights of the tile before from s. Fragments are read KAHEAD
    // instructions ahead; the scheduling barriers keep them there, and the compiler from spilling.
    // Weights are rounded to bf16 for the matrix product, whose operands are of one type (by 2^-8 relative
    // at most, independently of each other: an output's error grows from the 0.0017 of its own rounding
    // to 0.0022 at most in the listed cases); their sum l is of the unrounded ones.
    float mu = 0.0f;
    auto weight_pair = [&](int i) __attribute__((always_inline)) {
        const float x = __builtin_amdgcn_exp2f(fmaf(s[i / T::NO][i % T::NO], a.c, -mu));
        const float y = __builtin_amdgcn_exp2f(fmaf(s[(i + 1) / T::NO][(i + 1) % T::NO], a.c, -mu));
        l += x;
        l += y;
        pf[i / 8][i % 8 / 2] = pack_bf16(x, y);
    };
    auto all_weights = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::NS; i += 2) weight_pair(i);
    };
    auto scores = [&](acc_t (&sum)[NT], auto with_weights) __attribute__((always_inline)) {
        lds_u8 *at[KA];
        find_keys(st, at);
        auto key_frag = [&](int e) __attribute__((always_inline)) {
            const int k = e / NT, u = e % NT;
            return *(const lds_u32x4 *)(at[k % KA] + (u * T::ROWS / 8) * (SEGS * 1024) + (k / KA) * 1024);
        };
        u32x4_t kf[S::KAHEAD + 1];
#pragma unroll
        for (int e = 0; e < S::KAHEAD; ++e) kf[e] = key_frag(e);
        static_for<NK>([&](auto e) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (e + S::KAHEAD < NK) kf[(e + S::KAHEAD) % (S::KAHEAD + 1)] = key_frag(e + S::KAHEAD);
            __builtin_amdgcn_sched_barrier(0);
            sum[e % NT] = T::mfma(kf[e % (S::KAHEAD + 1)], qf[e / NT], e / NT ? sum[e % NT] : acc_t{0.0f});
            if constexpr (with_weights.value) {
#pragma unroll
                for (int i = 0; i < T::NS / 2; ++i)
                    if (i * NK / (T::NS / 2) == e) weight_pair(2 * i);
            }
            pieces_at<BLOCKS>(e, ISSUES, src);
        });
        in_vgpr(sum);
    };
    // O^T += V^T P^T. An A fragment of V^T is dim tile i, key step x; B register pairs hold keys
    // place(8x + j), j = 0 .. 7, and so does it. With care, of the values only the finite
    // ones, or `others`.
    auto add_values = [&](lds_u8 *tile, auto with_care, bool others) __attribute__((always_inline)) {
        lds_u8 *at[VA][2];
        find_values(tile, at);
        auto value = [&](int i, int x) __attribute__((always_inline)) {
            u32x4_t f;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                lds_u8 *p = at[i % VA][hh] + (i / VA) * 1024 + 2 * x * (SEGS * 1024);
                const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
                f[2 * hh] = v[0];
                f[2 * hh + 1] = v[1];
            }
            return f;
        };
        if constexpr (with_care.value) {
#pragma unroll
            for (int i = 0; i < S::ND; ++i) {
#pragma unroll
                for (int x = 0; x < XS; ++x) {
                    __builtin_amdgcn_sched_barrier(0);
                    o[i] = T::mfma(pick_values(value(i, x), others), pf[x], o[i]);
                }
                if constexpr (!S::FLOW) {
#pragma unroll
                    for (int x = 0; x < XS; ++x)
                        if (!others) pieces_at<BLOCKS>(NK + i * XS + x, ISSUES, src);
                }
            }
            return;
        }
        u32x4_t vf[S::VAHEAD + 1];
#pragma unroll
        for (int e = 0; e < S::VAHEAD; ++e) vf[e] = value(e / XS, e % XS);
        static_for<NV>([&](auto e) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
            constexpr int then = e + S::VAHEAD;
            if constexpr (then < NV) vf[then % (S::VAHEAD + 1)] = value(then / XS, then % XS);
            __builtin_amdgcn_sched_barrier(0);
            o[e / XS] = T::mfma(vf[e % (S::VAHEAD + 1)], pf[e % XS], o[e / XS]);
            if constexpr (!S::FLOW) pieces_at<BLOCKS>(NK + e, ISSUES, src);
        });
    };
    // The same for tile t with scores that are not finite, of which some rows see less than others. A
    // latent that is not finite must not reach rows that do not see it, whose weight 0 times it is NaN;
    // for rows that see it that product is right (its score is -inf, weight 0, or they are NaN
    // throughout): they get +inf and -inf, each a product of the largest number, the others 0. One
    // loop, not three copies: the 128-row shape has no registers to spare.
    auto add_values_carefully = [&](lds_u8 *tile, auto sees) __attribute__((always_inline)) {
#pragma clang loop unroll(disable)
        for (int pass = 0; pass < 3; ++pass) {
            if (pass) {
                const uint32_t sign = pass == 1 ? 0u : 0x80008000u;
#pragma unroll
                for (int i = 0; i < T::NS; i += 2) pf[i / 8][i % 8 / 2] = seen_pair(sees(i), sees(i + 1)) ^ sign;
            }
            add_values(tile, std::true_type(), pass > 0);
        }
        in_acc(o);
    };

    bool leading = true;                                 // the run's first unit
    while (lo < hi) {
        const int len = uniform_len(a, req);
        const Tiles span = tiles_of(a, len);
        const int tiles = span.count;
        const int places = tiles + a.lead, first = (int)((lo - base) % places);
        const int g = own_group + (int)((lo - base) / places), taken = (int)min((int64_t)(places - first), hi - lo);
        const int t0 = max(0, first - a.lead), t1 = first + taken - a.lead;
        if (t1 <= 0) break;                                      // see Cursor
        // keys this lane's row sees: it is row (token, head) of the request; rows past the last repeat it
        const int limit = max(0, len - a.tokens + 1 + min(g * S::MB + wr * T::ROWS + row, a.rows - 1) / a.heads);
        int whole = max(0, len - a.tokens + 1) / KT;             // tiles before this: all rows see all of them
        int some = 0;                                            // (with a window: those from this one on)
        if constexpr (MASKED) {
            // The row's words, and where its window begins, come to LDS: the masks of a unit's few tiles that are
            // not seen whole are made from them where they are needed, and no registers are held for them.
            const int j = min(g * S::MB + wr * T::ROWS + row, a.rows - 1) / a.heads;
            uint32_t *mine = masks + wave * T::ROWS * (MOST_WORDS + 1) + row;
            int begin = 0;
            if (a.tree) {
                whole = max(0, len - a.tokens) / KT;
                const int32_t *words = a.tree + req * a.tree_row + (int64_t)j * a.words;
                for (int w = grp; w < a.words; w += 64 / T::ROWS) mine[w * T::ROWS] = words[w];
                if (a.window) begin = len - a.tokens + 1 - a.window + min(max(a.depth[req * a.depth_row + j], 0), a.tokens - 1);
            } else if (a.window) {
                begin = limit - a.window;
            }
            if (grp == 0) mine[MOST_WORDS * T::ROWS] = max(0, begin);
            if (a.window) some = (max(0, len - a.window) + KT - 1) / KT;
        }
        // of tile t of the line, the keys that this lane's row sees: bit b for key b of it
        auto seen_keys = [&](int t) __attribute__((always_inline)) -> uint32_t {
            const int k0 = span.at(t) * KT;
            if constexpr (!MASKED) {
                return keys_below(limit, k0);
            } else {
                const uint32_t *mine = masks + wave * T::ROWS * (MOST_WORDS + 1) + row;
                const int own = len - a.tokens;                  // the first new token
                uint32_t seen = keys_below(a.tree ? own : limit, k0);
                if (a.window) seen &= keys_below(a.sinks, k0) | ~keys_below((int)mine[MOST_WORDS * T::ROWS], k0);
                if (a.tree && k0 + KT > own) {
                    const int first = k0 - own, w = first >> 5;  // w of -1: the tile begins in the context
                    const uint32_t low = w >= 0 && w < a.words ? mine[w * T::ROWS] : 0u;
                    const uint32_t high = w + 1 < a.words ? mine[(w + 1) * T::ROWS] : 0u;
                    seen |= (uint32_t)(((uint64_t)high << 32 | low) >> (first & 31)) & keys_below(len, k0);
                }
                return seen;
            }
        };

        for (int qi = 0; qi < QT; ++qi) {
            step();
            pieces_at<BLOCKS>(0, 1, src);
            if (qi == wr * T::ROWS / KT) {
                lds_u8 *at[KA];
                find_keys(st + wr * T::ROWS % KT / 8 * (SEGS * 1024), at);
#pragma unroll
                for (int k = 0; k < S::KS; ++k) qf[k] = *(const lds_u32x4 *)(at[k % KA] + (k / KA) * 1024);
            }
        }
        float zero = 0.0f;
        asm volatile("" : "+v"(zero));                   // here: a vector of zeros kept for it would go to scratch memory
#pragma unroll
        for (int i = 0; i < S::ND; ++i)
#pragma unroll
            for (int j = 0; j < T::NO; ++j) o[i][j] = zero;
        in_acc(o);
        m = -INFINITY;
        l = 0.0f;

        // Tile t's scores are in s. What the next step needs to know of them: the row's largest, and
        // whether a masked tile holds one that is not finite.
        float top;
        bool odd, grow;
        auto inspect = [&](int t) __attribute__((always_inline)) {
            odd = false;
            const int at = MASKED ? span.at(t) : t;
            if (at >= whole || (MASKED && at < some)) {
                const uint32_t keys = MASKED ? seen_keys(t) >> T::place(0, grp) : 0u;
#pragma unroll
                for (int i = 0; i < T::NS; ++i) {
                    const float x = s[i / T::NO][i % T::NO];
                    const bool seen = MASKED ? keys >> T::place(i, 0) & 1 : t * KT + T::place(i, grp) < limit;
                    odd |= !finite_f32(x);               // so is the key's row, or a query
                    s[i / T::NO][i % T::NO] = seen ? x : -INFINITY;
                }
                odd = __any(odd);
            }
            top = s[0][0];
#pragma unroll
            for (int i = 1; i < T::NS; ++i) top = fmaxf(top, s[i / T::NO][i % T::NO]);
            top = row_max<T>(top) * a.c;
            grow = __any(top > m + kSlack);
            mu = m == -INFINITY ? 0.0f : m;
        };
        // moves the row's reference maximum to what the scores need
        auto rescale = [&](bool first) __attribute__((always_inline)) {
            const float up = fmaxf(m, top);
            const float alpha = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            mu = m == -INFINITY ? 0.0f : m;
            l *= alpha;
            grow = false;
            if (first) return;                           // the sums are 0 yet
#pragma unroll
            for (int i = 0; i < S::ND; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                o[i] *= alpha;
                in_acc(o);
            }
        };
        auto sees_of = [&](int t) __attribute__((always_inline)) {
            const uint32_t keys = MASKED ? seen_keys(t) : 0u;
            const int left = limit - t * KT;
            return [=](int i) { return MASKED ? keys >> T::place(i, grp) & 1 : T::place(i, grp) < left; };
        };
        // The inner loops have no branch that touches the output sums: one that did would move all
        // of them between register files in every iteration. A reference maximum that moves and a
        // non-finite score in a masked tile leave them.
        bool scored = false;
        if constexpr (S::FLOW) {
            for (int t = t0;;) {
                if (!scored) {
                    step();
                    scores(s, std::false_type());
                    inspect(t);
                    scored = true;
                }
                while (!odd && !grow && t + 1 < t1) {
                    step();
                    scores(next, std::true_type());
                    add_values(st_before, std::false_type(), false);
#pragma unroll
                    for (int u = 0; u < NT; ++u) s[u] = next[u];
                    inspect(++t);
                }
                if (grow) {
                    rescale(t == t0);
                    if (!odd && t + 1 < t1) continue;
                }
                all_weights();
                if (odd) add_values_carefully(st, sees_of(t));     // rare
                else add_values(st, std::false_type(), false);
                in_acc(o);
                if (++t == t1) break;
                scored = false;
            }
        } else {
            for (int t = t0;;) {
                do {
                    if (!scored) {
                        step();
                        scores(s, std::false_type());
                        inspect(t);
                    }
                    scored = false;
                    if (odd || grow) break;
                    all_weights();
                    add_values(st, std::false_type(), false);
                } while (++t < t1);
                if (t >= t1) break;
                if (grow) rescale(t == t0);
                if (!odd) {
                    scored = true;
                    continue;
                }
                all_weights();
                add_values_carefully(st, sees_of(t));      // rare
                if (++t >= t1) break;
            }
        }
        l = row_sum<T>(l);

        const int r = g * S::MB + wr * T::ROWS + T::row(own_lane()), rc = min(r, a.rows - 1);
        const int j = rc / a.heads, h = rc - j * a.heads;
        const int64_t qr = (int64_t)req * a.tokens + j;
        const bool uncut = t0 == 0 && t1 == tiles;
        if (t0 == 0 && tid == 0)
            a.cuts[(int64_t)req * a.all_groups + g] = make_int2(
                2 * me + (leading ? 0 : 1), uncut ? me : run0 + run_of(line.total, grid, lo - first + places - 1));
        if (uncut) {
            if (r < a.rows) {                            // the lanes of a row are in this together
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;  // no key: zeros
                uint16_t *op = a.out + qr * a.o_row + h * a.o_head + d0;
                if (a.lse && grp == 0 && wave / WR == 0) a.lse[qr * a.heads + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;
#pragma unroll
                for (int i = 0; i < S::ND; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    acc_t y[1] = {o[i]};                 // out of the accumulation registers tile by tile
                    in_vgpr(y);
                    u32x2_t v[S::NO4];
#pragma unroll
                    for (int x = 0; x < S::NO4; ++x)
                        v[x] = u32x2_t{pack_bf16(y[0][4 * x] * inv, y[0][4 * x + 1] * inv),
                                       pack_bf16(y[0][4 * x + 2] * inv, y[0][4 * x + 3] * inv)};
                    if constexpr (T::ROWS == 32) {       // the two lanes of a row trade halves: 16-byte stores
#pragma unroll
                        for (int x = 0; x < S::NO4; x += 2) {
                            const auto p = __builtin_amdgcn_permlane32_swap(v[x][0], v[x + 1][0], false, false);
                            const auto q = __builtin_amdgcn_permlane32_swap(v[x][1], v[x + 1][1], false, false);
                            *reinterpret_cast<u32x4_t *>(op + i * T::DIMS + 8 * (x + grp)) = u32x4_t{p[0], q[0], p[1], q[1]};
                        }
                    } else {
                        *reinterpret_cast<u32x2_t *>(op + i * T::DIMS + T::place(0, grp)) = v[0];
                    }
                }
            }
        } else if (r < a.rows) {                         // no partials of rows that repeat the last
            float *part = a.work + (2 * (int64_t)me + (leading ? 0 : 1)) * part_floats<S::MB>();
            f32x4_t *ps = reinterpret_cast<f32x4_t *>(part) + wave * (S::ND * S::NO4 * 64) + lane;
#pragma unroll
            for (int i = 0; i < S::ND; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                acc_t y[1] = {o[i]};
                in_vgpr(y);
#pragma unroll
                for (int x = 0; x < S::NO4; ++x)
                    ps[(i * S::NO4 + x) * 64] = f32x4_t{y[0][4 * x], y[0][4 * x + 1], y[0][4 * x + 2], y[0][4 * x + 3]};
            }
            if (grp == 0 && wave / WR == 0) {
                part[(int64_t)S::MB * L + wr * T::ROWS + row] = m;
                part[(int64_t)S::MB * (L + 1) + wr * T::ROWS + row] = l;
            }
        }
        leading = false;
        lo += taken;
        if (lo == base + (int64_t)places * a.groups) {
            base = lo;
            ++req;
        }
    }
}

// Workgroups that can have tiles: at most one a CU, and no more than the line can have of them (the places of no work
// are not counted).
int takers(const DecodeArgs &a, int most) {
    const int64_t tiles = std::max<int64_t>(1, ((int64_t)a.max_pages * a.page + KT - 1) / KT);
    return (int)std::min<int64_t>(most, (int64_t)a.batch * a.all_groups * tiles);
}

// Joins the partial sums of the units that were cut between workgroups. A wave's lanes are PL groups:
// each takes the same 64 / PL float4 of a unit's sums, of every PL-th partial. WP waves share a
// unit's partials further and meet in LDS; each lane asks for 4 partials at once. With few units the
// latency of these loads bounds it (256 partials of 32 rows, 17 MB: 7.0 us, of which the launch and the
// look-up of the cuts are most; 8.5 with whole waves on a partial), with many their bytes
// (350 partials of 128 rows, 92 MB: 22 us, 4.7 TB/s; 8 of them at once gain nothing there and cost small joins 1
// us).
template <typename T, int WR, int WD, int WP, int PL>
__global__ __launch_bounds__(WP > 4 ? WP * 64 : 256) void latent_join_kernel(DecodeArgs a) {
    typedef Shape<T, WR, WD> S;
    constexpr int LANES = 64 / PL, TURNS = WP * PL;      // float4s a wave; partials taken side by side
    constexpr int PER = S::MB * L / 4 / LANES;           // waves' shares of a unit
    constexpr int QUADS = WP > 4 ? 1 : 4 / WP;           // of them, a workgroup's
    static_assert(PER % QUADS == 0, "whole workgroups a unit");
    __shared__ f32x4_t so[WP > 1 ? QUADS * WP : 1][64];
    __shared__ float sm[WP > 1 ? QUADS * WP : 1][64], sl[WP > 1 ? QUADS * WP : 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int unit = blockIdx.x / (PER / QUADS);
    const int at = (blockIdx.x % (PER / QUADS) * QUADS + wave / WP) * LANES + lane % LANES;     // float4 of the unit
    const int turn = wave % WP * PL + lane / LANES;
    const int2 cut = a.cuts[unit];
    const int b0 = cut.x >> 1, pieces = cut.y - b0 + 1;
    if (pieces <= 1) return;
    const int req = unit / a.all_groups, g = unit % a.all_groups;

    // at = (wave of the writer, 4-register group, its lane) in the partial's order; see the writer
    constexpr int PERW = S::ND * S::NO4;
    const int wl = at % 64, ww = at / 64 / PERW, rest = at / 64 % PERW, i = rest / S::NO4, x = rest % S::NO4;
    const int row = (ww % WR) * T::ROWS + T::row(wl);
    float m = -INFINITY, l = 0.0f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    auto merge = [&](float pm, float pl, f32x4_t po) {
        const float n = fmaxf(m, pm);
        const float ca = m == n ? 1.0f : __builtin_amdgcn_exp2f(m - n);
        const float cb = pm == n ? 1.0f : __builtin_amdgcn_exp2f(pm - n);
        m = n;
        l = l * ca + pl * cb;
        o = o * ca + po * cb;
    };
    // partial j: the first workgroup's is its run's first or last, the others' their runs' first
    auto partial = [&](int j) {
        return a.work + (j == 0 ? (int64_t)cut.x : 2 * (int64_t)(b0 + j)) * part_floats<S::MB>();
    };
    const int r = g * S::MB + row;
    for (int j = r < a.rows ? turn : pieces; j < pieces; j += 4 * TURNS) {
        float pm[4], pl[4];
        f32x4_t po[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (j + u * TURNS >= pieces) break;
            const float *part = partial(j + u * TURNS);
            pm[u] = part[(int64_t)S::MB * L + row];
            pl[u] = part[(int64_t)S::MB * (L + 1) + row];
            po[u] = reinterpret_cast<const f32x4_t *>(part)[at];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u * TURNS < pieces) merge(pm[u], pl[u], po[u]);
    }
    if constexpr (PL > 1) {                              // the lanes' groups, in order: the first's lanes end with all
        for (int u = 1; u < min(PL, pieces); ++u) {
            const int from = u * LANES + lane % LANES;
            const float pm = __shfl(m, from), pl = __shfl(l, from);
            const f32x4_t po = {__shfl(o[0], from), __shfl(o[1], from), __shfl(o[2], from), __shfl(o[3], from)};
            if (lane < LANES) merge(pm, pl, po);
        }
    }
    if constexpr (WP > 1) {
        so[wave][lane] = o;
        sm[wave][lane] = m;
        sl[wave][lane] = l;
        __syncthreads();
        if (turn) return;
        for (int u = 1; u < min(WP, (pieces + PL - 1) / PL); ++u) merge(sm[wave + u][lane], sl[wave + u][lane], so[wave + u][lane]);
    } else if (turn) {
        return;
    }
    if (r >= a.rows) return;
    const int64_t qr = (int64_t)req * a.tokens + r / a.heads;
    const int h = r % a.heads;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const u32x2_t y = {pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    const int dim = (ww / WR) * (L / WD) + i * T::DIMS + T::place(4 * x, T::grp(wl));
    *reinterpret_cast<u32x2_t *>(a.out + qr * a.o_row + h * a.o_head + dim) = y;
    if (a.lse && T::grp(wl) == 0 && ww / WR == 0 && rest == 0)
        a.lse[qr * a.heads + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int WR, int WD, int WP, int PL>
hipError_t launch_join(const DecodeArgs &a, hipStream_t stream) {
    constexpr int PER = Shape<T, WR, WD>::MB * L / 4 / (64 / PL), QUADS = WP > 4 ? 1 : 4 / WP;
    const unsigned blocks = (unsigned)((int64_t)a.batch * a.all_groups * (PER / QUADS));
    hipLaunchKernelGGL((latent_join_kernel<T, WR, WD, WP, PL>), dim3(blocks), dim3(WP > 4 ? WP * 64 : 256), 0, stream, a);
    return hipGetLastError();
}

template <typename T, int WR, int WD, typename A>
hipError_t launch_shape(A a, bool blocks, hipStream_t stream) {
    constexpr bool MASKED = std::is_same_v<A, MaskedArgs>;
    // see shared_run: as many on each XCD
    const unsigned workgroups = a.side > 1 ? (unsigned)((a.grid + 7) / 8 * 8) : (unsigned)a.grid;
    a.cuts = reinterpret_cast<int2 *>(a.work + 2 * a.grid * part_floats<Shape<T, WR, WD>::MB>());
    bool launched = false;
    if constexpr (Shape<T, WR, WD>::MB > 16) {
        if (blocks) {
            hipLaunchKernelGGL((latent_decode_kernel<T, WR, WD, MASKED, true>), dim3(workgroups), dim3(THREADS), 0, stream, a);
            launched = true;
        }
    }
    if (!launched)
        hipLaunchKernelGGL((latent_decode_kernel<T, WR, WD, MASKED, false>), dim3(workgroups), dim3(THREADS), 0, stream, a);
    hipError_t err = hipGetLastError();
    // one workgroup takes every run whole: nothing to join
    if (err != hipSuccess || a.grid == 1) return err;
    // takers of a unit's partials: about as many as it has on average, unless that makes more waves
    // than the chip holds at once (8 requests x 4000 keys x 128 heads 47 us with 16, 44 with 4)
    const int64_t units = (int64_t)a.batch * a.all_groups, waves = units * (Shape<T, WR, WD>::MB * L / 4 / 64), room = 16384;
    const int pieces = takers(a, a.grid);
    if (pieces > 64 * units && waves * 64 <= room) return launch_join<T, WR, WD, 16, 4>(a, stream);
    if (pieces > 16 * units && waves * 16 <= room) return launch_join<T, WR, WD, 16, 1>(a, stream);
    if (pieces > 4 * units) return launch_join<T, WR, WD, 4, 1>(a, stream);
    return launch_join<T, WR, WD, 1, 1>(a, stream);
}

// Rows a workgroup for a request of `rows` query rows: the smallest shape that holds them, since each
// wave computes all rows of its shape (64 requests x 3000 keys, in us: 16 rows 42 in the 16-row shape,
// 48 in the 32-row one, 86 in the 128-row one; 32 rows 49, 49, 88; 64 rows 64 and 90).
int block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

}  // namespace

int64_t latent_decode_workspace_bytes(int64_t batch, int64_t tokens, int64_t heads, int cus) {
    const int64_t rows = tokens * heads;
    if (batch == 0 || rows == 0) return 0;
    const int mb = block_rows(rows);
    return 2 * (int64_t)cus * mb * (L + 2) * (int64_t)sizeof(float) + batch * ((rows + mb - 1) / mb) * (int64_t)sizeof(int2);
}

// Threads of the join kernel where one wave takes all of a unit's partials: one for each 4 numbers of an
// output. (Where more waves share them the units are fewer than the CUs, and far from any limit.)
int64_t latent_decode_join_threads(int64_t batch, int64_t tokens, int64_t heads) {
    const int64_t rows = tokens * heads;
    const int mb = block_rows(rows);
    return batch * ((rows + mb - 1) / mb) * mb * (L / 4);
}

static DecodeArgs decode_args(const skinny_latent_decode_args &p, int cus) {
    DecodeArgs a;
    a.q = static_cast<const uint16_t *>(p.q);
    a.q_row = p.q_row_stride;
    a.q_head = p.q_head_stride;
    a.cache = static_cast<const uint16_t *>(p.cache);
    a.c_page = p.cache_page_stride;
    a.c_row = p.cache_row_stride;
    a.table = p.table;
    a.t_row = p.table_stride;
    a.lens = p.lens;
    a.out = static_cast<uint16_t *>(p.out);
    a.o_row = p.out_row_stride;
    a.o_head = p.out_head_stride;
    a.lse = p.lse;
    a.work = static_cast<float *>(p.workspace);
    a.batch = (int)p.batch;
    a.tokens = (int)p.tokens;
    a.heads = (int)p.heads;
    a.pages = (int)p.pages;
    a.page = (int)p.page;
    a.max_pages = (int)p.max_pages;
    a.rows = a.tokens * a.heads;
    reciprocal(a.page, a.page_mul, a.page_shift);
    reciprocal(a.heads, a.head_mul, a.head_shift);
    const int mb = block_rows(a.rows);
    a.all_groups = (a.rows + mb - 1) / mb;
    a.c = p.scale * kLog2e;
    // side by side where that leaves few CUs idle: at most an eighth (29 groups 24 of 256; see shared_run)
    const int most = takers(a, cus);
    const bool shared = a.all_groups <= most && most % a.all_groups * 8 <= most;
    a.side = shared ? a.all_groups : 1;
    a.groups = a.all_groups / a.side;
    // with 0, 3, 6 and 8 places in us: 32 requests x 192 rows x 4096 keys 87, 84, 84, 84, 8 x 1024 x 8000 145, 142, 138,
    // 138, 96 x 128 x 4000 126, 122, 119, 120; with 64 rows and 0, 2, 4, 6: 4 windows of 1000 15.2, 13.6, 13.1, 13.8
    a.lead = p.batch * a.groups > 1 ? (mb == 128 ? 6 : mb == 64 ? 4 : 2) : 0;
    // No more workgroups than the line can have places, those of no work among them: with one for each tile alone, short
    // lines left some workgroups with nothing and others with two tiles (2 requests x 40 keys x 64 heads 12.9 us, 10.2 so;
    // 3 x 87 x 32 heads 9.9, 8.9).
    a.grid = (int)std::min<int64_t>(cus, most + (int64_t)a.batch * a.all_groups * a.lead);
    return a;
}

template <typename A>
static hipError_t launch(const A &a, hipStream_t stream) {
    // a page's bytes, and a lane's from its request's first query, fit 31 bits
    const int64_t most = (int64_t)1 << 29;
    const bool blocks = a.page % 8 == 0 && a.c_row < most / a.page && (a.pages <= 1 || a.c_page < most) &&
                        a.q_row < most / a.tokens && a.q_head < most / a.heads;
    switch (block_rows(a.rows)) {
        case 16: return launch_shape<Tile16, 1, 4>(a, blocks, stream);
        case 32: return launch_shape<Tile16, 2, 2>(a, blocks, stream);
        case 64: return launch_shape<Tile16, 4, 1>(a, blocks, stream);
        default: return launch_shape<Tile32, 4, 1>(a, blocks, stream);
    }
}

hipError_t launch_latent_decode(const skinny_latent_decode_args &p, int cus, hipStream_t stream) {
    return launch(decode_args(p, cus), stream);
}

hipError_t launch_latent_masked_decode(const skinny_latent_decode_args &p, const skinny_latent_mask &m, int cus,
                                       hipStream_t stream) {
    // a window as long as a request can be hides nothing
    const int64_t window = m.window < p.max_pages * p.page ? m.window : 0;
    if (!m.tree && !window) return launch_latent_decode(p, cus, stream);
    MaskedArgs a;
    static_cast<DecodeArgs &>(a) = decode_args(p, cus);
    a.tree = m.tree;
    a.depth = m.depth;
    a.tree_row = m.tree_stride;
    a.depth_row = m.depth_stride;
    a.words = (int)((p.tokens + 31) / 32);
    a.window = (int)window;                              // fewer than 2^30
    a.sinks = window ? (int)std::min<int64_t>(m.sinks, INT_MAX / 2) : 0;
    return launch(a, stream);
}

}  // namespace skinny
