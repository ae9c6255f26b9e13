// latent_weights.hip -- what each cached key's softmax weights add up to over the newest tokens' rows.
//
// For request i with n = lens[i] cached rows c_k and R = tokens * heads query rows, of which row (j, h)
// sees keys k <= n - tokens + j:
//     weights[i, k] += sum over the rows that see k of exp(scale q . c_k - lse_row).
//
// What bounds it: up to some 300 rows a request the cache's bytes (1152 a key, at 2 * 576 operations a row),
// beyond them the matrix cores. A wave holds a tile of 32 keys in registers (144 of them, so that two
// waves fit a SIMD), and the request's query rows pass by in tiles of 32: every key is read once
// whatever the rows, a key is a lane's in S = Q K^T, its sum stays in that lane's registers, and one wave adds
// it to the weights: no partial sums, no order that could change.
//   * The tiles of all requests are one line, cut into equal runs, one a workgroup of 8 waves; a
//     run goes by chunks of up to 8 tiles of one request.
//   * Everything comes through one ring of LDS stages of 36 KB: a chunk's key tiles, each taken
//     out by its wave, then the query tiles, which all waves compute on. Two stages are in flight.
// Measured: 64 requests of 4000 .. 12000 keys x 16 rows 107 us (614 MB read, 5.8 TB/s), 2 of about 16000 x
// 1024 rows 47 us in a row of calls (34.6 GFLOP at least, 735 TFLOP/s; 55 alone, matrix cores busy 25% of the
// cycles): 1000 tiles of keys over 256 workgroups are runs of 4, each with the 32 query tiles behind it, and a
// step's barrier and addresses are not hidden by two waves a SIMD that a barrier keeps in step. Addresses of
// whole blocks by the scalar unit, as in latent_decode.hip, are slower here (137 and 56 us), and so are 16 x 16
// matrix instructions (58).
#include <algorithm>
#include <type_traits>

#include "latent_line.hpp"

namespace skinny {
namespace {

using namespace latent;
typedef Tile32 T;

constexpr int DIM = 576;                     // numbers of a cached row
constexpr int KT = 32;                       // keys, or query rows, a tile
constexpr int SEGS = DIM * 2 / 128;          // 128-byte pieces of a row
constexpr int STAGES = 4, LOOK = 2;          // stages in LDS, and of them in flight
constexpr int STAGE_BYTES = KT * DIM * 2;
constexpr int WAVES = 8, THREADS = WAVES * 64;
constexpr int PIECES = (SEGS + 1) / 2;       // two waves share 8 rows of a stage: 5 pieces and 4 (and one that loads nothing)
constexpr int PW = PIECES + 1;               // loads a wave issues a stage: a word and pieces
constexpr int SLOTS = 8, SLOT_BYTES = 128;   // 32 words each of so many stages: page ids of 8 rows, or 32 rows' log sums
constexpr int KS = DIM / T::KSTEP;           // K steps
constexpr float LEAD = 0.42f;                // what a query tile takes, in times of a tile of keys (30 requests of 2000 ..
                                             // 4000 keys x 512 rows 72 us, 90 with none, 82 with twice as much)
constexpr int AHEAD = 3;                     // fragments read ahead (2 and 4 take as long)

struct WeightArgs {
    const uint16_t *q;
    int64_t q_row, q_head;                   // strides in elements
    const uint16_t *cache;
    int64_t c_page, c_row;
    const int32_t *table;
    int64_t t_row;
    const int32_t *lens;
    const float *lse;
    float *weights;
    int64_t w_row;
    int batch, tokens, heads, pages, page, max_pages, columns;
    int rows, qtiles, groups, grid;          // rows a request, their tiles; groups: 1, see Line
    int lead;                                // see request_tiles
    uint32_t page_mul, head_mul;             // see quotient
    int page_shift, head_shift;
    float c;                                 // scale * log2(e)
};

__device__ __forceinline__ int clamp_len(const WeightArgs &a, int n) { return min(max(n, 0), a.max_pages * a.page); }
__device__ __forceinline__ int uniform_len(const WeightArgs &a, int i) {     // see latent_decode.hip
    typedef const __attribute__((address_space(4))) int32_t *constant_ptr;
    return clamp_len(a, ((constant_ptr)(uintptr_t)a.lens)[i]);
}
// tiles of the keys that have a column
__device__ __forceinline__ int tiles_of(const WeightArgs &a, int len) { return (min(len, a.columns) + KT - 1) / KT; }
// What a request takes of the line: its tiles, and ahead of them `lead` places of no work, so that a run that
// ends one request and begins the next, which makes two chunks of it, is given less of them.
__device__ __forceinline__ int request_tiles(const WeightArgs &a, int i) {
    const int tiles = tiles_of(a, clamp_len(a, a.lens[i]));
    return tiles ? tiles + a.lead : 0;
}

// Lane l's 4 bytes at src, of the lower 32 lanes, to lds + 4 l (called with all lanes active; see load_lds_word).
__device__ __forceinline__ void load_lds_words(const void *src, int lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_hi, 0\n\tglobal_load_lds_dword %1, off\n\ts_mov_b32 exec_hi, -1"
                 :: "s"(lds), "v"(src) : "memory");
}

// The items of a run, in order: for each chunk its key tiles, then all query tiles of its request.
struct Chunks {
    int req, len, tiles;                     // request
    int t, keys, x;                          // chunk: its first tile, its number of tiles, next item
    int64_t left;                            // tiles of the run from this chunk on
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void enter(const WeightArgs &a) {     // finds the chunk from tile t on
        if (t < 0) {
            left += t;
            t = 0;
        }
        while (left > 0 && t >= tiles) {
            if (++req == a.batch) {                      // lengths that change under the call: the run ends here
                left = 0;
                break;
            }
            len = uniform_len(a, req);
            tiles = tiles_of(a, len);
            t = 0;
            if (tiles) left -= a.lead;
        }
        keys = (int)min((int64_t)min(WAVES, tiles - t), left);
        x = 0;
    }
    __device__ __forceinline__ void next(const WeightArgs &a) {
        if (++x == keys + a.qtiles) {
            left -= keys;
            t += keys;
            enter(a);
        }
    }
};
struct Due {
    int row, req, kind;                      // kind 0: none, 1: queries, 2: keys
};

__global__ __launch_bounds__(THREADS) void latent_key_weights_kernel(WeightArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE_BYTES + WAVES * SLOTS * SLOT_BYTES];
    __shared__ int64_t sh[WAVES + 2];
    __shared__ float halves[WAVES / 2][KT];
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    const int row = T::row(lane), grp = T::grp(lane);

    Line<WeightArgs, THREADS> line;
    line.measure(a, (int64_t)a.batch * ((a.columns + KT - 1) / KT + a.lead), sh);
    const int grid = (int)min((int64_t)a.grid, line.total);
    if ((int)blockIdx.x >= grid) return;
    const int64_t lo = run_start(line.total, grid, blockIdx.x), hi = run_start(line.total, grid, blockIdx.x + 1);
    Chunks c, todo;
    int64_t base;
    line.find(a, lo, sh, c.req, base);
    c.len = uniform_len(a, c.req);
    c.tiles = tiles_of(a, c.len);
    c.t = (int)(lo - base) - a.lead;
    c.left = hi - lo;
    c.enter(a);
    todo = c;                                            // c: what is staged next, todo: what is worked on next

    lds_u8 *ring = (lds_u8 *)lds;
    lds_u8 *words = ring + STAGES * STAGE_BYTES + wave * (SLOTS * SLOT_BYTES);
    // staging: waves 2b and 2b + 1 take rows 8b .. 8b + 7 of a tile, lane l row l / 8; the first of them
    // the row's pieces 0 .. 4, the second 5 .. 8
    const int first_own = 8 * (wave >> 1), own = first_own + (lane >> 3);
    const int chunk = ((lane & 7) ^ swz(own)) * 8 + (wave & 1) * (PIECES * 64);
    auto plan = [&](int slot) __attribute__((always_inline)) {
        Due d{0, c.req, 0};
        const void *word = a.table;
        if (c.more()) {
            if (c.x < c.keys) {                          // keys past the end repeat the last one
                const int first = (c.t + c.x) * KT, k = min(first + first_own + (lane & 7), c.len - 1);
                word = a.table + c.req * a.t_row + page_of(a, k);        // lane l: row l of the wave's
                d.row = min(first + own, c.len - 1);
                d.kind = 2;
            } else {                                     // rows past the last repeat it
                const int first = (c.x - c.keys) * KT;
                word = a.lse + (int64_t)c.req * a.rows + min(first + (lane & 31), a.rows - 1);
                d.row = min(first + own, a.rows - 1);
                d.kind = 1;
            }
            c.next(a);
        }
        load_lds_words(word, lds_address(words + slot % SLOTS * SLOT_BYTES));
        return d;
    };
    const uint16_t *from = a.cache;
    int to = 0;
    uint64_t live = 0;                                   // there is an item to stage: all lanes, or none
    auto aim = [&](const Due &d, int slot) __attribute__((always_inline)) {
        if (d.kind == 2) {                               // ids outside the pool are clamped
            typedef __attribute__((address_space(3))) const int32_t lds_i32;
            const int id = *(lds_i32 *)(words + slot % SLOTS * SLOT_BYTES + (lane >> 3) * 4);
            const int place = d.row - page_of(a, d.row) * a.page;
            from = a.cache + (int64_t)min(max(id, 0), a.pages - 1) * a.c_page + (int64_t)place * a.c_row + chunk;
        } else if (d.kind == 1) {
            const int j = quotient(d.row, a.head_mul, a.head_shift), h = d.row - j * a.heads;
            from = a.q + ((int64_t)d.req * a.tokens + j) * a.q_row + h * a.q_head + chunk;
        }
        to = lds_address(ring + slot % STAGES * STAGE_BYTES + (wave >> 1) * (SEGS * 1024) + (wave & 1) * (PIECES * 1024));
        live = lanes_if(d.kind != 0);
    };
    // the item's pieces that go out with group `at` of `of` (both known when compiled)
    auto pieces_at = [&](int at, int of) __attribute__((always_inline)) {
        if (0 * of / PIECES == at) load_lds_piece_in<0>(live, from, to);
        if (1 * of / PIECES == at) load_lds_piece_in<1>(live, from, to);
        if (2 * of / PIECES == at) load_lds_piece_in<2>(live, from, to);
        if (3 * of / PIECES == at) load_lds_piece_in<3>(live, from, to);
        if (4 * of / PIECES == at) load_lds_piece_in<4>(wave & 1 ? 0 : live, from, to);
    };
    static_assert(PIECES == 5, "five pieces");
    // two waves that share a tile work at step n on item n - 1, and on the weights of item n - 3
    static_assert(LOOK + 2 <= STAGES, "a stage is not filled while it is worked on");
    static_assert(2 * LOOK + 4 <= SLOTS, "an item's word stays until it has been worked on");
    // Item n is worked on after step n, which takes the word of item n + 2 LOOK and aims at item n + LOOK, whose
    // pieces go out between the matrix instructions that follow, to where item n - 2 was. Of the loads issued later
    // than item n's there are those of LOOK - 1 items, each with a word.
    Due due[LOOK];
    {
        Due early[LOOK];
#pragma unroll
        for (int x = 0; x < LOOK; ++x) early[x] = plan(x);
#pragma unroll
        for (int x = 0; x < LOOK; ++x) {
            due[x] = plan(LOOK + x);
            if (x == 0) {
                wait_vmcnt<1>();
                asm volatile("" ::: "memory");           // the words are read behind the wait
            }
            aim(early[x], x);
            pieces_at(0, 1);
        }
    }
    int n = -1;
    auto stage_of = [&](int x) __attribute__((always_inline)) { return ring + x % STAGES * STAGE_BYTES; };
    auto step = [&]() __attribute__((always_inline)) {
        ++n;
        wait_vmcnt<PW *(LOOK - 1)>();
        lds_barrier();
        const Due d = plan(n + 2 * LOOK);
        aim(due[0], n + LOOK);
#pragma unroll
        for (int x = 0; x + 1 < LOOK; ++x) due[x] = due[x + 1];
        due[LOOK - 1] = d;
    };
    // fragment places within a stage: see latent_decode.hip
    constexpr int KA = 64 / T::KSTEP;
    const int kbase = (row >> 3) * (SEGS * 1024) + (row & 7) * 128 + ((grp ^ swz(row)) << 4);
    auto find_rows = [&](lds_u8 *st, lds_u8 *(&at)[KA]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < KA; ++j) {
            int p = (int)(uintptr_t)st + (kbase ^ (j * T::KSTEP * 2));
            asm volatile("" : "+v"(p));                  // one register, the rest is in the instruction
            at[j] = (lds_u8 *)(uintptr_t)(uint32_t)p;
        }
    };

    u32x4_t kf[KS];
    while (todo.more()) {
        // A chunk of half as many tiles as waves or fewer: two waves of a SIMD share a tile, and of the query
        // tiles, which then come two a turn, each takes one (2 requests of 16000 keys x 1024 rows 62 -> 55 us)
        const int share = todo.keys <= WAVES / 2 ? 2 : 1;
        const int mine = share == 2 ? wave % (WAVES / 2) : wave, turn = share == 2 ? wave / (WAVES / 2) : 0;
        for (int x = 0; x < todo.keys; ++x) {
            step();
            pieces_at(0, 1);
            if (x == mine) {
                lds_u8 *at[KA];
                find_rows(stage_of(n), at);
#pragma unroll
                for (int k = 0; k < KS; ++k) kf[k] = *(const lds_u32x4 *)(at[k % KA] + (k / KA) * 1024);
            }
        }
        const bool busy = mine < todo.keys;
        const int k0 = (todo.t + mine) * KT, key = k0 + row, first = todo.len - a.tokens;
        // rows that see this lane's key: from here on. The others lie in the tiles before `some`
        const int least = max(0, key - first) * a.heads;
        const int some = max(0, k0 + KT - 1 - first) * a.heads;
        float sum[4] = {};
        f32x16_t s, before;                              // scores of a query tile, and of the one before it
        // Weights of tile x, whose scores are in `before`, worked on at step n_x. Register i holds row
        // place(i, grp) of the tile; quad() reads the log sums of registers 4 q .. 4 q + 3, weigh() adds one's weight.
        f32x4_t m;
        auto quad = [&](int q, int n_x) __attribute__((always_inline)) {
            typedef __attribute__((address_space(3))) const f32x4_t lds_f32x4;
            m = *(lds_f32x4 *)(words + n_x % SLOTS * SLOT_BYTES + T::place(4 * q, 0) * 4 + grp * 16);
        };
        auto weigh = [&](int i, int x, bool whole) __attribute__((always_inline)) {
            const float e = __builtin_amdgcn_exp2f(fmaf(before[i], a.c, m[i & 3] * -kLog2e));
            const int r = x * KT + T::place(i, grp);
            sum[i & 3] += whole || (r >= least && r < a.rows) ? e : 0.0f;
        };
        // S = Q K^T of tile x, staged at step n_x, and between the matrix instructions the weights of the wave's tile before
        // (mode 0: there is none, 1: all rows see all keys, 2: some may not). Fragments are read so many
        // instructions ahead (a read takes some 130 cycles, an instruction 32); the scheduling barriers keep them there.
        auto scores = [&](int x, int n_x, auto mode) __attribute__((always_inline)) {
            lds_u8 *at[KA];
            find_rows(stage_of(n_x), at);
            constexpr int QUAD = KS / 4;                 // instructions beside which four weights are added
            u32x4_t qf[AHEAD + 1];
            auto read = [&](int e) __attribute__((always_inline)) {
                qf[e % (AHEAD + 1)] = *(const lds_u32x4 *)(at[e % KA] + (e / KA) * 1024);
            };
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) read(e);
#pragma unroll
            for (int e = 0; e < KS; ++e) {
                __builtin_amdgcn_sched_barrier(0);
                if (e + AHEAD < KS) read(e + AHEAD);
                __builtin_amdgcn_sched_barrier(0);
                s = T::mfma(qf[e % (AHEAD + 1)], kf[e], e ? s : f32x16_t{0.0f});
                if constexpr (mode.value > 0) {
                    if (e % QUAD == 0) quad(e / QUAD, n_x - share);
                    if (e % QUAD >= QUAD - 4) weigh(e / QUAD * 4 + e % QUAD - (QUAD - 4), x - share, mode.value == 1);
                }
                pieces_at(e, KS);
            }
        };
        int last = 0, n_last = 0;                        // the wave's last tile
        for (int x0 = 0; x0 < a.qtiles; x0 += share) {
            step();
            const bool two = share == 2 && x0 + 1 < a.qtiles;
            if (two) {
                pieces_at(0, 1);
                step();
            }
            const int x = x0 + turn, n_x = two ? n - 1 + turn : n;
            if (!busy || x >= a.qtiles) {
                pieces_at(0, 1);
                continue;
            }
            if (x0 == 0) scores(x, n_x, std::integral_constant<int, 0>());
            else if ((x - share) * KT >= some) scores(x, n_x, std::integral_constant<int, 1>());
            else scores(x, n_x, std::integral_constant<int, 2>());
            before = s;
            last = x;
            n_last = n_x;
        }
        float total = 0.0f;
        if (busy && turn < a.qtiles) {
#pragma unroll
            for (int i = 0; i < T::NS; ++i) {
                if (i % 4 == 0) quad(i / 4, n_last);
                weigh(i, last, false);
            }
            total = row_sum<T>((sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
        if (share == 2) {                                // the two waves' sums, always in this order
            if (turn == 1 && grp == 0) halves[mine][row] = total;
            lds_barrier();
            total += halves[mine][row];
        }
        // the only addition to this place in the call, so that nothing depends on an order; without a load
        // whose wait would be for the ring's loads too
        if (busy && turn == 0 && grp == 0 && key < min(todo.len, a.columns))
            unsafeAtomicAdd(a.weights + todo.req * a.w_row + key, total);
        todo.left -= todo.keys;
        todo.t += todo.keys;
        todo.enter(a);
    }
}

}  // namespace

hipError_t launch_latent_key_weights(const skinny_latent_key_weights_args &p, int cus, hipStream_t stream) {
    WeightArgs a;
    a.q = static_cast<const uint16_t *>(p.q);
    a.q_row = p.q_row_stride;
    a.q_head = p.q_head_stride;
    a.cache = static_cast<const uint16_t *>(p.cache);
    a.c_page = p.cache_page_stride;
    a.c_row = p.cache_row_stride;
    a.table = p.table;
    a.t_row = p.table_stride;
    a.lens = p.lens;
    a.lse = p.lse;
    a.weights = p.weights;
    a.w_row = p.weights_stride;
    a.batch = (int)p.batch;
    a.tokens = (int)p.tokens;
    a.heads = (int)p.heads;
    a.pages = (int)p.pages;
    a.page = (int)p.page;
    a.max_pages = (int)p.max_pages;
    a.columns = (int)std::min<int64_t>(p.columns, p.max_pages * p.page);
    a.rows = a.tokens * a.heads;
    a.qtiles = (a.rows + KT - 1) / KT;
    a.groups = 1;
    a.lead = (int)(a.qtiles * LEAD);
    reciprocal(a.page, a.page_mul, a.page_shift);
    reciprocal(a.heads, a.head_mul, a.head_shift);
    a.c = p.scale * kLog2e;
    // no more workgroups than the line can have tiles
    a.grid = (int)std::min<int64_t>(cus, (int64_t)a.batch * ((a.columns + KT - 1) / KT + a.lead));
    if (a.grid == 0) return hipSuccess;
    hipLaunchKernelGGL(latent_key_weights_kernel, dim3((unsigned)a.grid), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace skinny
