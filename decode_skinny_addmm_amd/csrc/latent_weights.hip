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
#include <algorithm>

#include "latent_line.hpp"

namespace skinny {
namespace {

using namespace latent;
typedef Tile32 T;

constexpr int DIM = 576;                     // numbers of a cached row
constexpr int KT = 32;                       // keys, or query rows, a tile
constexpr int SEGS = DIM * 2 / 128;          // 128-byte pieces of a row
constexpr int STAGES = 3, LOOK = STAGES - 1; // stages in LDS, and of them in flight
constexpr int STAGE_BYTES = KT * DIM * 2;
constexpr int WAVES = 8, THREADS = WAVES * 64;
constexpr int PIECES = (SEGS + 1) / 2;       // two waves share 8 rows of a stage: 5 pieces and 4 (and one that loads nothing)
constexpr int PW = PIECES + 1;               // loads a wave issues a stage: a word and pieces
constexpr int SLOTS = 8;                     // words of that many stages: page ids, or rows' log sums
constexpr int KS = DIM / T::KSTEP;           // K steps

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
    uint32_t page_mul;                       // see page_of
    int page_shift;
    float c;                                 // scale * log2(e)
};

__device__ __forceinline__ int clamp_len(const WeightArgs &a, int n) { return min(max(n, 0), a.max_pages * a.page); }
__device__ __forceinline__ int uniform_len(const WeightArgs &a, int i) {     // see latent_decode.hip
    typedef const __attribute__((address_space(4))) int32_t *constant_ptr;
    return clamp_len(a, ((constant_ptr)(uintptr_t)a.lens)[i]);
}
// tiles of the keys that have a column
__device__ __forceinline__ int tiles_of(const WeightArgs &a, int len) { return (min(len, a.columns) + KT - 1) / KT; }
__device__ __forceinline__ int request_tiles(const WeightArgs &a, int i) { return tiles_of(a, clamp_len(a, a.lens[i])); }

// The items of a run, in order: for each chunk its key tiles, then all query tiles of its request.
struct Chunks {
    int req, len, tiles;                     // request
    int t, keys, x;                          // chunk: its first tile, its number of tiles, next item
    int64_t left;                            // tiles of the run from this chunk on
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void enter(const WeightArgs &a) {     // finds the chunk from tile t on
        while (left > 0 && t >= tiles) {
            if (++req == a.batch) {                      // lengths that change under the call: the run ends here
                left = 0;
                break;
            }
            len = uniform_len(a, req);
            tiles = tiles_of(a, len);
            t = 0;
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
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE_BYTES + WAVES * SLOTS * 256];
    __shared__ int64_t sh[WAVES + 2];
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    const int row = T::row(lane), grp = T::grp(lane);

    Line<WeightArgs, THREADS> line;
    line.measure(a, sh);
    const int grid = (int)min((int64_t)a.grid, line.total);
    if ((int)blockIdx.x >= grid) return;
    const int64_t lo = run_start(line.total, grid, blockIdx.x), hi = run_start(line.total, grid, blockIdx.x + 1);
    Chunks c, todo;
    int64_t base;
    line.find(a, lo, sh, c.req, base);
    c.len = uniform_len(a, c.req);
    c.tiles = tiles_of(a, c.len);
    c.t = (int)(lo - base);
    c.left = hi - lo;
    c.enter(a);
    todo = c;                                            // c: what is staged next, todo: what is worked on next

    lds_u8 *ring = (lds_u8 *)lds;
    lds_u8 *words = ring + STAGES * STAGE_BYTES + wave * (SLOTS * 256);
    // staging: waves 2b and 2b + 1 take rows 8b .. 8b + 7 of a tile, lane l row l / 8; the first of them
    // the row's pieces 0 .. 4, the second 5 .. 8
    const int own = 8 * (wave >> 1) + (lane >> 3), chunk = ((lane & 7) ^ swz(own)) * 8 + (wave & 1) * (PIECES * 64);
    auto plan = [&](int slot) __attribute__((always_inline)) {
        Due d{0, c.req, 0};
        const void *word = a.table;
        if (c.more()) {
            if (c.x < c.keys) {                          // keys past the end repeat the last one
                const int k = min((c.t + c.x) * KT + own, c.len - 1), page = page_of(a, k);
                word = a.table + c.req * a.t_row + page;
                d.row = k - page * a.page;
                d.kind = 2;
            } else {                                     // rows past the last repeat it
                const int first = (c.x - c.keys) * KT;
                word = a.lse + (int64_t)c.req * a.rows + min(first + (lane & 31), a.rows - 1);
                d.row = min(first + own, a.rows - 1);
                d.kind = 1;
            }
            c.next(a);
        }
        load_lds_word(word, lds_address(words + slot % SLOTS * 256));
        return d;
    };
    auto stage = [&](const Due &d, int slot) __attribute__((always_inline)) {
        const uint16_t *from = a.cache;
        if (d.kind == 2) {                               // ids outside the pool are clamped
            const int id = *(__attribute__((address_space(3))) const int32_t *)(words + slot % SLOTS * 256 + lane * 4);
            from = a.cache + (int64_t)min(max(id, 0), a.pages - 1) * a.c_page + (int64_t)d.row * a.c_row + chunk;
        } else if (d.kind == 1) {
            const int j = d.row / a.heads, h = d.row - j * a.heads;
            from = a.q + ((int64_t)d.req * a.tokens + j) * a.q_row + h * a.q_head + chunk;
        }
        const int to = lds_address(ring + slot % STAGES * STAGE_BYTES + (wave >> 1) * (SEGS * 1024) + (wave & 1) * (PIECES * 1024));
        load_lds_piece_if<0>(d.kind != 0, from, to);
        load_lds_piece_if<1>(d.kind != 0, from, to);
        load_lds_piece_if<2>(d.kind != 0, from, to);
        load_lds_piece_if<3>(d.kind != 0, from, to);
        load_lds_piece_if<4>(d.kind != 0 && !(wave & 1), from, to);
    };
    static_assert(PIECES == 5 && LOOK == 2, "five pieces, two stages ahead");
    // Item n is worked on after step n, which takes the word of item n + 4 and stages item n + 2 where item
    // n - 1 was. Of the loads issued later than item n's there are those of item n + 1 and the word with them.
    Due due[LOOK];
    {
        const Due first = plan(0), second = plan(1);
        due[0] = plan(2);
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");                   // the words are read behind the wait
        stage(first, 0);
        due[1] = plan(3);
        stage(second, 1);
    }
    int n = -1;
    lds_u8 *st = ring;
    auto step = [&]() __attribute__((always_inline)) {
        ++n;
        wait_vmcnt<PW>();
        lds_barrier();
        const Due d = plan(n + 2 * LOOK);
        stage(due[0], n + LOOK);
        due[0] = due[1];
        due[1] = d;
        st = ring + n % STAGES * STAGE_BYTES;
    };
    // fragment places within a stage: see latent_decode.hip
    constexpr int KA = 64 / T::KSTEP;
    const int kbase = (row >> 3) * (SEGS * 1024) + (row & 7) * 128 + ((grp ^ swz(row)) << 4);
    auto find_rows = [&](lds_u8 *(&at)[KA]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < KA; ++j) {
            int p = (int)(uintptr_t)st + (kbase ^ (j * T::KSTEP * 2));
            asm volatile("" : "+v"(p));                  // one register, the rest is in the instruction
            at[j] = (lds_u8 *)(uintptr_t)(uint32_t)p;
        }
    };

    u32x4_t kf[KS];
    while (todo.more()) {
        for (int x = 0; x < todo.keys; ++x) {
            step();
            if (x == wave) {
                lds_u8 *at[KA];
                find_rows(at);
#pragma unroll
                for (int k = 0; k < KS; ++k) kf[k] = *(const lds_u32x4 *)(at[k % KA] + (k / KA) * 1024);
            }
        }
        const bool busy = wave < todo.keys;
        const int k0 = (todo.t + wave) * KT, key = k0 + row, first = todo.len - a.tokens;
        // rows that see this lane's key: from here on. The others lie in the tiles before `some`
        const int least = max(0, key - first) * a.heads;
        const int some = max(0, k0 + KT - 1 - first) * a.heads;
        float sum[T::NS] = {};
        for (int x = 0; x < a.qtiles; ++x) {
            step();
            if (!busy) continue;
            lds_u8 *at[KA];
            find_rows(at);
            f32x16_t s = {0.0f};
            constexpr int G = 6, NG = KS / G;            // fragments are read a group ahead
            u32x4_t qf[2][G];
            auto group = [&](int g) __attribute__((always_inline)) {
#pragma unroll
                for (int e = g * G; e < g * G + G; ++e) qf[g & 1][e % G] = *(const lds_u32x4 *)(at[e % KA] + (e / KA) * 1024);
            };
            group(0);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                __builtin_amdgcn_sched_barrier(0);
                if (g + 1 < NG) group(g + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = g * G; e < g * G + G; ++e) s = T::mfma(qf[g & 1][e % G], kf[e], s);
            }
            // register i holds row place(i, grp) of the tile
            const lds_u8 *lse = words + n % SLOTS * 256 + grp * 16;
            const int r0 = x * KT + T::place(0, grp);
            const bool whole = x * KT >= some && x * KT + KT <= a.rows;
#pragma unroll
            for (int i = 0; i < T::NS; i += 4) {
                typedef __attribute__((address_space(3))) const f32x4_t lds_f32x4;
                const f32x4_t m = *(lds_f32x4 *)(lse + 8 * i) * kLog2e;
#pragma unroll
                for (int y = i; y < i + 4; ++y) {
                    const float e = __builtin_amdgcn_exp2f(fmaf(s[y], a.c, -m[y - i]));
                    const int r = r0 + T::place(y, 0);
                    sum[y] += whole || (r >= least && r < a.rows) ? e : 0.0f;
                }
            }
        }
        if (busy) {
#pragma unroll
            for (int d = T::NS / 2; d > 0; d >>= 1)
#pragma unroll
                for (int i = 0; i < d; ++i) sum[i] += sum[i + d];
            const float total = row_sum<T>(sum[0]);
            // the only addition to this place in the call, so that nothing depends on an order; without
            // a load whose wait would be for the ring's loads too
            if (grp == 0 && key < min(todo.len, a.columns)) unsafeAtomicAdd(a.weights + todo.req * a.w_row + key, total);
        }
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
    page_reciprocal(a.page, a.page_mul, a.page_shift);
    a.c = p.scale * kLog2e;
    // no more workgroups than the line can have tiles
    a.grid = (int)std::min<int64_t>(cus, (int64_t)a.batch * ((a.columns + KT - 1) / KT));
    if (a.grid == 0) return hipSuccess;
    hipLaunchKernelGGL(latent_key_weights_kernel, dim3((unsigned)a.grid), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

}  // namespace skinny
