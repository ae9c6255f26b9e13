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
// Measured: one request of 131071 keys x 32 heads 32 us (151 MB, 4.8 TB/s; its inner loop 6 TB/s) and 7
// for the join; 96 requests of about 4000 keys x 128 heads 132 us (485 MB read, 92 MB of partials
// written) and 22 for the join; 64 requests of 3000 keys x 64 heads 55 us (240 MB read) and 7.6 for the
// join. With 128 rows the matrix instructions take 40% of a wave's time (33% of the kernel's, with its
// start and its uneven end), and neither they nor memory bound it alone: in this layout of one wave a
// SIMD, registers full of sums and queries leave no room to run a tile's softmax beside the next one's
// products.
#include <algorithm>
#include <type_traits>

#include "latent.hpp"

namespace skinny {
namespace {

using namespace latent;

constexpr int L = 512, DIM = 576;            // latents, numbers of a cached row
constexpr int KT = 32;                       // keys a tile
constexpr int SEGS = DIM * 2 / 128;          // 128-byte pieces of a row
constexpr int STAGES = 4;
constexpr int STAGE_BYTES = KT * DIM * 2;
constexpr int PW = SEGS + 1;                 // loads a wave issues per stage: a page id and pieces
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
    int rows, groups, grid;                  // rows a request, row groups a request, workgroups
    uint32_t page_mul;                       // k / page = (k * page_mul) >> (32 + page_shift); 0: page is 1
    int page_shift;
    float c;                                 // scale * log2(e)
};

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
// tiles of a request; one at least, so that an empty one's outputs are written too
__device__ __forceinline__ int request_tiles(const DecodeArgs &a, int i) {
    return max(1, (request_len(a, i) + KT - 1) / KT);
}

// Sum of v over the workgroup's threads before this one, and over all of them.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sh, int64_t &total) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 63) sh[wave] = s;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < wave) before += sh[w];
        total += sh[w];
    }
    return before + s - v;
}

// Where the line of tiles lies: its length, and for place x the request it belongs to and the place
// of that request's first tile. Thread i counts requests i * per .. i * per + per - 1.
struct Line {
    int64_t total, before;                   // of this thread's requests
    int per;
    __device__ __forceinline__ void measure(const DecodeArgs &a, int64_t *sh) {
        per = (a.batch + THREADS - 1) / THREADS;
        int64_t v = 0;
        for (int i = threadIdx.x * per; i < min(a.batch, (int)(threadIdx.x + 1) * per); ++i) v += request_tiles(a, i);
        before = block_scan(v * a.groups, sh, total);
        total = uniform(total);
    }
    __device__ __forceinline__ void find(const DecodeArgs &a, int64_t x, int64_t *sh, int &req, int64_t &base) const {
        int64_t at = before;
        for (int i = threadIdx.x * per; i < min(a.batch, (int)(threadIdx.x + 1) * per); ++i) {
            const int64_t n = (int64_t)request_tiles(a, i) * a.groups;
            if (at <= x && x < at + n) {
                sh[4] = i;
                sh[5] = at;
            }
            at += n;
        }
        __syncthreads();
        req = uniform((int)sh[4]);
        base = uniform(sh[5]);
    }
};

// Runs that the line is cut into: at most one a CU, and with many rows fewer where that leaves less
// work. A run of r tiles takes r t, and the total / r runs leave partials of b bytes each, written and
// read at rate w: r t + 2 b total / (r w) is least at r = sqrt(2 b total / (w t)), so that there are
// sqrt(total) sqrt(w t / 2 b) runs. With the measured t = 1.7 us for 64 rows and 2.4 for 128 (64 requests
// of 3000, 6000 and 12000 keys give 1.8 to 1.9 and 2.2 to 2.6, which moves the factors by 6% at most)
// and w = 4.5 TB/s (128 heads: 32 requests x 1000 keys 57 -> 50 us, one of 10000 37 -> 34; 64 heads:
// 2 x 3000 26 -> 25; of 16 and 32 rows the partials are too small to matter).
template <int MB>
__device__ __forceinline__ int runs(int most, int64_t total) {
    const int grid = (int)min((int64_t)most, total);
    if constexpr (MB < 64) return grid;
    constexpr float FACTOR = MB == 64 ? 5.4f : 4.5f;
    return min(grid, max(1, (int)(FACTOR * sqrtf((float)total))));
}

// Workgroup b's run of the line: [b * total / grid, (b + 1) * total / grid). Runs leave partials
// 2b (of the run's first unit) and 2b + 1 (of its last, if that is another).
__device__ __forceinline__ int64_t run_start(int64_t total, int grid, int b) { return total * b / grid; }
// the workgroup whose run holds place x (no run is empty: grid <= total)
__device__ __forceinline__ int run_of(int64_t total, int grid, int64_t x) { return (int)(((x + 1) * grid - 1) / total); }

template <typename T, int WR, int WD>
struct Shape {
    static constexpr int MB = T::ROWS * WR;              // rows a workgroup
    static constexpr int ND = L / T::DIMS / WD;          // dim tiles a wave
    static constexpr int KS = DIM / T::KSTEP;            // K steps of the score product
    static constexpr int NO4 = T::NO / 4;                // 4-register groups of a dim tile
    // softmax of a tile beside the score product of the next: takes registers that 128 rows x 512
    // sums leave no room for
    static constexpr bool FLOW = MB < 128;
    // fragments read ahead of the matrix instructions (they need about 130 cycles; a 32 x 32
    // instruction takes 32 of them): of keys, and of dim tiles of values. With 128 rows more of them
    // cost more than they hide (groups of 6 and 2: 83 -> 86 us for 32 requests x 128 heads x 4000 keys)
    static constexpr int KG = MB == 128 ? 4 : 6, VG = MB < 128 && ND >= 4 ? 2 : 1;
};

// What a workgroup stages, in order: for each unit (request and row group) of its run, the unit's
// query rows as QT tiles of 32 rows, then its tiles of keys. One stream through the ring, so that
// a unit's first tiles are loaded while the last one's outputs are written.
struct Cursor {
    int req, g, len, tiles, t, t0, end;      // unit; next item: query tile t + QT if t < 0, else key tile t
    int64_t left;                            // key tiles of the run from this unit on
    bool more;
    __device__ __forceinline__ void enter(const DecodeArgs &a, int first, int qt) {
        len = uniform_len(a, req);
        tiles = max(1, (len + KT - 1) / KT);
        t = -qt;
        t0 = first;
        end = (int)min((int64_t)tiles, first + left);
    }
};
// An item whose load is due: this lane's row (of the request's queries, or of its cache page).
struct Due {
    int row, req;
    int kind;                                // 0: none, 1: queries, 2: keys
};

// of a row's pieces, those that go out with group `at` of `of` (both known when compiled)
template <int I = 0>
__device__ __forceinline__ void pieces_at(int at, int of, bool on, const void *src, int lds) {
    if constexpr (I < SEGS) {
        if (I * of / SEGS == at) load_lds_piece_if<I>(on, src, lds);
        pieces_at<I + 1>(at, of, on, src, lds);
    }
}

template <typename T, int WR, int WD>
__global__ __launch_bounds__(THREADS) void latent_decode_kernel(DecodeArgs a) {
    typedef Shape<T, WR, WD> S;
    typedef typename T::acc_t acc_t;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE_BYTES + 4 * STAGES * 256];
    __shared__ int64_t sh[8];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int row = T::row(lane), grp = T::grp(lane);
    const int wr = wave % WR, d0 = (wave / WR) * (L / WD);
    constexpr int QT = (S::MB + KT - 1) / KT;            // query tiles a unit

    Line line;
    line.measure(a, sh);
    const int grid = uniform(runs<S::MB>(a.grid, line.total));
    if ((int)blockIdx.x >= grid) return;
    int64_t lo = run_start(line.total, grid, blockIdx.x);
    const int64_t hi = run_start(line.total, grid, blockIdx.x + 1);
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
    c.more = true;
    {
        const int tiles = max(1, (uniform_len(a, req) + KT - 1) / KT);
        c.g = (int)((lo - base) / tiles);
        c.enter(a, (int)((lo - base) % tiles), QT);
    }
    // takes the next item; its page ids go to place `slot` of the ids' ring
    auto plan = [&](int slot) __attribute__((always_inline)) {
        Due d{0, c.req, 0};
        const int32_t *id = a.table;
        if (c.more) {
            const int kl = 8 * wave + (own_lane() >> 3);
            if (c.t < 0) {                               // rows past the last repeat it
                d.row = min(c.g * S::MB + (c.t + QT) * KT + kl, a.rows - 1);
                d.kind = 1;
                if (++c.t == 0) c.t = c.t0;
            } else {                                     // keys past the end repeat the last one: masked
                const int k = max(0, min(c.t * KT + kl, c.len - 1));
                const int page = a.page_mul ? (int)(__umulhi((uint32_t)k, a.page_mul) >> a.page_shift) : k;
                id = a.table + c.req * a.t_row + page;
                d.row = k - page * a.page;
                d.kind = 2;
                if (++c.t == c.end) {
                    c.left -= c.end - c.t0;
                    c.more = c.left > 0;
                    if (c.more) {
                        if (++c.g == a.groups) {
                            c.g = 0;
                            ++c.req;
                        }
                        c.enter(a, 0, QT);
                    }
                }
            }
        }
        load_lds_word(id, lds_address(ids + slot % STAGES * 256));
        return d;
    };
    // where a due item's pieces come from and go to
    const uint16_t *from = a.cache;
    int to = 0;
    auto aim = [&](const Due &d, int slot) __attribute__((always_inline)) {
        const int x = own_lane();
        const int chunk = ((x & 7) ^ swz(8 * wave + (x >> 3))) * 8;
        if (d.kind == 2) {                               // ids outside the pool are clamped
            const int id = *(__attribute__((address_space(3))) const int32_t *)(ids + slot % STAGES * 256 + x * 4);
            from = a.cache + (int64_t)min(max(id, 0), a.pages - 1) * a.c_page + (int64_t)d.row * a.c_row + chunk;
        } else {
            const int j = d.row / a.heads, h = d.row - j * a.heads;
            from = a.q + ((int64_t)d.req * a.tokens + j) * a.q_row + h * a.q_head + chunk;
        }
        to = lds_address(ring + slot % STAGES * STAGE_BYTES + wave * (SEGS * 1024));
    };
    // Item n is staged after step n, which takes the ids of item n + 2 LOOK and aims at item n + LOOK;
    // the pieces of the latter go out between the matrix instructions that follow, one at a time
    // (ten loads in a row hold a wave up for 1100 cycles). The stage that they fill is free: the
    // value product is done with item n - 1, or, where it runs one step behind the score product,
    // with item n - 2.
    constexpr int LOOK = S::FLOW ? 2 : 3;
    static_assert(LOOK <= QT + 1, "the items issued before the first step exist");
    int n = -1;
    Due due[LOOK];                                       // the next items to be issued
    {
        Due early[LOOK];
#pragma unroll
        for (int x = 0; x < LOOK; ++x) early[x] = plan(x);
        due[0] = plan(LOOK);
        aim(early[0], 0);                                // queries: their ids are not needed
        load_lds_pieces<SEGS>(from, to);
        wait_vmcnt<SEGS>();
#pragma unroll
        for (int x = 1; x < LOOK; ++x) {
            due[x] = plan(LOOK + x);
            aim(early[x], x);
            load_lds_pieces<SEGS>(from, to);
        }
    }
    lds_u8 *st = ring, *st_before = ring;
    bool live = false;                                   // there is an item to issue
    auto step = [&]() __attribute__((always_inline)) {
        ++n;
        wait_vmcnt<PW *(LOOK - 1)>();
        lds_barrier();
        live = due[0].kind != 0;
        const Due d = plan(n + 2 * LOOK);
        if (live) aim(due[0], n + LOOK);
#pragma unroll
        for (int x = 0; x + 1 < LOOK; ++x) due[x] = due[x + 1];
        due[LOOK - 1] = d;
        st_before = st;
        st = ring + n % STAGES * STAGE_BYTES;
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
                at[j][hh] = place_of(from, (vbase ^ (j * T::DIMS * 2) ^ (HALF == 8 ? hh * 16 : 0)) + hh * (HALF / 8) * (SEGS * 1024));
    };

    constexpr int NT = KT / T::ROWS;                     // key subtiles: 1 or 2
    constexpr int XS = T::NS / 8;                        // key steps of the value product
    constexpr int KG = S::KG, NG = S::KS * NT / KG;      // fragments a group, groups of the score product
    static_assert(KG * NG == S::KS * NT, "whole groups");
    // places between matrix instructions where pieces go out: all of a step's, if a value product
    // follows each score product
    constexpr int ISSUES = S::FLOW ? NG : NG + S::ND / S::VG;
    u32x4_t qf[S::KS], pf[XS];
    acc_t o[S::ND], s[NT], next[NT];
    float m, l;

    // S^T = K Q^T of the staged tile into `sum`, and beside it, in slices between the matrix
    // instructions, the softmax weights of the tile before from s. Fragments are read a group
    // ahead; the scheduling barriers keep the groups apart, and the compiler from spilling.
    // Weights are rounded to bf16 for the matrix product, whose operands are of one type (by 2^-8 relative
    // at most, independently of each other: an output's error grows from the 0.0017 of its own rounding
    // to 0.0022 at most in the listed cases); their sum l is of the unrounded ones.
    float mu = 0.0f;
    auto weight_slice = [&](int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
        for (int i = i0; i < i1; i += 2) {
            const float x = __builtin_amdgcn_exp2f(fmaf(s[i / T::NO][i % T::NO], a.c, -mu));
            const float y = __builtin_amdgcn_exp2f(fmaf(s[(i + 1) / T::NO][(i + 1) % T::NO], a.c, -mu));
            l += x;
            l += y;
            pf[i / 8][i % 8 / 2] = pack_bf16(x, y);
        }
    };
    auto scores = [&](acc_t (&sum)[NT], auto with_weights) __attribute__((always_inline)) {
        lds_u8 *at[KA];
        find_keys(st, at);
        auto key_frag = [&](int e) __attribute__((always_inline)) {
            const int k = e / NT, u = e % NT;
            return *(const lds_u32x4 *)(at[k % KA] + (u * T::ROWS / 8) * (SEGS * 1024) + (k / KA) * 1024);
        };
        u32x4_t kf[2][KG];
#pragma unroll
        for (int e = 0; e < KG; ++e) kf[0][e] = key_frag(e);
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
            __builtin_amdgcn_sched_barrier(0);
            if (gi + 1 < NG) {
#pragma unroll
                for (int e = 0; e < KG; ++e) kf[(gi + 1) & 1][e] = key_frag((gi + 1) * KG + e);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < KG; ++e) {
                const int k_at = gi * KG + e;
                sum[k_at % NT] = T::mfma(kf[gi & 1][e], qf[k_at / NT], k_at / NT ? sum[k_at % NT] : acc_t{0.0f});
            }
            if constexpr (with_weights.value) weight_slice(T::NS / 2 * gi / NG * 2, T::NS / 2 * (gi + 1) / NG * 2);
            pieces_at(gi, ISSUES, live, from, to);
        }
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
                if constexpr (!S::FLOW)
                    if (i % S::VG == S::VG - 1) pieces_at(NG + i / S::VG, ISSUES, live && !others, from, to);
            }
            return;
        }
        constexpr int VG = S::VG;
        u32x4_t vf[2][VG * XS];
#pragma unroll
        for (int e = 0; e < VG * XS; ++e) vf[0][e] = value(e / XS, e % XS);
#pragma unroll
        for (int i = 0; i < S::ND; i += VG) {
            __builtin_amdgcn_sched_barrier(0);
            if (i + VG < S::ND) {
#pragma unroll
                for (int e = 0; e < VG * XS; ++e) vf[(i / VG + 1) & 1][e] = value(i + VG + e / XS, e % XS);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < VG * XS; ++e) {
                o[i + e / XS] = T::mfma(vf[i / VG & 1][e], pf[e % XS], o[i + e / XS]);
            }
            if constexpr (!S::FLOW) pieces_at(NG + i / VG, ISSUES, live, from, to);
        }
    };
    // The same for tile t with scores that are not finite, of which some rows see less than others. A
    // latent that is not finite must not reach rows that do not see it, whose weight 0 times it is NaN;
    // for rows that see it that product is right (its score is -inf, weight 0, or they are NaN
    // throughout): they get +inf and -inf, each a product of the largest number, the others 0. One
    // loop, not three copies: the 128-row shape has no registers to spare.
    auto add_values_carefully = [&](lds_u8 *tile, int t, int limit) __attribute__((always_inline)) {
#pragma clang loop unroll(disable)
        for (int pass = 0; pass < 3; ++pass) {
            if (pass) {
                const uint32_t sign = pass == 1 ? 0u : 0x80008000u;
                const int left = limit - t * KT;
#pragma unroll
                for (int i = 0; i < T::NS; i += 2)
                    pf[i / 8][i % 8 / 2] = seen_pair(T::place(i, grp) < left, T::place(i + 1, grp) < left) ^ sign;
            }
            add_values(tile, std::true_type(), pass > 0);
        }
        in_acc(o);
    };

    bool leading = true;                                 // the run's first unit
    while (lo < hi) {
        const int len = uniform_len(a, req), tiles = max(1, (len + KT - 1) / KT);
        const int g = (int)((lo - base) / tiles), t0 = (int)((lo - base) % tiles);
        const int t1 = (int)min((int64_t)tiles, t0 + (hi - lo));
        // keys this lane's row sees: it is row (token, head) of the request; rows past the last repeat it
        const int limit = max(0, len - a.tokens + 1 + min(g * S::MB + wr * T::ROWS + row, a.rows - 1) / a.heads);
        const int whole = max(0, len - a.tokens + 1) / KT;       // tiles before this: all rows see all of them

        for (int qi = 0; qi < QT; ++qi) {
            step();
            pieces_at(0, 1, live, from, to);
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
            if (t >= whole) {
#pragma unroll
                for (int i = 0; i < T::NS; ++i) {
                    const float x = s[i / T::NO][i % T::NO];
                    const bool seen = t * KT + T::place(i, grp) < limit, fin = finite_f32(x);
                    odd |= !fin;                         // so is the key's row, or a query
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
        auto rescale = [&]() __attribute__((always_inline)) {
            const float up = fmaxf(m, top);
            const float alpha = up == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            mu = m == -INFINITY ? 0.0f : m;
            l *= alpha;
            grow = false;
#pragma unroll
            for (int i = 0; i < S::ND; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                o[i] *= alpha;
                in_acc(o);
            }
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
                    rescale();
                    if (!odd && t + 1 < t1) continue;
                }
                weight_slice(0, T::NS);
                if (odd) add_values_carefully(st, t, limit);     // rare
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
                    weight_slice(0, T::NS);
                    add_values(st, std::false_type(), false);
                } while (++t < t1);
                if (t >= t1) break;
                if (grow) rescale();
                if (!odd) {
                    scored = true;
                    continue;
                }
                weight_slice(0, T::NS);
                add_values_carefully(st, t, limit);      // rare
                if (++t >= t1) break;
            }
        }
        l = row_sum<T>(l);

        const int r = g * S::MB + wr * T::ROWS + T::row(own_lane()), rc = min(r, a.rows - 1);
        const int j = rc / a.heads, h = rc - j * a.heads;
        const int64_t qr = (int64_t)req * a.tokens + j;
        const bool uncut = t0 == 0 && t1 == tiles;
        if (t0 == 0 && tid == 0)
            a.cuts[(int64_t)req * a.groups + g] = make_int2(
                2 * blockIdx.x + (leading ? 0 : 1), uncut ? (int)blockIdx.x : run_of(line.total, grid, lo + tiles - 1));
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
        } else {
            float *part = a.work + (2 * (int64_t)blockIdx.x + (leading ? 0 : 1)) * part_floats<S::MB>();
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
        lo += t1 - t0;
        if (lo == base + (int64_t)tiles * a.groups) {
            base = lo;
            ++req;
        }
    }
}

// Joins the partial sums of the units that were cut between workgroups. A wave's lanes are PL groups:
// each takes the same 64 / PL float4 of a unit's sums, of every PL-th partial. WP waves share a
// unit's partials further and meet in LDS; each lane asks for 4 partials at once. With few units the
// latency of these loads bounds it (256 partials of 32 rows, 17 MB: 7.0 us, of which the launch and the
// look-up of the cuts are most; 8.5 with whole waves on a partial), with many their bytes
// (350 partials of 128 rows, 92 MB: 22 us, 4.7 TB/s).
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
    const int req = unit / a.groups, g = unit % a.groups;

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
    for (int j = turn; j < pieces; j += 4 * TURNS) {
        float pm[4], pl[4];
        f32x4_t po[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float *part = partial(min(j + u * TURNS, pieces - 1));
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
    const int r = g * S::MB + row;
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
    const unsigned blocks = (unsigned)((int64_t)a.batch * a.groups * (PER / QUADS));
    hipLaunchKernelGGL((latent_join_kernel<T, WR, WD, WP, PL>), dim3(blocks), dim3(WP > 4 ? WP * 64 : 256), 0, stream, a);
    return hipGetLastError();
}

template <typename T, int WR, int WD>
hipError_t launch_shape(DecodeArgs a, hipStream_t stream) {
    a.cuts = reinterpret_cast<int2 *>(a.work + 2 * a.grid * part_floats<Shape<T, WR, WD>::MB>());
    hipLaunchKernelGGL((latent_decode_kernel<T, WR, WD>), dim3((unsigned)a.grid), dim3(THREADS), 0, stream, a);
    hipError_t err = hipGetLastError();
    // one workgroup takes every run whole: nothing to join
    if (err != hipSuccess || a.grid == 1) return err;
    // takers of a unit's partials: about as many as it has on average, unless that makes more waves
    // than the chip holds at once (8 requests x 4000 keys x 128 heads 47 us with 16, 44 with 4)
    const int64_t units = (int64_t)a.batch * a.groups, waves = units * (Shape<T, WR, WD>::MB * L / 4 / 64), room = 16384;
    if (a.grid > 64 * units && waves * 64 <= room) return launch_join<T, WR, WD, 16, 4>(a, stream);
    if (a.grid > 16 * units && waves * 16 <= room) return launch_join<T, WR, WD, 16, 1>(a, stream);
    if (a.grid > 4 * units) return launch_join<T, WR, WD, 4, 1>(a, stream);
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

hipError_t launch_latent_decode(const skinny_latent_decode_args &p, int cus, hipStream_t stream) {
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
    // 2^bits >= page > 2^(bits - 1): the reciprocal 2^(31 + bits) / page, rounded up, fits 32 bits, and
    // for k < 2^30 its rounding adds less than 2^-(1 + bits) < 1 / page to the quotient: exact
    int bits = 1;
    while ((1 << bits) < a.page) ++bits;
    a.page_mul = a.page == 1 ? 0 : (uint32_t)((((uint64_t)1 << (31 + bits)) + a.page - 1) / a.page);
    a.page_shift = bits - 1;
    const int mb = block_rows(a.rows);
    a.groups = (a.rows + mb - 1) / mb;
    a.c = p.scale * kLog2e;
    // no more workgroups than the line can have tiles
    const int64_t most = (int64_t)a.batch * a.groups * std::max<int64_t>(1, (p.max_pages * p.page + KT - 1) / KT);
    a.grid = (int)std::min<int64_t>(cus, most);
    switch (mb) {
        case 16: return launch_shape<Tile16, 1, 4>(a, stream);
        case 32: return launch_shape<Tile16, 2, 2>(a, stream);
        case 64: return launch_shape<Tile16, 4, 1>(a, stream);
        default: return launch_shape<Tile32, 4, 1>(a, stream);
    }
}

}  // namespace skinny
