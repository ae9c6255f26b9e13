// latent_decode.hip -- absorbed latent attention of new tokens over a paged latent cache.
//
// For request i with n = lens[i] cached rows c_k = [z_k, r_k] (512 latents, 64 rotated numbers)
// and its `tokens` newest positions, query (j, h) attends to keys k < n - tokens + j + 1:
//     s_k = scale * q . c_k,   out = sum_k softmax(s)_k z_k,   lse = log sum_k exp(s_k).
//
// What bounds it: each cached row is 1152 bytes and serves tokens * heads queries at 2 * 1088
// operations each, so up to 128 query rows a request the cache's bytes bound it.
//   * A workgroup holds all query rows of a request (up to 128; more go in groups) and reads a
//     contiguous run of its keys once, in tiles of 32 keys through a ring of 4 LDS stages (three
//     stages, 110 KB, are in flight behind the one computed on). Keys and values are the same
//     staged rows.
//   * One workgroup a CU; the tiles of all requests are one line, cut into equal runs, one a
//     workgroup, whatever the lengths (which only the device knows). A request cut between
//     workgroups leaves fp32 partial sums in the workspace, joined by a second kernel.
//   * 4 waves as WR row groups x WD groups of latent dims: each wave computes the whole scores
//     of its rows (repeated by the WD waves: matrix time is spare, and no scores cross waves)
//     and its dims of the output, so the only barrier is the ring's.
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
constexpr int PW = SEGS + 1;                 // loads a wave issues per stage: pieces and page id
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
    float c;                                 // scale * log2(e)
};

// One partial: MB rows x 512 sums in the waves' own register order, then MB maxima, MB sums.
template <int MB>
__host__ __device__ constexpr int64_t part_floats() { return (int64_t)MB * (L + 2); }

__device__ __forceinline__ int request_len(const DecodeArgs &a, int i) {
    const int64_t cap = (int64_t)a.max_pages * a.page;
    const int n = max(a.lens[i], 0);
    return cap < n ? (int)cap : n;
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

// Total tiles over all requests and row groups.
__device__ int64_t all_tiles(const DecodeArgs &a, int64_t *sh) {
    int64_t v = 0, total;
    for (int i = threadIdx.x; i < a.batch; i += THREADS) v += request_tiles(a, i);
    block_scan(v, sh, total);
    return total * a.groups;
}

// The request that place x of the line of tiles belongs to, and the place of its first tile.
// sh: 8 words; the caller's threads all get the answer.
__device__ void find_request(const DecodeArgs &a, int64_t x, int64_t *sh, int &req, int64_t &base) {
    int64_t carry = 0;
    for (int i0 = 0; i0 < a.batch; i0 += THREADS) {
        const int i = i0 + threadIdx.x;
        const int64_t v = i < a.batch ? (int64_t)request_tiles(a, i) * a.groups : 0;
        int64_t total;
        const int64_t at = carry + block_scan(v, sh, total);
        if (v > 0 && at <= x && x < at + v) {
            sh[4] = i;
            sh[5] = at;
        }
        carry += total;
        if (x < carry) break;                // uniform: carry and x are the same in every thread
    }
    __syncthreads();
    req = uniform((int)sh[4]);
    base = uniform(sh[5]);
    __syncthreads();
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
    // fragments read ahead of the matrix instructions (they need about 130 cycles; a 32 x 32
    // instruction takes 32 of them): of keys, and of dim tiles of values
    static constexpr int KG = WR == 4 ? 4 : 6, VG = ND >= 4 ? 2 : 1;
};

// One run of tiles [t0, t1) of one request and row group: the wave's sums, maximum and total.
// limit: keys that the lane's row sees; first: the fewest that any row of the request sees.
template <typename T, int WR, int WD>
__device__ __forceinline__ void run_tiles(const DecodeArgs &a, uint8_t *lds, const uint16_t *qp, int req, int len, int t0, int t1, int limit, int first,
                                          typename T::acc_t (&o)[Shape<T, WR, WD>::ND], float &m, float &l) {
    typedef Shape<T, WR, WD> S;
    typedef typename T::acc_t acc_t;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = T::row(lane), grp = T::grp(lane);
    const int d0 = (wave / WR) * (L / WD);               // this wave's first latent dim
    lds_u8 *ring = (lds_u8 *)lds;
    lds_u8 *ids = ring + STAGES * STAGE_BYTES + wave * (STAGES * 256);

    // staging: wave w takes keys 8w .. 8w+7 of a tile, lane l row l / 8. Keys past the end repeat
    // the last one (their scores are masked, and what they hold is never an unwritten row)
    const int kl = 8 * wave + (lane >> 3);
    const int chunk = ((lane & 7) ^ swz(kl)) * 8;
    const int32_t *trow = a.table + (int64_t)req * a.t_row;
    auto key_at = [&](int t) { return max(0, min(t * KT + kl, len - 1)); };
    auto fetch_id = [&](int t) {                         // page id of this lane's key of tile t
        load_lds_word(trow + key_at(t) / a.page, lds_address(ids + (t % STAGES) * 256));
    };
    auto issue = [&](int t, int id) {                    // tile t -> slot t % STAGES
        const int k = key_at(t);
        const int pg = min(max(id, 0), a.pages - 1);     // ids outside the pool are clamped
        const uint16_t *src = a.cache + (int64_t)pg * a.c_page + (int64_t)(k % a.page) * a.c_row + chunk;
        load_lds_pieces<SEGS>(src, lds_address(ring + (t % STAGES) * STAGE_BYTES + wave * (SEGS * 1024)));
    };
    auto read_id = [&](int t) {
        return *(__attribute__((address_space(3))) const int32_t *)(ids + (t % STAGES) * 256 + lane * 4);
    };

#pragma unroll
    for (int i = 0; i < S::ND; ++i)
#pragma unroll
        for (int j = 0; j < T::NO; ++j) o[i][j] = 0.0f;
    m = -INFINITY;
    l = 0.0f;

    // the first tiles' ids come straight into registers, the later ones' with the stage before
    int id0[STAGES - 1];
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) id0[s] = trow[key_at(t0 + s) / a.page];
    asm volatile("" ::: "memory");                       // the queries' loads go out behind the ids'
    u32x4_t qf[S::KS];
#pragma unroll
    for (int k = 0; k < S::KS; ++k) qf[k] = *reinterpret_cast<const u32x4_t *>(qp + k * T::KSTEP + grp * 8);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (t0 + s < t1) {
            fetch_id(t0 + s + STAGES - 1);
            issue(t0 + s, id0[s]);
        }
    }
    // Fragment places within a stage, with the swizzle worked out once. Score product: key row
    // `row` of each subtile (subtiles start at multiples of 16 rows: the same swizzle), K step k
    // reads 16-byte chunk k * KSTEP / 8 + grp of the row: one of KA places a 128-byte piece.
    constexpr int KA = 64 / T::KSTEP;
    int koff[KA];
#pragma unroll
    for (int j = 0; j < KA; ++j)
        koff[j] = (row >> 3) * (SEGS * 1024) + (row & 7) * 128 + (((j * (T::KSTEP / 8) + grp) ^ swz(row)) << 4);
    // Value product: 16-lane group reads keys kv + 0 .. 3 at dims dv + 0 .. 15; the dim tile's
    // place in its 128-byte piece and the half of the key step change the swizzle
    constexpr int VA = 64 / T::DIMS;
    const int kv = T::place(0, grp) + ((lane & 15) >> 2);
    const int dv = (T::ROWS == 32 ? ((lane >> 4) & 1) * 16 : 0) + (lane & 3) * 4;
    int voff[VA][2];
#pragma unroll
    for (int j = 0; j < VA; ++j)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = kv + T::place(4 * hh, 0), ch = (j * T::DIMS + dv) >> 3;
            voff[j][hh] = (r >> 3) * (SEGS * 1024) + (d0 >> 6) * 1024 + (r & 7) * 128 + ((ch ^ swz(r)) << 4) + (dv & 4) * 2;
        }
    constexpr int NT = KT / T::ROWS;                     // key subtiles: 1 or 2
    constexpr int XS = T::NS / 8;                        // key steps of the value product
    acc_t s[NT];
    u32x4_t pf[XS];
    lds_u8 *st;
    // waits for tile t, frees slot (t - 1) % STAGES and refills it
    auto stage = [&](int t) {
        wait_stages<PW, STAGES - 2>(min(STAGES - 2, t1 - 1 - t));
        lds_barrier();
        if (t + STAGES - 1 < t1) {
            const int id = read_id(t + STAGES - 1);
            asm volatile("" ::: "memory");
            fetch_id(t + 2 * (STAGES - 1));
            issue(t + STAGES - 1, id);
        }
        st = ring + (t % STAGES) * STAGE_BYTES;
    };
    // S^T = K Q^T. Fragments are read a group ahead of their matrix instructions; the scheduling
    // barriers keep the compiler from reading whole tiles ahead and spilling
    auto scores = [&]() {
        constexpr int KG = S::KG, NG = S::KS * NT / KG;  // fragments a group, groups
        static_assert(KG * NG == S::KS * NT, "whole groups");
        auto key_frag = [&](int e) {
            const int k = e / NT, u = e % NT;
            return *(const lds_u32x4 *)(st + koff[k % KA] + (u * T::ROWS / 8) * (SEGS * 1024) + (k / KA) * 1024);
        };
#pragma unroll
        for (int u = 0; u < NT; ++u) s[u] = acc_t{0.0f};
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
#pragma unroll
            for (int e = 0; e < KG; ++e) {
                const int at = gi * KG + e;
                s[at % NT] = T::mfma(kf[gi & 1][e], qf[at / NT], s[at % NT]);
            }
        }
        in_vgpr(s);
    };
    auto largest = [&]() {
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < T::NS; ++i) top = fmaxf(top, s[i / T::NO][i % T::NO]);
        return row_max<T>(top) * a.c;
    };
    // Softmax weights against the reference maximum. They are rounded to bf16 for the matrix
    // product (relative 2^-9 each, as the values are); their sum l is of the unrounded ones
    auto weights = [&](float mu) {
        float p[T::NS];
#pragma unroll
        for (int i = 0; i < T::NS; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(s[i / T::NO][i % T::NO], a.c, -mu));
            l += p[i];
        }
#pragma unroll
        for (int i = 0; i < T::NS / 2; ++i) pf[i / 4][i % 4] = pack_bf16(p[2 * i], p[2 * i + 1]);
    };
    // A fragment of V^T: dim tile i, key step x. B register pairs hold keys place(8x + j), j =
    // 0 .. 7, and so does this
    auto value = [&](int i, int x) {
        u32x4_t f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            lds_u8 *at = st + voff[i % VA][hh] + (i / VA) * 1024 + 2 * x * (SEGS * 1024);
            const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
            f[2 * hh] = v[0];
            f[2 * hh + 1] = v[1];
        }
        return f;
    };
    // O^T += V^T P^T; with clean, non-finite values count as 0
    auto add_values = [&](auto clean) {
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
#pragma unroll
            for (int e = 0; e < VG * XS; ++e) {
                u32x4_t f = vf[i / VG & 1][e];
                if constexpr (clean.value) f = finite_values(f);
                o[i + e / XS] = T::mfma(f, pf[e % XS], o[i + e / XS]);
            }
        }
    };
    in_acc(o);
    in_vgpr(qf);                                         // their wait is here, not in the loop

    // The inner loop has no branch that touches the output sums: one that did would move all of
    // them between register files in every iteration. A reference maximum that moves and a
    // masked score that is not finite leave the loop and come back.
    const int whole = first / KT;                        // tiles before this are seen whole by every row
    bool scored = false;                                 // tile t's scores are at hand
    for (int t = t0; t < t1;) {
        float top;
        bool odd = false;
        do {
            if (!scored) {
                stage(t);
                scores();
                if (t >= whole) {
#pragma unroll
                    for (int i = 0; i < T::NS; ++i) {
                        const float x = s[i / T::NO][i % T::NO];
                        const bool seen = t * KT + T::place(i, grp) < limit, fin = finite_f32(x);
                        // not finite: so is the key's row, or a query. A row that sees it gets NaN
                        odd |= !fin;
                        s[i / T::NO][i % T::NO] = seen ? (fin ? x : NAN) : -INFINITY;
                    }
                    odd = __any(odd);
                }
                top = largest();
                if (odd || __any(top > m + kSlack)) break;
            }
            weights(m == -INFINITY ? 0.0f : m);
            add_values(std::false_type());
            scored = false;
        } while (++t < t1);
        if (t >= t1) break;
        const float n = fmaxf(m, top);
        const float alpha = n == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - n);
        m = n;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < S::ND; ++i) {
            o[i] *= alpha;
            in_acc(o);
        }
        scored = !odd;
        if (odd) {                                       // rare
            weights(m == -INFINITY ? 0.0f : m);
            add_values(std::true_type());
            in_acc(o);
            ++t;
        }
    }
    l = row_sum<T>(l);
    wait_vmcnt<0>();
    lds_barrier();                                       // the ring is free again
}

template <typename T, int WR, int WD>
__global__ __launch_bounds__(THREADS) void latent_decode_kernel(DecodeArgs a) {
    typedef Shape<T, WR, WD> S;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE_BYTES + 4 * STAGES * 256];
    __shared__ int64_t sh[8];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = T::row(lane), grp = T::grp(lane);
    const int wr = wave % WR, d0 = (wave / WR) * (L / WD);

    const int64_t total = uniform(all_tiles(a, sh));
    const int grid = (int)min((int64_t)a.grid, total);
    if ((int)blockIdx.x >= grid) return;
    int64_t lo = run_start(total, grid, blockIdx.x);
    const int64_t hi = run_start(total, grid, blockIdx.x + 1);
    int req;
    int64_t base;
    find_request(a, lo, sh, req, base);
    bool leading = true;                                 // the run's first piece
    while (lo < hi) {
        const int len = uniform(request_len(a, req)), tiles = max(1, (len + KT - 1) / KT);
        const int g = (int)((lo - base) / tiles), t0 = (int)((lo - base) % tiles);
        const int t1 = (int)min((int64_t)tiles, t0 + (hi - lo));

        // this lane's row of the request: token j, head h; rows past the last repeat it
        const int r = g * S::MB + wr * T::ROWS + row;
        const int rc = min(r, a.rows - 1);
        const int j = rc / a.heads, h = rc % a.heads;
        const int64_t qr = (int64_t)req * a.tokens + j;
        const uint16_t *qp = a.q + qr * a.q_row + h * a.q_head;
        const int limit = max(0, len - a.tokens + j + 1);        // keys this row sees
        const int first = max(0, len - a.tokens + 1);            // keys that the request's first token sees
        typename T::acc_t o[S::ND];
        float m, l;
        run_tiles<T, WR, WD>(a, lds, qp, req, len, t0, t1, limit, first, o, m, l);
        const bool uncut = t0 == 0 && t1 == tiles;
        if (t0 == 0 && tid == 0)
            a.cuts[(int64_t)req * a.groups + g] = make_int2(
                2 * blockIdx.x + (leading ? 0 : 1), uncut ? (int)blockIdx.x : run_of(total, grid, lo + tiles - 1));
        if (uncut) {
            if (r < a.rows) {
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;   // no key: zeros
                uint16_t *op = a.out + qr * a.o_row + h * a.o_head;
#pragma unroll
                for (int i = 0; i < S::ND; ++i)
#pragma unroll
                    for (int x = 0; x < S::NO4; ++x) {
                        const u32x2_t v = {pack_bf16(o[i][4 * x] * inv, o[i][4 * x + 1] * inv),
                                           pack_bf16(o[i][4 * x + 2] * inv, o[i][4 * x + 3] * inv)};
                        *reinterpret_cast<u32x2_t *>(op + d0 + i * T::DIMS + T::place(4 * x, grp)) = v;
                    }
                if (a.lse && grp == 0 && wave / WR == 0)
                    a.lse[qr * a.heads + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;
            }
        } else {
            float *part = a.work + (2 * (int64_t)blockIdx.x + (leading ? 0 : 1)) * part_floats<S::MB>();
            f32x4_t *ps = reinterpret_cast<f32x4_t *>(part) + wave * (S::ND * S::NO4 * 64) + lane;
#pragma unroll
            for (int i = 0; i < S::ND; ++i)
#pragma unroll
                for (int x = 0; x < S::NO4; ++x)
                    ps[(i * S::NO4 + x) * 64] = f32x4_t{o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]};
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

// Joins the partial sums of the units that were cut between workgroups. A wave takes 64 float4 of a
// unit's sums, WP waves take its partials in turn and meet in LDS; each asks for 4 partials at
// once, since nothing but the latency of these loads bounds the kernel.
template <typename T, int WR, int WD, int WP>
__global__ __launch_bounds__(WP > 4 ? WP * 64 : 256) void latent_join_kernel(DecodeArgs a) {
    typedef Shape<T, WR, WD> S;
    constexpr int PER = S::MB * L / 4 / 64;              // waves' shares of a unit
    constexpr int QUADS = WP > 4 ? 1 : 4 / WP;           // of them, a workgroup's
    static_assert(PER % QUADS == 0, "whole workgroups a unit");
    __shared__ f32x4_t so[WP > 1 ? QUADS * WP : 1][64];
    __shared__ float sm[WP > 1 ? QUADS * WP : 1][64], sl[WP > 1 ? QUADS * WP : 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int unit = blockIdx.x / (PER / QUADS);
    const int quad = blockIdx.x % (PER / QUADS) * QUADS + wave / WP, turn = wave % WP;
    const int2 cut = a.cuts[unit];
    const int b0 = cut.x >> 1, pieces = cut.y - b0 + 1;
    if (pieces <= 1) return;
    const int req = unit / a.groups, g = unit % a.groups;

    // quad = (wave of the writer, 4-register group) in the partial's order; see the writer
    constexpr int PERW = S::ND * S::NO4;
    const int ww = quad / PERW, rest = quad % PERW, i = rest / S::NO4, x = rest % S::NO4;
    const int row = (ww % WR) * T::ROWS + T::row(lane);
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
    for (int j = turn; j < pieces; j += 4 * WP) {
        float pm[4], pl[4];
        f32x4_t po[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float *part = partial(min(j + u * WP, pieces - 1));
            pm[u] = part[(int64_t)S::MB * L + row];
            pl[u] = part[(int64_t)S::MB * (L + 1) + row];
            po[u] = reinterpret_cast<const f32x4_t *>(part)[(int64_t)quad * 64 + lane];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u * WP < pieces) merge(pm[u], pl[u], po[u]);
    }
    if constexpr (WP > 1) {
        so[wave][lane] = o;
        sm[wave][lane] = m;
        sl[wave][lane] = l;
        __syncthreads();
        if (turn) return;
        for (int u = 1; u < min(WP, pieces); ++u) merge(sm[wave + u][lane], sl[wave + u][lane], so[wave + u][lane]);
    }
    const int r = g * S::MB + row;
    if (r >= a.rows) return;
    const int64_t qr = (int64_t)req * a.tokens + r / a.heads;
    const int h = r % a.heads;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const u32x2_t y = {pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    const int dim = (ww / WR) * (L / WD) + i * T::DIMS + T::place(4 * x, T::grp(lane));
    *reinterpret_cast<u32x2_t *>(a.out + qr * a.o_row + h * a.o_head + dim) = y;
    if (a.lse && T::grp(lane) == 0 && ww / WR == 0 && rest == 0)
        a.lse[qr * a.heads + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int WR, int WD, int WP>
hipError_t launch_join(const DecodeArgs &a, hipStream_t stream) {
    constexpr int PER = Shape<T, WR, WD>::MB * L / 4 / 64, QUADS = WP > 4 ? 1 : 4 / WP;
    const unsigned blocks = (unsigned)((int64_t)a.batch * a.groups * (PER / QUADS));
    hipLaunchKernelGGL((latent_join_kernel<T, WR, WD, WP>), dim3(blocks), dim3(WP > 4 ? WP * 64 : 256), 0, stream, a);
    return hipGetLastError();
}

template <typename T, int WR, int WD>
hipError_t launch_shape(DecodeArgs a, hipStream_t stream) {
    a.cuts = reinterpret_cast<int2 *>(a.work + 2 * a.grid * part_floats<Shape<T, WR, WD>::MB>());
    hipLaunchKernelGGL((latent_decode_kernel<T, WR, WD>), dim3((unsigned)a.grid), dim3(THREADS), 0, stream, a);
    hipError_t err = hipGetLastError();
    // one workgroup takes every run whole: nothing to join
    if (err != hipSuccess || a.grid == 1) return err;
    // waves that share a unit's partials: about as many as it has on average
    const int64_t units = (int64_t)a.batch * a.groups;
    if (a.grid > 16 * units) return launch_join<T, WR, WD, 16>(a, stream);
    if (a.grid > 4 * units) return launch_join<T, WR, WD, 4>(a, stream);
    return launch_join<T, WR, WD, 1>(a, stream);
}

// Rows a workgroup for a request of `rows` query rows: the smallest shape that holds them.
int block_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

}  // namespace

int64_t latent_decode_workspace_bytes(int64_t batch, int64_t tokens, int64_t heads, int cus) {
    const int64_t rows = tokens * heads;
    if (batch == 0 || rows == 0) return 0;
    const int mb = block_rows(rows);
    return 2 * (int64_t)cus * mb * (L + 2) * (int64_t)sizeof(float) + batch * ((rows + mb - 1) / mb) * (int64_t)sizeof(int2);
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
    const int mb = block_rows(a.rows);
    a.groups = (a.rows + mb - 1) / mb;
    a.c = p.scale * kLog2e;
    // no more workgroups than the line can have tiles
    const int64_t most = (int64_t)a.batch * a.groups * std::max<int64_t>(1, (p.max_pages * p.page + KT - 1) / KT);
    a.grid = (int)std::min<int64_t>(cus, most);
    switch (mb) {
        case 16: return launch_shape<Tile16, 1, 4>(a, stream);
        case 32: return launch_shape<Tile32, 1, 4>(a, stream);
        case 64: return launch_shape<Tile32, 2, 2>(a, stream);
        default: return launch_shape<Tile32, 4, 1>(a, stream);
    }
}

}  // namespace skinny
