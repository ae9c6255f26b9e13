// latent_prefill.hip -- expanded latent attention of prompts: each head's own keys and values
// (128 numbers each) next to the 64 rotated numbers of a key that all heads share.
//
// Sequence i has queries cu_q[i] .. cu_q[i + 1] and keys cu_k[i] .. cu_k[i + 1]; per head
//     s = scale * (q[:128] . k + q[128:] . k_rot),   out = softmax(s) v,   lse = log sum exp(s);
// causal: the last query sees the last key, the one before it one key fewer, and so on.
//
// What bounds it: the matrix cores (2 * 320 operations a query-key pair and head) and beside
// them the exponentials. A workgroup of 4 waves holds 128 query rows of one head, 32 a wave, in
// registers, and reads keys and values in tiles of 64 through two LDS stages of 40 KB; two
// workgroups share a CU, so that one's softmax runs beside the other's matrix instructions.
// Where the queries are too few to fill the chip, a row's keys are split over several
// workgroups and their partial sums joined by a second kernel. Long sequences go to the wide form
// below. Measured: 6 prompts of 217 .. 1294 tokens x 32 heads 72 us (144 MB at least: 2 TB/s, 480
// TFLOP/s; not causal 103 us, 670 TFLOP/s), 16 prompts of about 256 42 us (3.6 TB/s), one prompt of 129 x
// 8 heads 9.5 us. Beside its matrix instructions (27% of the cycles with the 6 prompts) a tile waits for
// all its loads, and each matrix instruction for its fragment from LDS, which is not read ahead as in the wide form.
#include <algorithm>
#include <type_traits>

#include "latent.hpp"

namespace skinny {
namespace {

using namespace latent;
typedef Tile32 T;

constexpr int HD = 128, ROT = 64, DQ = HD + ROT;
constexpr int WAVES = 4, THREADS = WAVES * 64;
constexpr int BM = WAVES * T::ROWS;          // query rows a workgroup
constexpr int KT = 64;                       // keys a tile
constexpr int KSEG = DQ * 2 / 128, VSEG = HD * 2 / 128;
constexpr int K_BYTES = KT * DQ * 2, STAGE_BYTES = K_BYTES + KT * HD * 2;
constexpr int STAGES = 2;
constexpr int KS = DQ / T::KSTEP;            // K steps of the score product
constexpr int ND = HD / T::DIMS;             // dim tiles of the output
constexpr int NT = KT / T::ROWS;             // key subtiles
constexpr int NP = NT * T::NS;               // weights a lane holds

// the place in a tile of a lane's weight j, counted from its first
__host__ __device__ constexpr int place0(int j) { return j / T::NS * T::ROWS + 8 * (j % T::NS >> 2) + (j & 3); }

struct PrefillArgs {
    const uint16_t *q, *k, *v, *kr;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, kr_row;
    const int32_t *cu_q, *cu_k;
    uint16_t *out;
    int64_t o_row, o_head;
    float *lse;
    float *work;                             // split: per split, row and head: 128 sums, then maximum, total
    int64_t nq, nk;
    int batch, heads, tiles, splits;         // tiles: most query tiles that nq rows in batch sequences can need
    int average;                             // keys a sequence
    float c;
    bool causal;
};

// One row's partial: 128 sums; maxima and totals follow all rows' sums.
__host__ __device__ inline int64_t split_floats(int64_t nq, int64_t heads) { return nq * heads * (HD + 2); }

// cu[i], never outside 0 .. n
__device__ __forceinline__ int start(const int32_t *cu, int i, int64_t n) { return (int)min((int64_t)max(cu[i], 0), n); }

// v's sum over the lanes up to this one: within rows of 16 lanes, then over the rows.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);      // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);      // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);      // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);      // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);      // row_bcast:15 to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);      // row_bcast:31 to rows 2 and 3
    return v;
}

// The sequence and its query tile that are number `at` of all: first the tiles that see more keys
// than sequences have on average, then the others, each sequence's from its last, so that a long
// prompt among short ones does not start last (4000 tokens before 30 x 200, 16 heads: 162 -> 123 us;
// all in order of their keys costs short prompts 1 us a workgroup to find). Sequence -1: there
// are fewer.
template <int BM>
__device__ __forceinline__ int find_tile(const PrefillArgs &a, int at, int &tile) {
    const int lane = threadIdx.x & 63;
    auto rows = [&](int i) { return i < a.batch ? max(0, start(a.cu_q, i + 1, a.nq) - start(a.cu_q, i, a.nq)) : 0; };
    if (a.batch == 1) {
        tile = (rows(0) + BM - 1) / BM - 1 - at;
        return tile >= 0 ? 0 : -1;
    }
    for (int rest = 0; rest < 2; ++rest) {
        for (int i0 = 0; i0 < a.batch; i0 += 64) {
            const int i = i0 + lane, lq = rows(i), all = (lq + BM - 1) / BM;
            const int lk = i < a.batch ? max(0, start(a.cu_k, i + 1, a.nk) - start(a.cu_k, i, a.nk)) : 0;
            // its tiles with more keys than the average: all, or from the one of the first such row on
            const int from = a.causal ? max(0, a.average - (lk - lq)) / BM : 0;
            const int most = lk > a.average ? all - from : 0;
            const int n = rest ? all - most : most, skip = rest ? most : 0;
            const int s = wave_scan(n);
            const uint64_t past = __ballot(s > at);
            if (past) {
                const int w = __builtin_ctzll(past);
                tile = __builtin_amdgcn_readlane(all - 1 - skip + (s - n), w) - at;
                return i0 + w;
            }
            at -= __builtin_amdgcn_readlane(s, 63);
        }
    }
    return -1;
}

// One pass over key tiles [t0, t1). limit: keys that the lane's row sees; first: the fewest that
// any row of the workgroup sees. safe: non-finite values in tiles that some row sees in part
// reach only the rows that see them (see split_value).
__device__ __forceinline__ void run_tiles(const PrefillArgs &a, uint8_t *lds, const u32x4_t (&qf)[KS], int head,
                                          int64_t k0row, int lk, int t0, int t1, int limit, int first, bool safe,
                                          f32x16_t (&o)[ND], float &m, float &l) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = T::row(lane), grp = T::grp(lane);
    lds_u8 *ring = (lds_u8 *)lds;

    // staging: wave w takes the 8-row groups 2w and 2w + 1 of a tile. Rows past the last key
    // repeat it (their scores are masked)
    auto issue = [&](int t) {
        lds_u8 *st = ring + (t & 1) * STAGE_BYTES;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int rg = 2 * wave + u, r = 8 * rg + (lane >> 3);
            const int chunk = ((lane & 7) ^ swz(r)) * 8;
            const int64_t key = k0row + min(t * KT + r, lk - 1);
            const uint16_t *kp = a.k + key * a.k_row + head * a.k_head + chunk;
            const uint16_t *rp = a.kr + key * a.kr_row + chunk;
            const uint16_t *vp = a.v + key * a.v_row + head * a.v_head + chunk;
            const int kd = lds_address(st + rg * (KSEG * 1024)), vd = lds_address(st + K_BYTES + rg * (VSEG * 1024));
            load_lds_pieces<2>(kp, kd);
            load_lds_pieces<1>(rp, kd + 2048);
            load_lds_pieces<2>(vp, vd);
        }
    };
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int j = 0; j < T::NO; ++j) o[i][j] = 0.0f;
    m = -INFINITY;
    l = 0.0f;
    // fragment places within a stage, with the swizzle worked out once: see latent_decode.hip
    int koff[4], voff[2][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        koff[j] = (row >> 3) * (KSEG * 1024) + (row & 7) * 128 + (((2 * j + grp) ^ swz(row)) << 4);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = 8 * hh + 4 * grp + ((lane & 15) >> 2);
            const int ch = 4 * j + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            voff[j][hh] = K_BYTES + hh * (VSEG * 1024) + (r & 7) * 128 + ((ch ^ swz(r)) << 4) + (lane & 1) * 8;
        }
    if (t0 < t1) issue(t0);
    for (int t = t0; t < t1; ++t) {
        wait_vmcnt<0>();
        lds_barrier();                       // tile t is staged, the other stage is free
        if (t + 1 < t1) issue(t + 1);
        lds_u8 *st = ring + (t & 1) * STAGE_BYTES;
        f32x16_t s[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int j = 0; j < T::NO; ++j) s[u][j] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const u32x4_t kf = *(const lds_u32x4 *)(st + koff[k % 4] + u * (T::ROWS / 8) * (KSEG * 1024) +
                                                        (k / 4) * 1024);
                s[u] = T::mfma(kf, qf[k], s[u]);
            }
        }
        float p[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) p[i] = s[i / T::NS][i % T::NS];
        const int k0 = t * KT;
        const bool mixed = k0 + KT > first;
        if (mixed) {
            const int left = limit - k0 - T::place(0, grp);      // keys from the lane's first on
#pragma unroll
            for (int i = 0; i < NP; ++i) p[i] = place0(i) < left ? p[i] : -INFINITY;
        }
        float top = p[0];
#pragma unroll
        for (int i = 1; i < NP; ++i) top = fmaxf(top, p[i]);
        top = row_max<T>(top) * a.c;
        if (__any(top > m + kSlack)) {
            const float n = fmaxf(m, top);
            const float alpha = n == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - n);
            m = n;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
                for (int j = 0; j < T::NO; ++j) o[i][j] *= alpha;
        }
        const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], a.c, -mu));
            l += p[i];
        }
        // weights are rounded to bf16 for the matrix product, whose operands are of one type (by 2^-8
        // relative at most, independently of each other: an output's error grows from the 0.0016 of
        // its own rounding to 0.0019 .. 0.0023); their sum l is of the unrounded ones
        u32x4_t pf[NP / 8];
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) pf[i / 4][i % 4] = pack_bf16(p[2 * i], p[2 * i + 1]);
        auto value = [&](int i, int x) {     // dim tile i, 16 keys x
            u32x4_t f;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                lds_u8 *at = st + voff[i % 2][hh] + (i / 2) * 1024 + 2 * x * (VSEG * 1024);
                const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)at));
                f[2 * hh] = v[0];
                f[2 * hh + 1] = v[1];
            }
            return f;
        };
        if (!(mixed && safe)) {
#pragma unroll
            for (int x = 0; x < NP / 8; ++x)
#pragma unroll
                for (int i = 0; i < ND; ++i) o[i] = T::mfma(value(i, x), pf[x], o[i]);
        } else {
            u32x4_t see[NP / 8];
#pragma unroll
            for (int j = 0; j < NP; j += 2)
                see[j / 8][j % 8 / 2] = seen_pair(place0(j) < limit - k0 - T::place(0, grp),
                                                  place0(j + 1) < limit - k0 - T::place(0, grp));
#pragma unroll
            for (int x = 0; x < NP / 8; ++x)
#pragma unroll
                for (int i = 0; i < ND; ++i) {
                    u32x4_t g, a1, a2;
                    split_value(value(i, x), g, a1, a2);
                    o[i] = T::mfma(g, pf[x], o[i]);
                    o[i] = T::mfma(a1, see[x], o[i]);
                    o[i] = T::mfma(a2, see[x], o[i]);
                }
        }
    }
    l = row_sum<T>(l);
    lds_barrier();
}

// Whether the flag is set in any lane of the workgroup (in the ring's memory: two workgroups'
// rings are all of a CU's LDS). The ring is free before and after.
template <int N>
__device__ __forceinline__ bool any_wave(bool flag, uint8_t *lds) {
    volatile int *w = reinterpret_cast<volatile int *>(lds);
    const bool mine = __any(flag);
    if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = mine;
    __syncthreads();
    int any = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) any |= w[i];
    __syncthreads();
    return any;
}

// What workgroup blockIdx.x works on: split of the keys, head, query tile by its number in the order
// of find_tile. Long ones come first, whatever the head, so that the chip is full to the end (8192
// tokens x 32 heads: 10% fewer cycles than one head after the other). Workgroups go
// to the XCDs in turn; where the heads divide evenly over them an XCD takes whole heads, so that its
// L2 holds the keys and values that its workgroups read at about the same time.
__device__ __forceinline__ void block_order(const PrefillArgs &a, int &split, int &head, int &at) {
    int b = blockIdx.x;
    split = b % a.splits;
    b /= a.splits;
    if (a.heads % 8 == 0 && a.splits == 1) {
        const int j = b >> 3, own = a.heads / 8;
        head = (b & 7) + 8 * (j % own);
        at = j / own;
    } else {
        head = b % a.heads;
        at = b / a.heads;
    }
}

// A row's results: the output and lse, or its split's partial. The two lanes of a row trade halves, for
// 16-byte stores (6 prompts of 217 .. 1294 tokens x 32 heads: 75 us with 8-byte ones, 69 with these;
// whole rows by way of LDS are no faster).
__device__ __forceinline__ void put_row(const PrefillArgs &a, int split, int64_t qr, int head, int grp,
                                        const f32x16_t (&o)[ND], float m, float l) {
    if (a.splits == 1) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;          // no key: zeros
        uint16_t *op = a.out + qr * a.o_row + head * a.o_head;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int x = 0; x < T::NO / 4; x += 2) {
                const auto p = __builtin_amdgcn_permlane32_swap(pack_bf16(o[i][4 * x] * inv, o[i][4 * x + 1] * inv),
                                                                pack_bf16(o[i][4 * x + 4] * inv, o[i][4 * x + 5] * inv), false, false);
                const auto q = __builtin_amdgcn_permlane32_swap(pack_bf16(o[i][4 * x + 2] * inv, o[i][4 * x + 3] * inv),
                                                                pack_bf16(o[i][4 * x + 6] * inv, o[i][4 * x + 7] * inv), false, false);
                *reinterpret_cast<u32x4_t *>(op + i * T::DIMS + 8 * (x + grp)) = u32x4_t{p[0], q[0], p[1], q[1]};
            }
        if (a.lse && grp == 0) a.lse[qr * a.heads + head] = (m + __builtin_amdgcn_logf(l)) * kLn2;
    } else {
        const int64_t at_row = qr * a.heads + head, all = a.nq * a.heads;
        float *part = a.work + split * split_floats(a.nq, a.heads);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int x = 0; x < T::NO / 4; ++x)
                *reinterpret_cast<f32x4_t *>(part + at_row * HD + i * T::DIMS + T::place(4 * x, grp)) =
                    f32x4_t{o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]};
        if (grp == 0) {
            part[all * HD + at_row] = m;
            part[all * (HD + 1) + at_row] = l;
        }
    }
}

__device__ __forceinline__ bool not_finite(const f32x16_t (&o)[ND]) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int j = 0; j < T::NO; ++j) odd |= !finite_f32(o[i][j]);
    return odd;
}

__global__ __launch_bounds__(THREADS, 2) void latent_prefill_kernel(PrefillArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * STAGE_BYTES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = T::row(lane), grp = T::grp(lane);
    int split, head, at;
    block_order(a, split, head, at);
    int tile = 0;
    int seq = find_tile<BM>(a, at, tile);
    if (seq < 0) return;
    asm volatile("" : "+v"(seq), "+v"(tile));            // as scalars, they and what follows crowd the scalar registers
    const int q0 = start(a.cu_q, seq, a.nq), lq = start(a.cu_q, seq + 1, a.nq) - q0;
    const int k0 = start(a.cu_k, seq, a.nk), lk = max(0, start(a.cu_k, seq + 1, a.nk) - k0);
    const int r = tile * BM + wave * T::ROWS + row, rc = min(r, lq - 1);

    u32x4_t qf[KS];
    const uint16_t *qp = a.q + ((int64_t)q0 + rc) * a.q_row + head * a.q_head + grp * 8;
#pragma unroll
    for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const u32x4_t *>(qp + k * T::KSTEP);

    // keys that this row, the workgroup's first row and its last row see
    auto sees = [&](int x) { return a.causal ? max(0, min(lk, lk - lq + 1 + x)) : lk; };
    const int limit = sees(rc), first = sees(tile * BM), last = sees(min(tile * BM + BM, lq) - 1);
    const int n = (last + KT - 1) / KT;
    const int t0 = (int)((int64_t)n * split / a.splits), t1 = (int)((int64_t)n * (split + 1) / a.splits);
    f32x16_t o[ND];
    float m, l;
    bool safe = false;
    for (;;) {
        run_tiles(a, lds, qf, head, k0, lk, t0, t1, limit, first, safe, o, m, l);
        // a non-finite result where some rows see fewer keys than others: once more, key by key
        if (safe || !any_wave<WAVES>(not_finite(o) && t1 * KT > first, lds)) break;
        safe = true;
    }
    if (r < lq) put_row(a, split, (int64_t)q0 + r, head, grp, o, m, l);
}

// ---- the wide form: 256 query rows a workgroup --------------------------------------------
// 8 waves of 32 rows, two on each SIMD, that take turns: while waves 0 .. 3 run the matrix
// instructions of a tile (the value product of the tile before, then its score product), waves
// 4 .. 7 run their softmax, and the other way round; a barrier ends each turn. Left to themselves
// two waves of a SIMD fall into step, and then neither hides the other (measured with the narrow
// form at 8192 tokens x 32 heads: matrix and vector time add up, 675 us). Keys and
// values are staged four tiles deep, all of a CU's LDS. Measured there: 607 us, 1130 TFLOP/s; the
// matrix cores are busy for 59% of the cycles, at the 1.75 GHz that the power limit leaves (a
// library product of 16384^3 reaches 1600 TFLOP/s); not causal, 4096 tokens x 32 heads, 314 us, 1090
// TFLOP/s. One wave a SIMD with 64 rows, which reads LDS
// half as often, takes 787 us: it has to issue all vector and matrix instructions by itself.
constexpr int WIDE_WAVES = 8, WIDE_THREADS = WIDE_WAVES * 64, WIDE_BM = WIDE_WAVES * T::ROWS;
constexpr int V_BYTES = KT * HD * 2, K_RING = 4, V_RING = 4;
constexpr int WIDE_LDS = K_RING * K_BYTES + V_RING * V_BYTES;
constexpr int GROUP_LOADS = KSEG + VSEG;                 // a wave's, of a tile's keys and a tile's values
static_assert(WIDE_WAVES * 8 == KT, "a wave stages 8 rows");

__global__ __launch_bounds__(WIDE_THREADS) void latent_prefill_wide_kernel(PrefillArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[WIDE_LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int row = T::row(lane), grp = T::grp(lane);
    int split, head, at, tile = 0;
    block_order(a, split, head, at);
    const int seq = find_tile<WIDE_BM>(a, at, tile);
    if (seq < 0) return;
    const int q0 = uniform(start(a.cu_q, seq, a.nq)), lq = uniform(start(a.cu_q, seq + 1, a.nq)) - q0;
    const int k0 = uniform(start(a.cu_k, seq, a.nk)), lk = max(0, uniform(start(a.cu_k, seq + 1, a.nk)) - k0);
    tile = uniform(tile);
    const int r0 = tile * WIDE_BM + wave * T::ROWS;      // the wave's first row
    auto sees = [&](int x) __attribute__((always_inline)) { return a.causal ? max(0, min(lk, lk - lq + 1 + x)) : lk; };
    const int r = r0 + row, rc = min(r, lq - 1);
    const int64_t qr = (int64_t)q0 + rc;
    const int limit = sees(rc);
    // key tiles: the workgroup's, and of them the wave's; whole: seen whole by every row of the wave
    const int n = (sees(min(tile * WIDE_BM + WIDE_BM, lq) - 1) + KT - 1) / KT;
    const int t0 = (int)((int64_t)n * split / a.splits), t1 = (int)((int64_t)n * (split + 1) / a.splits);
    const int cnt = t1 - t0;
    const int last = r0 < lq ? (sees(min(r0 + T::ROWS, lq) - 1) + KT - 1) / KT : 0;
    const int cw = max(0, min(last, t1) - t0), first = sees(min(r0, lq - 1));
    const int whole = max(0, first / KT - t0);

    lds_u8 *kring = (lds_u8 *)lds, *vring = kring + K_RING * K_BYTES;
    const int lrow = 8 * wave + (lane >> 3);             // staging: this lane's row of a tile
    const int chunk = ((lane & 7) ^ swz(lrow)) * 8;
    const uint16_t *kbase = a.k + head * a.k_head + chunk, *rbase = a.kr + chunk, *vbase = a.v + head * a.v_head + chunk;
    // past the last tile it is loaded again, so that the counts stay even
    auto key_of = [&](int i) __attribute__((always_inline)) { return (int64_t)k0 + min(min(t0 + i, t1 - 1) * KT + lrow, lk - 1); };
    auto load = [&](int i) __attribute__((always_inline)) {
        const int64_t key = key_of(i);
        const int kd = lds_address(kring + (i % K_RING) * K_BYTES + wave * (KSEG * 1024));
        load_lds_pieces<2>(kbase + key * a.k_row, kd);
        load_lds_pieces<1>(rbase + key * a.kr_row, kd + 2048);
        load_lds_pieces<2>(vbase + key * a.v_row, lds_address(vring + (i % V_RING) * V_BYTES + wave * (VSEG * 1024)));
    };
    int koff[4], voff[2][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        koff[j] = (row >> 3) * (KSEG * 1024) + (row & 7) * 128 + (((2 * j + grp) ^ swz(row)) << 4);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int x = 8 * hh + 4 * grp + ((lane & 15) >> 2);
            const int ch = 4 * j + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            voff[j][hh] = hh * (VSEG * 1024) + (x & 7) * 128 + ((ch ^ swz(x)) << 4) + (lane & 1) * 8;
        }

    u32x4_t qf[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k)
        qf[k] = *reinterpret_cast<const u32x4_t *>(a.q + qr * a.q_row + head * a.q_head + k * T::KSTEP + grp * 8);
    f32x16_t o[ND], s[NT];
    float m, l;
    u32x4_t pf[NP / 8];

    auto softmax = [&](int i) __attribute__((always_inline)) {
        if (i >= whole) {
            const int left = limit - (t0 + i) * KT - T::place(0, grp);   // keys from the lane's first on
#pragma unroll
            for (int j = 0; j < NP; ++j)
                s[j / T::NS][j % T::NS] = place0(j) < left ? s[j / T::NS][j % T::NS] : -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int j = 1; j < NP; ++j) top = fmaxf(top, s[j / T::NS][j % T::NS]);
        top = row_max<T>(top) * a.c;
        if (__any(top > m + kSlack)) {
            const float next = fmaxf(m, top);
            const float alpha = next == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= alpha;
        }
        // weights are rounded to bf16 for the matrix product, see run_tiles
        const float mu = m == -INFINITY ? 0.0f : m;
        float p[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            p[j] = __builtin_amdgcn_exp2f(fmaf(s[j / T::NS][j % T::NS], a.c, -mu));
            l += p[j];
        }
#pragma unroll
        for (int j = 0; j < NP / 2; ++j) pf[j / 4][j % 4] = pack_bf16(p[2 * j], p[2 * j + 1]);
    };
    // Places of a staged tile's fragments, one register each; the rest of an address is in the
    // instruction. (Held in a register so that the compiler does not keep one for every fragment.)
    auto place_of = [&](lds_u8 *st, int off) __attribute__((always_inline)) {
        int at = (int)(uintptr_t)st + off;
        asm volatile("" : "+v"(at));
        return (lds_u8 *)(uintptr_t)(uint32_t)at;
    };
    lds_u8 *kat[4], *vat[2][2];
    auto find_keys = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) kat[j] = place_of(kring + (i % K_RING) * K_BYTES, koff[j]);
    };
    auto find_values = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) vat[j / 2][j % 2] = place_of(vring + (i % V_RING) * V_BYTES, voff[j / 2][j % 2]);
    };
    auto value = [&](int d, int x) __attribute__((always_inline)) {      // dim tile d, 16 keys x
        u32x4_t f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            lds_u8 *p = vat[d % 2][hh] + (d / 2) * 1024 + 2 * x * (VSEG * 1024);
            const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
            f[2 * hh] = v[0];
            f[2 * hh + 1] = v[1];
        }
        return f;
    };
    // Matrix instructions of a turn: the value product of the tile before (O^T += V^T P^T), the
    // score product of this one (S^T = K Q^T), or both. Fragments are read from LDS a group ahead
    // (a read takes some 130 cycles, more when four waves read; an instruction takes 32), the
    // first group of the value product before the turn; the scheduling barriers keep the groups
    // apart.
    constexpr int G = 8, NV = NP / 8 * ND, NK = KS * NT;
    static_assert(NV % G == 0 && NK % G == 0, "whole groups");
    u32x4_t f[2][G];
    auto key_group = [&](int g) __attribute__((always_inline)) {
#pragma unroll
        for (int e = g * G; e < g * G + G; ++e)
            f[g & 1][e % G] = *(const lds_u32x4 *)(kat[e / NT % 4] + e % NT * (T::ROWS / 8) * (KSEG * 1024) + e / NT / 4 * 1024);
    };
    auto value_group = [&](int g) __attribute__((always_inline)) {
#pragma unroll
        for (int e = g * G; e < g * G + G; ++e) f[g & 1][e % G] = value(e % ND, e / ND);
    };
    static_assert(NV / G % 2 == 0, "the key groups follow in the other half of f");
    auto value_products = [&](bool keys_follow) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < NV / G; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            if (g + 1 < NV / G) value_group(g + 1);
            else if (keys_follow) key_group(0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = g * G; e < g * G + G; ++e) o[e % ND] = T::mfma(f[g & 1][e % G], pf[e / ND], o[e % ND]);
        }
    };
    auto score_products = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < NK / G; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            if (g + 1 < NK / G) key_group(g + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = g * G; e < g * G + G; ++e)
                s[e % NT] = T::mfma(f[g & 1][e % G], qf[e / NT], e / NT ? s[e % NT] : f32x16_t{0.0f});
        }
    };
    // the value product where a value that is not finite may reach only the rows that see it
    auto value_products_carefully = [&](int i) __attribute__((always_inline)) {
        const int left = limit - (t0 + i) * KT - T::place(0, grp);
#pragma unroll
        for (int x = 0; x < NP / 8; ++x) {
            u32x4_t see;
#pragma unroll
            for (int j = 0; j < 8; j += 2) see[j / 2] = seen_pair(place0(8 * x + j) < left, place0(8 * x + j + 1) < left);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                __builtin_amdgcn_sched_barrier(0);
                u32x4_t g, a1, a2;
                split_value(value(d, x), g, a1, a2);
                o[d] = T::mfma(g, pf[x], o[d]);
                o[d] = T::mfma(a1, see, o[d]);
                o[d] = T::mfma(a2, see, o[d]);
            }
        }
    };
    // Turns. Waves 0 .. 3 have their matrix turn of tile i in turn 2i of the workgroup and their
    // softmax turn in 2i + 1, the later ones each one turn after. A wave loads its share of a tile's
    // keys and values at the start of its softmax turn of two (the later waves: three) tiles before
    // and waits for it at the end of the next one, whose barrier shows it to all in time. The
    // stages filled held a tile that both groups are done with.
    const bool later = wave >= WIDE_WAVES / 2;
    auto next_turn = [&]() __attribute__((always_inline)) {
        wait_vmcnt<GROUP_LOADS>();
        lds_barrier();
    };
    auto pass = [&](auto careful) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] = f32x16_t{0.0f};
        m = -INFINITY;
        l = 0.0f;
        if (cnt <= 0) return;
        for (int i = 0; i < (later ? 3 : 2); ++i) load(i);
        in_vgpr(qf);                                     // their wait is here, not in the loop
        wait_vmcnt<0>();
        lds_barrier();
        if (later) lds_barrier();
        if (cw > 0) {
            find_keys(0);
            key_group(0);
            score_products();
            next_turn();
            load(later ? 3 : 2);
            softmax(0);
            find_values(0);
            if constexpr (!careful.value) value_group(0);
            next_turn();
        }
        for (int i = 1; i < cw; ++i) {
            find_keys(i);
            __builtin_amdgcn_s_setprio(1);
            if constexpr (careful.value) {
                value_products_carefully(i - 1);
                key_group(0);
            } else {
                value_products(true);
            }
            score_products();
            __builtin_amdgcn_s_setprio(0);
            next_turn();
            load(later ? i + 3 : i + 2);
            softmax(i);
            find_values(i);
            if constexpr (!careful.value) value_group(0);
            next_turn();
        }
        if (cw > 0) {
            if constexpr (careful.value) value_products_carefully(cw - 1);
            else value_products(false);
        }
        for (int i = cw; i < cnt; ++i) {                 // tiles that this wave's rows do not see
            next_turn();
            load(later ? i + 3 : i + 2);
            next_turn();
        }
        if (!later) lds_barrier();
        l = row_sum<T>(l);
        wait_vmcnt<0>();
        lds_barrier();
    };
    pass(std::false_type());
    // a non-finite result where some rows see fewer keys than others: once more, with care
    if (any_wave<WIDE_WAVES>(not_finite(o) && t1 * KT > sees(tile * WIDE_BM), lds)) pass(std::true_type());
    if (r < lq) put_row(a, split, qr, head, grp, o, m, l);
}

// Joins the splits of a row and head: 32 lanes, 4 numbers each.
__global__ __launch_bounds__(256) void latent_prefill_join_kernel(PrefillArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), all = a.nq * a.heads;
    const int x = threadIdx.x & 31;
    if (at >= all) return;
    float m = -INFINITY, l = 0.0f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) {
        const float *part = a.work + s * split_floats(a.nq, a.heads);
        const float pm = part[all * HD + at], pl = part[all * (HD + 1) + at];
        const f32x4_t po = *reinterpret_cast<const f32x4_t *>(part + at * HD + 4 * x);
        const float n = fmaxf(m, pm);
        const float ca = m == n ? 1.0f : __builtin_amdgcn_exp2f(m - n);
        const float cb = pm == n ? 1.0f : __builtin_amdgcn_exp2f(pm - n);
        m = n;
        l = l * ca + pl * cb;
        o = o * ca + po * cb;
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    const int64_t qr = at / a.heads, head = at % a.heads;
    *reinterpret_cast<u32x2_t *>(a.out + qr * a.o_row + head * a.o_head + 4 * x) =
        u32x2_t{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    if (a.lse && x == 0) a.lse[at] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// How a call of these sizes runs. The wide form where sequences have rows to fill it and keys enough
// for its longer start (causal, 32 heads, wide and narrow in us: 16 prompts of 256 48 and 43, 8 of 512
// 51 and 50, 8 of 1024 130 and 138, 2 of 2048 92 and 105, 4 chunks of 300 after 4000 keys 136 and 168).
struct Plan {
    bool wide;
    int64_t tiles;                           // most query tiles that nq rows in batch sequences can need
    int splits;
};
Plan plan(int64_t nq, int64_t nk, int64_t batch, int64_t heads, int cus) {
    Plan p;
    p.wide = nq / batch >= 192 && nk / batch >= 1024;
    const int bm = p.wide ? WIDE_BM : BM;
    p.tiles = std::min(nq, (nq + batch * (bm - 1)) / bm);
    // Splits of the keys: as many as fill the CUs (one wide workgroup each, or two narrow ones),
    // while each keeps 8 key tiles of the average sequence (1024 rows x 16024 keys x 8 heads: 8 splits
    // 89 us, none 392)
    const int64_t room = (p.wide ? 1 : 2) * (int64_t)cus / std::max<int64_t>(1, p.tiles * heads);
    const int64_t most = std::max<int64_t>(1, nk / batch / (8 * KT));
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({room, most, 32}));
    return p;
}

}  // namespace

int64_t latent_prefill_workspace_bytes(int64_t nq, int64_t nk, int64_t batch, int64_t heads, int cus) {
    if (nq == 0 || batch == 0 || heads == 0) return 0;
    const int s = plan(nq, nk, batch, heads, cus).splits;
    return s == 1 ? 0 : s * split_floats(nq, heads) * (int64_t)sizeof(float);
}

hipError_t launch_latent_prefill(const skinny_latent_prefill_args &p, int cus, hipStream_t stream) {
    PrefillArgs a;
    a.q = static_cast<const uint16_t *>(p.q);
    a.k = static_cast<const uint16_t *>(p.k);
    a.v = static_cast<const uint16_t *>(p.v);
    a.kr = static_cast<const uint16_t *>(p.k_rot);
    a.q_row = p.q_row_stride;
    a.q_head = p.q_head_stride;
    a.k_row = p.k_row_stride;
    a.k_head = p.k_head_stride;
    a.v_row = p.v_row_stride;
    a.v_head = p.v_head_stride;
    a.kr_row = p.k_rot_stride;
    a.cu_q = p.cu_q;
    a.cu_k = p.cu_k;
    a.out = static_cast<uint16_t *>(p.out);
    a.o_row = p.out_row_stride;
    a.o_head = p.out_head_stride;
    a.lse = p.lse;
    a.work = static_cast<float *>(p.workspace);
    a.nq = p.nq;
    a.nk = p.nk;
    a.batch = (int)p.batch;
    a.heads = (int)p.heads;
    const Plan how = plan(p.nq, p.nk, p.batch, p.heads, cus);
    a.tiles = (int)how.tiles;
    a.average = (int)(p.nk / p.batch);
    a.splits = how.splits;
    a.c = p.scale * kLog2e;
    a.causal = p.causal != 0;
    const dim3 grid((unsigned)(a.tiles * a.heads * a.splits));
    if (how.wide)
        hipLaunchKernelGGL(latent_prefill_wide_kernel, grid, dim3(WIDE_THREADS), 0, stream, a);
    else
        hipLaunchKernelGGL(latent_prefill_kernel, grid, dim3(THREADS), 0, stream, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.splits == 1) return err;
    hipLaunchKernelGGL(latent_prefill_join_kernel, dim3((unsigned)((p.nq * a.heads + 7) / 8)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace skinny
