// latent_append.hip -- new tokens' rows into a paged latent cache, and their queries' positions.
//
// Per token: z = x / sqrt(mean(x^2) + eps) * w over the 512 latents (or x as it is, without a
// weight), r = the shared key's 64 numbers turned by the token's position; [z, r] goes to its
// slot. The rotated part of every head's query is turned by the same angles in the same pass.
//
// What bounds it: bytes (each number is read and written once); at few tokens, latency. A wave
// takes one token and a run of its heads, 8 heads at a time (8 lanes a head, 16 bytes a lane);
// lane k of the 8 holds the 4 pairs of frequencies 4k .. 4k + 3 in either order of pairs, so
// its cosines and sines stay in registers for all heads. Angles are taken in 64 bits (positions
// are many turns), one a lane for half the wave, and handed round by lane reads. Measured: 8191 tokens
// x 128 heads 61 us (287 MB, 4.7 TB/s; a large copy reaches 4.9), one token x 8 heads 2.6 us, of
// which the launch is most.
#include <algorithm>

#include "latent.hpp"

namespace skinny {
namespace {

using namespace latent;

constexpr int L = 512, ROT = 64;
constexpr int WAVES = 4;

struct AppendArgs {
    const uint16_t *kv;
    int64_t kv_row;
    uint16_t *cache;
    int64_t c_page, c_row;
    const int64_t *slots, *positions;
    const double *inv_freq;
    const uint16_t *weight;                  // NULL: latents are stored as they are
    float eps;
    const uint16_t *q;                       // NULL: no queries
    int64_t q_row, q_head;
    uint16_t *q_out;
    int64_t qo_row, qo_head;
    int64_t n, pages;
    int heads, page, chunk;                  // chunk: heads a wave, a multiple of 8
    bool interleaved;
};

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// The 8 numbers of lane k of a head: 4 neighbouring pairs, or 4 places of each half.
__device__ __forceinline__ u32x4_t load_pairs(const uint16_t *x, int k, bool interleaved) {
    if (interleaved) return *reinterpret_cast<const u32x4_t *>(x + 8 * k);
    const u32x2_t a = *reinterpret_cast<const u32x2_t *>(x + 4 * k);
    const u32x2_t b = *reinterpret_cast<const u32x2_t *>(x + ROT / 2 + 4 * k);
    return u32x4_t{a[0], a[1], b[0], b[1]};
}
__device__ __forceinline__ u32x4_t turn(u32x4_t v, const float (&c)[4], const float (&s)[4], bool interleaved) {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = interleaved ? lo_f32(v[i]) : (i & 1) ? hi_f32(v[i / 2]) : lo_f32(v[i / 2]);
        b[i] = interleaved ? hi_f32(v[i]) : (i & 1) ? hi_f32(v[2 + i / 2]) : lo_f32(v[2 + i / 2]);
    }
    float y[4], z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = a[i] * c[i] - b[i] * s[i];
        z[i] = b[i] * c[i] + a[i] * s[i];
    }
    if (interleaved)
        return u32x4_t{pack_bf16(y[0], z[0]), pack_bf16(y[1], z[1]), pack_bf16(y[2], z[2]), pack_bf16(y[3], z[3])};
    return u32x4_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
}
__device__ __forceinline__ void store_pairs(uint16_t *x, int k, u32x4_t v, bool interleaved) {
    if (interleaved) {
        *reinterpret_cast<u32x4_t *>(x + 8 * k) = v;
    } else {
        *reinterpret_cast<u32x2_t *>(x + 4 * k) = u32x2_t{v[0], v[1]};
        *reinterpret_cast<u32x2_t *>(x + ROT / 2 + 4 * k) = u32x2_t{v[2], v[3]};
    }
}

__global__ __launch_bounds__(WAVES * 64) void latent_append_kernel(AppendArgs a, int chunks) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = (int64_t)blockIdx.x * WAVES + (threadIdx.x >> 6);
    if (unit >= a.n * chunks) return;
    const int64_t tok = unit / chunks;
    const int part = (int)(unit % chunks);
    const int k = lane & 7;

    // loads first: the angle arithmetic below covers their latency
    const int64_t pos = a.positions[tok];
    const double freq = a.inv_freq[lane & 31];
    const uint16_t *src = a.kv + tok * a.kv_row;
    const bool rows = part == 0;             // this wave stores the cache row
    u32x4_t x = {0, 0, 0, 0}, rot = x, w = x;
    int64_t slot = -1;
    if (rows) {
        slot = a.slots[tok];
        x = *reinterpret_cast<const u32x4_t *>(src + 8 * lane);
        rot = load_pairs(src + L, k, a.interleaved);
        if (a.weight) w = *reinterpret_cast<const u32x4_t *>(a.weight + 8 * lane);
    }
    const double turns = (double)pos * freq * 0.15915494309189533577;
    float sn, cs;
    sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = __shfl(cs, 4 * k + i);
        s[i] = __shfl(sn, 4 * k + i);
    }
    if (rows) {
        if (a.weight) {
            float f[8], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[i] = (i & 1) ? hi_f32(x[i / 2]) : lo_f32(x[i / 2]);
                sum = fmaf(f[i], f[i], sum);
            }
            float one[1] = {sum};
            wave_transpose_reduce<1, 32>(one, lane);
            const float r = 1.0f / sqrtf(one[0] * (1.0f / L) + a.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = pack_bf16(f[2 * i] * r * lo_f32(w[i]), f[2 * i + 1] * r * hi_f32(w[i]));
        }
        const u32x4_t y = turn(rot, c, s, a.interleaved);
        if (slot >= 0 && slot < a.pages * a.page) {      // other slots: the row is dropped
            uint16_t *dst = a.cache + slot / a.page * a.c_page + slot % a.page * a.c_row;
            *reinterpret_cast<u32x4_t *>(dst + 8 * lane) = x;
            if (lane < 8) store_pairs(dst + L, k, y, a.interleaved);
        }
    }
    if (!a.q) return;
    const int h1 = min(a.heads, (part + 1) * a.chunk);
    const uint16_t *qs = a.q + tok * a.q_row;
    uint16_t *qd = a.q_out + tok * a.qo_row;
#pragma unroll 4
    for (int h = part * a.chunk + (lane >> 3); h < h1; h += 8) {
        const u32x4_t v = load_pairs(qs + h * a.q_head, k, a.interleaved);
        store_pairs(qd + h * a.qo_head, k, turn(v, c, s, a.interleaved), a.interleaved);
    }
}

}  // namespace

hipError_t launch_latent_append(const skinny_latent_append_args &p, hipStream_t stream) {
    AppendArgs a;
    a.kv = static_cast<const uint16_t *>(p.kv);
    a.kv_row = p.kv_stride;
    a.cache = static_cast<uint16_t *>(p.cache);
    a.c_page = p.cache_page_stride;
    a.c_row = p.cache_row_stride;
    a.slots = p.slots;
    a.positions = p.positions;
    a.inv_freq = p.inv_freq;
    a.weight = static_cast<const uint16_t *>(p.norm_weight);
    a.eps = p.eps;
    a.q = p.heads > 0 ? static_cast<const uint16_t *>(p.q) : nullptr;
    a.q_row = p.q_row_stride;
    a.q_head = p.q_head_stride;
    a.q_out = static_cast<uint16_t *>(p.q_out);
    a.qo_row = p.q_out_row_stride;
    a.qo_head = p.q_out_head_stride;
    a.n = p.n;
    a.pages = p.pages;
    a.heads = a.q ? (int)p.heads : 0;
    a.page = (int)p.page;
    a.interleaved = p.interleaved != 0;
    // heads a wave: all of a token's while that fills the chip (angles once a token), else as few as 8
    // (128 heads: 1 token 4.4 us against 7.4 in one wave, 256 tokens 4.8 against 9.6)
    const int all = std::max(8, (a.heads + 7) / 8 * 8);
    a.chunk = all;
    while (a.chunk > 8 && a.n * ((all + a.chunk - 1) / a.chunk) < 4096) a.chunk = (a.chunk / 2 + 7) / 8 * 8;
    const int chunks = a.heads ? (a.heads + a.chunk - 1) / a.chunk : 1;
    const int64_t blocks = (a.n * chunks + WAVES - 1) / WAVES;
    hipLaunchKernelGGL(latent_append_kernel, dim3((unsigned)blocks), dim3(WAVES * 64), 0, stream, a, chunks);
    return hipGetLastError();
}

}  // namespace skinny
