// latent_line.hpp -- one line of work for requests whose lengths only the device knows (gfx950 only).
//
// The key tiles of all requests, one request after the other (times `groups` for kernels that take a
// request's rows in groups), form a line. Workgroups take equal runs of it, whatever the lengths.
// An argument struct A names batch and groups, and request_tiles(a, i) what request i takes of the line.
#pragma once

#include <climits>

#include "latent.hpp"

namespace skinny {
namespace latent {

// Sum of v over the workgroup's threads before this one, and over all of them.
template <int THREADS>
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
// of that request's first tile. Up to 512 requests each wave works it out by itself, 32 bits allowing: lane i
// counts requests i * per .. i * per + per - 1, and nothing waits at a barrier (with this, and sums that are not
// rescaled while they are 0, a decode step of one request of 56 rows x 500 keys takes 10.2 us where it took 11.6).
// With more, thread i of the workgroup does.
template <typename A, int THREADS>
struct Line {
    static constexpr int WAVES = THREADS / 64;           // sh holds WAVES + 2 numbers
    static constexpr int MOST_PER_LANE = 8;
    int64_t total, before;                   // of this thread's requests
    int per, own;
    bool alone;
    __device__ __forceinline__ int64_t count(const A &a, int first) const {
        int64_t v = 0;
        for (int i = first; i < min(a.batch, first + per); ++i) v += request_tiles(a, i);
        return v * a.groups;
    }
    // most: an upper bound of total
    __device__ __forceinline__ void measure(const A &a, int64_t most, int64_t *sh) {
        alone = a.batch <= 64 * MOST_PER_LANE && most <= INT_MAX;
        if (alone) {
            const int lane = threadIdx.x & 63;
            per = (a.batch + 63) / 64;
            own = (int)count(a, lane * per);
            const int sum = wave_scan(own);
            before = sum - own;
            total = __builtin_amdgcn_readlane(sum, 63);
            return;
        }
        per = (a.batch + THREADS - 1) / THREADS;
        before = block_scan<THREADS>(count(a, threadIdx.x * per), sh, total);
        total = uniform(total);
    }
    __device__ __forceinline__ void find(const A &a, int64_t x, int64_t *sh, int &req, int64_t &base) const {
        if (alone) {
            const int w = __builtin_ctzll(__ballot(before <= x && x < before + own));
            base = __builtin_amdgcn_readlane((int)before, w);
            req = w * per;
            if (per == 1) return;
            for (;;) {
                const int64_t n = (int64_t)uniform(request_tiles(a, req)) * a.groups;
                if (x < base + n || req + 1 == a.batch) return;
                base += n;
                ++req;
            }
        }
        int64_t at = before;
        for (int i = threadIdx.x * per; i < min(a.batch, (int)(threadIdx.x + 1) * per); ++i) {
            const int64_t n = (int64_t)request_tiles(a, i) * a.groups;
            if (at <= x && x < at + n) {
                sh[WAVES] = i;
                sh[WAVES + 1] = at;
            }
            at += n;
        }
        __syncthreads();
        req = uniform((int)sh[WAVES]);
        base = uniform(sh[WAVES + 1]);
    }
};

// Workgroup b's run of the line: [b * total / grid, (b + 1) * total / grid). Runs leave partials
// 2b (of the run's first unit) and 2b + 1 (of its last, if that is another).
__device__ __forceinline__ int64_t run_start(int64_t total, int grid, int b) { return total * b / grid; }
// the workgroup whose run holds place x (no run is empty: grid <= total)
__device__ __forceinline__ int run_of(int64_t total, int grid, int64_t x) { return (int)(((x + 1) * grid - 1) / total); }

// k / d for 0 <= k < 2^30: (k * mul) >> (32 + shift), mul 0 for a d of 1.
// 2^bits >= d > 2^(bits - 1): the reciprocal 2^(31 + bits) / d, rounded up, fits 32 bits, and
// for k < 2^30 its rounding adds less than 2^-(1 + bits) < 1 / d to the quotient: exact
inline void reciprocal(int d, uint32_t &mul, int &shift) {
    int bits = 1;
    while ((1 << bits) < d) ++bits;
    mul = d == 1 ? 0 : (uint32_t)((((uint64_t)1 << (31 + bits)) + d - 1) / d);
    shift = bits - 1;
}
__device__ __forceinline__ int quotient(int k, uint32_t mul, int shift) {
    return mul ? (int)(__umulhi((uint32_t)k, mul) >> shift) : k;
}
template <typename A>
__device__ __forceinline__ int page_of(const A &a, int k) { return quotient(k, a.page_mul, a.page_shift); }

}  // namespace latent
}  // namespace skinny
