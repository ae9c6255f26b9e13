// latent.hpp -- device helpers shared by the latent attention kernels (gfx950 only).
#pragma once

#include <type_traits>

#include "common.hpp"

namespace skinny {
namespace latent {

typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// s_waitcnt immediate: at most n vector-memory operations outstanding (gfx9 encoding: vmcnt
// bits 3:0 and 15:14; expcnt and lgkmcnt at their maxima, i.e. not waited for).
template <int n>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(n >= 0 && n < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Barrier ordering the workgroup's LDS accesses: this wave's LDS reads are done, outstanding
// loads straight into LDS are not waited for (each wave has already waited for those it needs).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}

// f(0), f(1) ... f(N - 1), each number a constant of its own type: arrays that it indexes stay in registers
// where a loop would be unrolled too late for that.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void static_for(const F &f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        static_for<N, I + 1>(f);
    }
}

// ---- loads straight into LDS --------------------------------------------------------------
// lane l's 16 bytes at src (4 with load_lds_word) go to LDS address lds + 16 l (4 l), and of N
// pieces those at src + 128 i to lds + 1024 i + 16 l. lds is the same in all lanes. Written out
// because the compiler does not know which staged bytes a read of LDS needs: behind the builtin it
// waits for every load in flight before the next read, and the ring would hold one stage. Here
// the kernel's own counted waits order the two. (No vector register is written; M0, which nothing
// else in these kernels uses and the compiler never keeps, is given its required
// wait state, and the instruction's offset counts in both addresses.)
__device__ __forceinline__ int lds_address(lds_u8 *p) { return uniform((int)(uintptr_t)p); }

__device__ __forceinline__ void load_lds_word(const void *src, int lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :: "s"(lds), "v"(src) : "memory");
}

// piece I of a row: src + 128 I to lds + 1024 I
template <int I>
__device__ __forceinline__ void load_lds_piece(const void *src, int lds) {
    asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%3"
                 :: "s"(lds), "v"(src), "i"(896 * I), "i"(128 * I) : "memory", "scc");
}
template <int N, int I = 0>
__device__ __forceinline__ void load_lds_pieces(const void *src, int lds) {
    if constexpr (I < N) {
        load_lds_piece<I>(src, lds);
        load_lds_pieces<N, I + 1>(src, lds);
    }
}
// the same in the lanes of `lanes`, all or none of them: the count of loads in flight goes by either way
// (called with all lanes active)
__device__ __forceinline__ uint64_t lanes_if(bool on) {
    const uint32_t half = uniform(on ? -1 : 0);
    return (uint64_t)half << 32 | half;
}
template <int I>
__device__ __forceinline__ void load_lds_piece_in(uint64_t lanes, const void *src, int lds) {
    asm volatile("s_add_u32 m0, %0, %2\n\ts_mov_b64 exec, %4\n\tglobal_load_lds_dwordx4 %1, off offset:%3\n\t"
                 "s_mov_b64 exec, -1"
                 :: "s"(lds), "v"(src), "i"(896 * I), "i"(128 * I), "s"(lanes) : "memory", "scc");
}
// the same from `base`, the same in all lanes, and each lane's own bytes from there
template <int I>
__device__ __forceinline__ void load_lds_piece_in(uint64_t lanes, const void *base, uint32_t own, int lds) {
    asm volatile("s_add_u32 m0, %0, %2\n\ts_mov_b64 exec, %4\n\tglobal_load_lds_dwordx4 %1, %5 offset:%3\n\t"
                 "s_mov_b64 exec, -1"
                 :: "s"(lds), "v"(own), "i"(896 * I), "i"(128 * I), "s"(lanes), "s"(base) : "memory", "scc");
}

// ---- staged key and value rows ----------------------------------------------------------
// Rows come into LDS in blocks of 8 rows x 128 bytes (one direct-to-LDS instruction: lane l
// fills row l / 8, 16-byte place l % 8). Place p of row r holds chunk p ^ swz(r): the 32- or
// 16-row fragment reads of the score product and the transposed reads of the value product
// then both spread over all the banks.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// ---- matrix instruction shapes ----------------------------------------------------------
// Both attention kernels compute transposed products, so that a query row is a column of every
// accumulator and stays with one lane: S^T[key, row] = K Q^T, then O^T[dim, row] = V^T P^T.
// The accumulator registers of S^T, packed to bf16, are the second product's B fragment as they
// are, if its A fragment takes its keys in the same order; V^T is read from LDS with the
// transposing 64-bit read (each 16-lane group: 4 keys x 16 dims, a lane gets its dim's 4 keys).
struct Tile32 {                 // v_mfma_f32_32x32x16_bf16: 32 rows per wave
    static constexpr int ROWS = 32, KSTEP = 16, NS = 16, NO = 16, DIMS = 32;
    typedef f32x16_t acc_t;
    static __device__ __forceinline__ acc_t mfma(u32x4_t a, u32x4_t b, acc_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ int row(int lane) { return lane & 31; }
    static __device__ __forceinline__ int grp(int lane) { return lane >> 5; }
    // accumulator register i of lane group g holds matrix row (key or dim) place(i, g)
    static __host__ __device__ __forceinline__ constexpr int place(int i, int g) { return 8 * (i >> 2) + 4 * g + (i & 3); }
};
struct Tile16 {                 // v_mfma_f32_16x16x32_bf16: 16 rows per wave
    static constexpr int ROWS = 16, KSTEP = 32, NS = 8, NO = 4, DIMS = 16;
    typedef f32x4_t acc_t;
    static __device__ __forceinline__ acc_t mfma(u32x4_t a, u32x4_t b, acc_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ int row(int lane) { return lane & 15; }
    static __device__ __forceinline__ int grp(int lane) { return lane >> 4; }
    static __host__ __device__ __forceinline__ constexpr int place(int i, int g) { return 16 * (i >> 2) + 4 * g + (i & 3); }
};

// The largest / the sum of v over the lane groups that share a row.
template <typename T>
__device__ __forceinline__ float row_max(float v) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    if constexpr (T::ROWS == 16) {
        r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}
template <typename T>
__device__ __forceinline__ float row_sum(float v) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if constexpr (T::ROWS == 16) {
        r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

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

// Hold accumulators where they belong at this point: output sums in accumulation registers (a
// branch that rescales them would otherwise move all of them to ordinary ones and back in every
// iteration), scores in ordinary ones.
template <typename V, int N>
__device__ __forceinline__ void in_acc(V (&o)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+a"(o[i]));
}
template <typename V, int N>
__device__ __forceinline__ void in_vgpr(V (&s)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(s[i]));
}

// two floats to packed bf16, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), bf16x2_t));
}

__device__ __forceinline__ bool finite_f32(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// ---- non-finite values that some rows do not see ------------------------------------------
// In the value product a weight of 0 times a non-finite value is NaN, so such a value would reach
// rows whose mask hides it. split_value takes it out of a fragment f (g: the finite ones) and
// gives it back as a1 and a2: the largest number, signed, for an infinity, and both signs of it
// for a NaN. Against a B fragment of seen_pair's (the largest number where the row sees the
// key, else 0) those products overflow to the infinity or NaN that seeing rows must get, and are
// 0 for the others.
constexpr uint32_t kBig = 0x7F7Fu;
__device__ __forceinline__ void split_value(u32x4_t f, u32x4_t &g, u32x4_t &a1, u32x4_t &a2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t x = 0, y = 0, z = 0;
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            const uint32_t v = (f[i] >> h) & 0xFFFFu;
            const bool odd = (v & 0x7F80u) == 0x7F80u, nan = odd && (v & 0x7Fu);
            x |= (odd ? 0u : v) << h;
            y |= (nan ? kBig : odd ? (v & 0x8000u) | kBig : 0u) << h;
            z |= (nan ? 0x8000u | kBig : 0u) << h;
        }
        g[i] = x;
        a1[i] = y;
        a2[i] = z;
    }
}
__device__ __forceinline__ uint32_t seen_pair(bool lo, bool hi) { return (lo ? kBig : 0u) | (hi ? kBig << 16 : 0u); }

// f's finite values, with 0 for the rest; with others the largest number in the places of the rest, with
// 0 for the finite ones (others is the same in all lanes).
__device__ __forceinline__ u32x4_t pick_values(u32x4_t f, bool others) {
    const uint32_t keep = others ? 0u : ~0u, put = others ? kBig | kBig << 16 : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t odd = ((f[i] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) |
                             ((f[i] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
        f[i] = (f[i] & ~odd & keep) | (odd & put);
    }
    return f;
}

// A row's reference maximum follows the scores' only when they pass it by more than this (in
// powers of two): the sums then stay within 2^kSlack of their usual size, far inside fp32's
// range, and the outputs are rescaled a few times a row instead of at every new maximum.
constexpr float kSlack = 8.0f;

}  // namespace latent
}  // namespace skinny
