// Element types of the training-step operators (binary32, binary16, bfloat16
// and 8-bit e4m3) and cross-lane reductions over a 64-wide wavefront.
//
// Vectors are read and written at any element alignment: the hardware serves
// 64- and 128-bit global accesses at any byte address, so an odd row length or
// a tensor placed at an odd offset needs no element-by-element path (only a
// vector that would pass the end of its row or layer is taken apart).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gradagg.h"
#include "device.h"

namespace ga {

constexpr int kF32 = GA_FP32, kF16 = GA_FP16, kB16 = GA_BF16;

template <int T>
constexpr int kSize = T == kF32 ? 4 : 2;

// 64- and 128-bit words at the alignment of a 16-bit element.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two packed 16-bit values, widened exactly.
template <int T>
__device__ __forceinline__ void widen2(uint32_t u, float& a, float& b) {
    if constexpr (T == kF16) {
        const f16x2 h = __builtin_bit_cast(f16x2, u);
        a = (float)h.x;
        b = (float)h.y;
    } else {
        a = __uint_as_float(u << 16);
        b = __uint_as_float(u & 0xffff0000u);
    }
}

// Two values rounded to nearest even and packed.
template <int T>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (T == kF16) {
        const f16x2 h = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, h);
    } else {
        const bf16x2 h = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, h);
    }
}

// The value after rounding to T (as it will be read back).
template <int T>
__device__ __forceinline__ float rounded(float x) {
    if constexpr (T == kF32) return x;
    else if constexpr (T == kF16) return (float)(_Float16)x;
    else return (float)(__bf16)x;
}

template <int T>
__device__ __forceinline__ float load_one(uint64_t addr) {
    if constexpr (T == kF32) return *as_global<float>(addr);
    else if constexpr (T == kF16) return widen1(*as_global<uint16_t>(addr));
    else return __uint_as_float((uint32_t)*as_global<uint16_t>(addr) << 16);
}

template <int T>
__device__ __forceinline__ void store_one(uint64_t addr, float x) {
    if constexpr (T == kF32) *reinterpret_cast<__attribute__((address_space(1))) float*>(addr) = x;
    else *reinterpret_cast<__attribute__((address_space(1))) uint16_t*>(addr) = (uint16_t)narrow2<T>(x, 0.f);
}

// N (4 or 8) consecutive elements as stored, in 32-bit words.
template <int T, int N>
struct Raw {
    static constexpr int WORDS = N * kSize<T> / 4;
    uint32_t w[WORDS];

    template <bool NT = false>
    __device__ __forceinline__ void load(uint64_t addr) {
#pragma unroll
        for (int q = 0; q < WORDS; q += 4) {
            if constexpr (WORDS == 2) {
                const u32x2_any x = NT ? __builtin_nontemporal_load(as_global<u32x2_any>(addr))
                                       : *as_global<u32x2_any>(addr);
                w[0] = x.x;
                w[1] = x.y;
            } else {
                const u32x4_any x = NT ? __builtin_nontemporal_load(as_global<u32x4_any>(addr + 4 * q))
                                       : *as_global<u32x4_any>(addr + 4 * q);
                w[q] = x.x;
                w[q + 1] = x.y;
                w[q + 2] = x.z;
                w[q + 3] = x.w;
            }
        }
    }

    template <bool NT = false>
    __device__ __forceinline__ void store(uint64_t addr) const {
#pragma unroll
        for (int q = 0; q < WORDS; q += 4) {
            if constexpr (WORDS == 2) {
                auto* p = reinterpret_cast<__attribute__((address_space(1))) u32x2_any*>(addr);
                const u32x2_any x = {w[0], w[1]};
                if (NT) __builtin_nontemporal_store(x, p);
                else *p = x;
            } else {
                auto* p = reinterpret_cast<__attribute__((address_space(1))) u32x4_any*>(addr + 4 * q);
                const u32x4_any x = {w[q], w[q + 1], w[q + 2], w[q + 3]};
                if (NT) __builtin_nontemporal_store(x, p);
                else *p = x;
            }
        }
    }

    __device__ __forceinline__ void widen(float (&f)[N]) const {
        if constexpr (T == kF32) {
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = __uint_as_float(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < N; e += 2) widen2<T>(w[e / 2], f[e], f[e + 1]);
        }
    }

    __device__ __forceinline__ void narrow(const float (&f)[N]) {
        if constexpr (T == kF32) {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = __float_as_uint(f[e]);
        } else {
#pragma unroll
            for (int e = 0; e < N; e += 2) w[e / 2] = narrow2<T>(f[e], f[e + 1]);
        }
    }
};

// ---- cross-lane reductions -------------------------------------------------
// Within 16 lanes by data-parallel moves (xor 1, xor 2, mirrored 8, mirrored
// 16), across rows of 16 and halves of 32 by the row and half exchanges; every
// lane ends with the result.  Each step adds the same two values in both
// partners, so all lanes hold the same bits.

template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}

template <typename OP>
__device__ __forceinline__ uint32_t reduce16(uint32_t x, OP op) {
    x = op(x, lane_move<0xb1>(x));    // xor 1
    x = op(x, lane_move<0x4e>(x));    // xor 2
    x = op(x, lane_move<0x141>(x));   // mirror within 8
    return op(x, lane_move<0x140>(x));   // mirror within 16
}

// Sum over aligned runs of T lanes (16, 32 or 64).
template <int T>
__device__ __forceinline__ float lanes_sum_f32(float x) {
    const auto add = [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
    uint32_t u = reduce16(__float_as_uint(x), add);
    if constexpr (T >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        u = add(r[0], r[1]);
    }
    if constexpr (T >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        u = add(r[0], r[1]);
    }
    return __uint_as_float(u);
}

__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
    return x;
}

}  // namespace ga
