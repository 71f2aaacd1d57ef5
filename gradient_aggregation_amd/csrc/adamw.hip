// AdamW over every layer in one launch, with moments in binary32 or in 8-bit
// codes with a scale per 256 elements (ga_adamw_step).
//
// A wavefront takes 512 consecutive elements of the fused row: it reads the
// workers' gradients through the layer table (grads.h), the weights and the
// moments, and writes them back, so that every byte moves once and nothing of
// the mean gradient goes through memory.  Bound by memory: per element W * b
// (gradients) + 8 (w) + 16 (binary32 moments) or 4 + 1/16 (codes and scales) +
// 2 (low-precision copy) bytes, against some 40 to 70 instructions.  61M
// parameters of 16 binary16 workers: 565 us (6.0 TB/s); 61M with 8-bit states,
// bf16 gradients and copy: 164 us (6.0 TB/s); 7.6M with binary32 states, bf16
// gradients and copy: 37 us (5.7 TB/s); 29,354: 6 us.
//
// Codes are e4m3: 4 exponent bits, 3 mantissa bits.  The block maximum is a
// reduction over the lanes that hold the block's 256 elements, in registers;
// the second moment is held as its square root, which halves its range in
// powers of two.  Both are rounded at random: a code's step is 6% to 12%, and a
// moment that moves by less than half of that per step would never leave the
// code it is at if it were rounded to nearest.  A second moment with beta2 =
// 0.999 moves by 0.1% of its distance; a first moment by (1 - beta1) of its:
// after a gradient that becomes zero, weights would go on moving for ever
// (2800 steps at beta1 = 0.99: 12901 times lr, where the recurrence itself gives
// 114).  m to nearest stays as a choice, for states that were kept that way.
#include "grads.h"

namespace ga {

namespace {

constexpr int kThreads = 256;
constexpr float kCodeMax = 448.f;
constexpr uint32_t kFloorBits = (127u - 100u) << 23;   // 2^-100, the least block maximum

// 16 random bits for each element of a pair from its counter: multiply and
// xor-shift.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0xB7E15163u;
    x = (x ^ (x >> 15)) * 0x6A09E667u;
    return x ^ (x >> 16);
}

// Counters of m's bits are this far from those of v's: the two are rounded
// independently.
constexpr uint32_t kSeedM = 0xBB67AE85u;

// x cut at random to the grid of the codes: `bits` (below 2^20, a fraction of a
// step) is added to the 20 mantissa bits that go.  Below 2^-6 the codes are
// evenly spaced, like the binary32 values with 3 mantissa bits from 2^-6 to
// 2^-5: such an x is lifted there and lowered again, both exact but for what
// is below 2^-20 of a step.  0 stays 0, NaN stays NaN.
__device__ __forceinline__ float cut_at_random(float x, uint32_t bits) {
    float a = fabsf(x);
    a = a > kCodeMax ? kCodeMax : a;
    const float lift = a < 0x1p-6f ? 0x1p-6f : 0.f;
    const uint32_t z = (__float_as_uint(a + lift) + bits) & 0xfff00000u;
    return copysignf(__uint_as_float(z) - lift, x);
}

// 4 consecutive binary32 values at element i of p, 0 past P.
template <bool WHOLE>
__device__ __forceinline__ f32x4 load4(const float* p, int i, int64_t P) {
    if (WHOLE || i + 4 <= P) return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i));
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < P) r[e] = p[i + e];
    return r;
}

template <bool WHOLE>
__device__ __forceinline__ void store4(float* p, int i, int64_t P, const f32x4& x) {
    if (WHOLE || i + 4 <= P) {
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < P) p[i + e] = x[e];
    }
}

template <int T, bool WHOLE>
__device__ __forceinline__ void store4_narrow(void* p, int64_t e0, int i, int64_t P, const f32x4& x) {
    const uint64_t at = reinterpret_cast<uint64_t>(p) + (uint64_t)e0 * 2 + (uint32_t)i * 2;
    if (WHOLE || i + 4 <= P) {
        Raw<T, 4> r;
        r.narrow({x.x, x.y, x.z, x.w});
        r.template store<true>(at);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < P) store_one<T>(at + 2 * e, x[e]);
    }
}

// Square roots of 8 values >= 0.  EXACT: rounded correctly, for the roots that
// are held as codes: a code is cut from the root's bits, and a root one ulp off
// would now and then be the neighbouring code, a sixteenth away.  Else the
// hardware instruction, within 1 ulp (1.54 half steps over 2^20 values of every
// exponent).  It takes denormal values for zero, which only matters when one is
// there: then the small values are scaled up by 2^64 and the roots back by
// 2^-32, both exact.
template <bool EXACT>
__device__ __forceinline__ void roots(const float (&v)[8], float (&r)[8]) {
    if constexpr (EXACT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = sqrtf(v[e]);
        return;
    }
    uint32_t low = __float_as_uint(v[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) low = __float_as_uint(v[e]) < low ? __float_as_uint(v[e]) : low;
    if (low >= 0x00800000u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = __builtin_amdgcn_sqrtf(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool small = v[e] < 0x1p-64f;
            r[e] = __builtin_amdgcn_sqrtf(v[e] * (small ? 0x1p64f : 1.f)) * (small ? 0x1p-32f : 1.f);
        }
    }
}

// One tile.  WHOLE: it lies in one layer and inside P.
template <int T, int BITS, int LEV, bool WHOLE>
__device__ __forceinline__ void adamw_tile(const GradArgs& ga, const StepArgs& a, const TileRec& rec, int lane) {
    const int64_t tile = rec.tile, e0 = tile * kTile;
    const int at[2] = {lane * 4, 256 + lane * 4};   // from e0
    const int64_t P = WHOLE ? (int64_t)kTile : ga.P - e0;
    float clip = 1.f;
    if (a.clip) {
        if (a.clip->skip) return;
        clip = a.clip->scale;
    }

    f32x4 w[2], m[2], s[2];   // s: v for binary32 moments, its root for codes
    float ms[2], vs[2];
    uint32_t mc[2], vc[2];
    const auto load_state = [&] {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            w[q] = load4<WHOLE>(a.w + e0, at[q], P);
            if constexpr (BITS == 32) {
                m[q] = load4<WHOLE>(static_cast<const float*>(a.m) + e0, at[q], P);
                s[q] = load4<WHOLE>(static_cast<const float*>(a.v) + e0, at[q], P);
            } else {
                mc[q] = vc[q] = 0u;
                ms[q] = vs[q] = 0.f;
                if (WHOLE || q * GA_STATE_BLOCK < P) {
                    mc[q] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + e0 + at[q]);
                    vc[q] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + e0 + at[q]);
                    ms[q] = a.m_scale[tile * 2 + q];
                    vs[q] = a.v_scale[tile * 2 + q];
                }
            }
        }
    };
    // with several workers the leaves and their tree come first: the state's 24 registers beside them would cost a
    // wavefront per SIMD (61M parameters of 16 workers: 642 us; 588 us at four per SIMD)
    if constexpr (LEV == 1) load_state();
    float g[8];
    uint32_t dmask = 0;
    if constexpr (WHOLE) mean_grad_whole<T, LEV>(ga, tile, rec, lane, g);
    else mean_grad_part<T, LEV>(ga, tile, rec, lane, g, dmask);
    if constexpr (LEV > 1) load_state();
    const float keep = rec.flags & kTileDecay ? a.keep : 1.f;

    float mn[8], vn[8], root[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if constexpr (BITS == 8) {
            const auto ma = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[q], false);
            const auto mb = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[q], true);
            const auto va = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[q], false);
            const auto vb = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[q], true);
            m[q] = f32x4{ma[0] * ms[q], ma[1] * ms[q], mb[0] * ms[q], mb[1] * ms[q]};
            s[q] = f32x4{va[0] * vs[q], va[1] * vs[q], vb[0] * vs[q], vb[1] * vs[q]};
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 4 * q + e;
            const float gr = g[k] * clip;
            mn[k] = a.beta1 * m[q][e] + a.c1 * gr;
            const float v0 = BITS == 32 ? s[q][e] : s[q][e] * s[q][e];
            vn[k] = a.beta2 * v0 + (a.c2 * gr) * gr;
        }
    }
    roots<BITS == 8>(vn, root);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 4 * q + e;
            // the hardware reciprocal is within 1 ulp of 1/x for the denominators there are: eps is 0 or
            // normal, the root of the least v is 2^-74.5, and the largest are below 2^126
            const float up = mn[k] * __builtin_amdgcn_rcpf(fmaf(root[k], a.rbc2, a.eps));
            const float kp = WHOLE ? keep : (dmask >> k) & 1u ? a.keep : 1.f;
            w[q][e] = fmaf(-a.lr_t, up, w[q][e] * kp);
            if (BITS == 8 && !WHOLE && at[q] + e >= P) root[k] = mn[k] = 0.f;
        }
        store4<WHOLE>(a.w + e0, at[q], P, w[q]);
        if (a.copy) {
            if (a.copy_dtype == kB16) store4_narrow<kB16, WHOLE>(a.copy, e0, at[q], P, w[q]);
            else store4_narrow<kF16, WHOLE>(a.copy, e0, at[q], P, w[q]);
        }
        if constexpr (BITS == 32) {
            store4<WHOLE>(static_cast<float*>(a.m) + e0, at[q], P, f32x4{mn[4 * q], mn[4 * q + 1], mn[4 * q + 2], mn[4 * q + 3]});
            store4<WHOLE>(static_cast<float*>(a.v) + e0, at[q], P, f32x4{vn[4 * q], vn[4 * q + 1], vn[4 * q + 2], vn[4 * q + 3]});
        }
    }
    if constexpr (BITS == 8) {
        // The four block maxima (as bit patterns: a NaN wins) in one reduction: the halves of the wavefront take a
        // block each, then the even and odd rows of 16 lanes m and the root; row 0 ends with m of block 0, row 1
        // with its root, rows 2 and 3 with those of block 1.
        uint32_t top[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            top[0][q] = top[1][q] = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t ma = __float_as_uint(mn[4 * q + e]) & 0x7fffffffu;
                const uint32_t sa = __float_as_uint(root[4 * q + e]) & 0x7fffffffu;
                top[0][q] = top[0][q] > ma ? top[0][q] : ma;
                top[1][q] = top[1][q] > sa ? top[1][q] : sa;
            }
        }
        const auto larger = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
        uint32_t half[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const auto r = __builtin_amdgcn_permlane32_swap(top[j][0], top[j][1], false, false);
            half[j] = larger(r[0], r[1]);
        }
        const auto r16 = __builtin_amdgcn_permlane16_swap(half[0], half[1], false, false);
        uint32_t row = reduce16(larger(r16[0], r16[1]), larger);
        row = larger(row, kFloorBits);
        const float largest = __uint_as_float(row);
        const float unit = (1.f / largest) * kCodeMax;
        if ((lane & 15) == 0 && (WHOLE || (lane >> 5) * GA_STATE_BLOCK < P))
            (lane & 16 ? a.v_scale : a.m_scale)[tile * 2 + (lane >> 5)] = largest * (1.f / kCodeMax);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float mu = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(unit), 32 * q));
            const float su = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(unit), 32 * q + 16));
            const uint32_t pair = (uint32_t)((uint64_t)e0 >> 1) + a.seed + (uint32_t)(at[q] >> 1);
            const uint32_t rnd[2] = {mix(pair), mix(pair + 1u)};
            int cv = 0;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = root[4 * q + e];
                y[e] = __builtin_amdgcn_fmed3f(x * su, 0x1p-6f, kCodeMax);
                y[e] = x > 0.f ? y[e] : x;   // 0 stays 0, NaN stays NaN
            }
            // rounded by adding 20 random bits (16 of them, centred) to the 20 mantissa bits that go: the hardware's
            // stochastic conversion adds the upper 20 bits of its second operand
            cv = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], (rnd[0] << 16) | 0x8000u, cv, 0);
            cv = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], (rnd[0] & 0xffff0000u) | 0x8000u, cv, 1);
            cv = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], (rnd[1] << 16) | 0x8000u, cv, 2);
            cv = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], (rnd[1] & 0xffff0000u) | 0x8000u, cv, 3);
            float z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = mn[4 * q + e] * mu;
            if (a.m_rounding == GA_ROUND_RANDOM) {
                const uint32_t mr[2] = {mix(pair + kSeedM), mix(pair + kSeedM + 1u)};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[e] = cut_at_random(z[e], (e & 1 ? mr[e / 2] >> 12 & 0xffff0u : (mr[e / 2] & 0xffffu) << 4) | 8u);
            }
            int cm = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
            cm = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], cm, true);
            if (WHOLE || q * GA_STATE_BLOCK < P) {
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + e0 + at[q]) = (uint32_t)cm;
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + e0 + at[q]) = (uint32_t)cv;
            }
        }
    }
}

// Wavefronts per SIMD that the registers have to leave room for: trees of up to
// 8 levels fit the 128 registers of 4, deeper ones spill some.
template <int LEV>
constexpr int kWaves = LEV > 1 && LEV <= 8 ? 4 : 1;

template <int T, int BITS, int LEV>
__global__ __launch_bounds__(kThreads, kWaves<LEV>) void k_adamw(GradArgs ga, StepArgs a, int64_t n_tiles) {
    const int lane = threadIdx.x & 63;
    const int64_t slot = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (slot >= n_tiles) return;
    const TileRec rec = ga.tiles[slot];
    if (rec.flags & kTileWhole) adamw_tile<T, BITS, LEV, true>(ga, a, rec, lane);
    else adamw_tile<T, BITS, LEV, false>(ga, a, rec, lane);
}

template <int T, int BITS>
hipError_t adamw_launch(const Adamw& o, const uint64_t* layer_ptrs, const StepArgs& a, hipStream_t s) {
    const GradArgs g = grad_args(o, layer_ptrs);
    const unsigned blocks = (unsigned)((o.n_tiles + kThreads / 64 - 1) / (kThreads / 64));
    return with_levels(o.W, [&](auto lev) {
        hipLaunchKernelGGL((k_adamw<T, BITS, decltype(lev)::value>), dim3(blocks), dim3(kThreads), 0, s, g, a,
                           o.n_tiles);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_adamw(const Adamw& o, const uint64_t* layer_ptrs, const StepArgs& a, hipStream_t s) {
    if (o.bits == 8) {
        if (o.dtype == GA_FP32) return adamw_launch<kF32, 8>(o, layer_ptrs, a, s);
        if (o.dtype == GA_FP16) return adamw_launch<kF16, 8>(o, layer_ptrs, a, s);
        return adamw_launch<kB16, 8>(o, layer_ptrs, a, s);
    }
    if (o.dtype == GA_FP32) return adamw_launch<kF32, 32>(o, layer_ptrs, a, s);
    if (o.dtype == GA_FP16) return adamw_launch<kF16, 32>(o, layer_ptrs, a, s);
    return adamw_launch<kB16, 32>(o, layer_ptrs, a, s);
}

}  // namespace ga
