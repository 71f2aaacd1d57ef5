// AdamW over every layer in one launch, with moments in binary32 or in 8-bit
// codes with a scale per 256 elements (ga_adamw_step).
//
// A wavefront takes 512 consecutive elements of the fused row: it reads the
// workers' gradients through the layer table (grads.h), the weights and the
// moments, and writes them back, so that every byte moves once and nothing of
// the mean gradient goes through memory.  Bound by memory: per element W * b
// (gradients) + 8 (w) + 16 (binary32 moments) or 4 + 1/16 (codes and scales) +
// 2 (low-precision copy) bytes, against some 60 to 100 instructions.
//
// Codes are e4m3: 4 exponent bits, 3 mantissa bits.  The block maximum is a
// reduction over the lanes that hold the block's 256 elements, in registers;
// the second moment is held as its square root, which halves its range in
// powers of two, and is rounded at random: with beta2 = 0.999 a steady second
// moment moves by 0.05% per step, a code's step is 6% to 12%, and rounding to
// nearest would never leave the code it is at.
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

// 4 consecutive binary32 values at element i of p, 0 past P.
__device__ __forceinline__ f32x4 load4(const float* p, int64_t i, int64_t P) {
    if (i + 4 <= P) return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i));
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (i + e < P) r[e] = p[i + e];
    return r;
}

__device__ __forceinline__ void store4(float* p, int64_t i, int64_t P, const f32x4& x) {
    if (i + 4 <= P) {
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(p + i));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < P) p[i + e] = x[e];
    }
}

template <int T>
__device__ __forceinline__ void store4_narrow(void* p, int64_t i, int64_t P, const f32x4& x) {
    const uint64_t at = reinterpret_cast<uint64_t>(p) + (uint64_t)i * 2;
    if (i + 4 <= P) {
        Raw<T, 4> r;
        r.narrow({x.x, x.y, x.z, x.w});
        r.template store<true>(at);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < P) store_one<T>(at + 2 * e, x[e]);
    }
}

template <int T, int BITS, int LEV, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_adamw(GradArgs ga, StepArgs a, int64_t n_tiles) {
    const int lane = threadIdx.x & 63;
    const int64_t tile = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (tile >= n_tiles) return;
    const TileRec rec = ga.tiles[tile];
    const int64_t i0 = group_at<SPLIT>(tile, lane, 0), i1 = group_at<SPLIT>(tile, lane, 1);
    const int64_t at[2] = {i0, i1};
    float clip = 1.f;
    if (a.clip) {
        if (a.clip->skip) return;
        clip = a.clip->scale;
    }

    f32x4 w[2], m[2], s[2];   // s: v for binary32 moments, its root for codes
    float ms[2], vs[2];
    uint32_t mc[2], vc[2];
    const int64_t n_coded = (ga.P + GA_STATE_BLOCK - 1) / GA_STATE_BLOCK * GA_STATE_BLOCK;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        w[q] = load4(a.w, at[q], ga.P);
        if constexpr (BITS == 32) {
            m[q] = load4(static_cast<const float*>(a.m), at[q], ga.P);
            s[q] = load4(static_cast<const float*>(a.v), at[q], ga.P);
        } else {
            mc[q] = vc[q] = 0u;
            ms[q] = vs[q] = 0.f;
            if (at[q] < n_coded) {
                mc[q] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + at[q]);
                vc[q] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + at[q]);
                ms[q] = a.m_scale[at[q] / GA_STATE_BLOCK];
                vs[q] = a.v_scale[at[q] / GA_STATE_BLOCK];
            }
        }
    }

    float g[8];
    uint32_t dmask;
    mean_grad<T, LEV, SPLIT>(ga, tile, rec, lane, g, dmask);

    if constexpr (BITS == 8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const auto ma = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[q], false);
            const auto mb = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[q], true);
            const auto va = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[q], false);
            const auto vb = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[q], true);
            m[q] = f32x4{ma[0] * ms[q], ma[1] * ms[q], mb[0] * ms[q], mb[1] * ms[q]};
            s[q] = f32x4{va[0] * vs[q], va[1] * vs[q], vb[0] * vs[q], vb[1] * vs[q]};
        }
    }

    uint32_t mtop[2] = {0u, 0u}, stop[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float gr = g[4 * q + e] * clip;
            const float mn = fmaf(a.beta1, m[q][e], a.c1 * gr);
            const float v0 = BITS == 32 ? s[q][e] : s[q][e] * s[q][e];
            const float vn = fmaf(a.beta2, v0, (a.c2 * gr) * gr);
            const float root = sqrtf(vn);
            const float keep = (dmask >> (4 * q + e)) & 1u ? a.keep : 1.f;
            w[q][e] = fmaf(-a.lr_t, mn / fmaf(root, a.rbc2, a.eps), w[q][e] * keep);
            m[q][e] = mn;
            if constexpr (BITS == 32) {
                s[q][e] = vn;
            } else {
                const bool in = at[q] + e < ga.P;
                s[q][e] = in ? root : 0.f;
                m[q][e] = in ? mn : 0.f;
                const uint32_t ma = __float_as_uint(m[q][e]) & 0x7fffffffu, sa = __float_as_uint(s[q][e]) & 0x7fffffffu;
                mtop[q] = mtop[q] > ma ? mtop[q] : ma;
                stop[q] = stop[q] > sa ? stop[q] : sa;
            }
        }
        store4(a.w, at[q], ga.P, w[q]);
        if (a.copy) {
            if (a.copy_dtype == kB16) store4_narrow<kB16>(a.copy, at[q], ga.P, w[q]);
            else store4_narrow<kF16>(a.copy, at[q], ga.P, w[q]);
        }
        if constexpr (BITS == 32) {
            store4(static_cast<float*>(a.m), at[q], ga.P, m[q]);
            store4(static_cast<float*>(a.v), at[q], ga.P, s[q]);
        }
    }
    if constexpr (BITS == 8) {
        // the block's largest magnitudes (as bit patterns: a NaN wins), in every lane of the block
        if constexpr (SPLIT) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                mtop[q] = wave_max_u32(mtop[q]);
                stop[q] = wave_max_u32(stop[q]);
            }
        } else {
            mtop[0] = mtop[1] = half_max_u32(mtop[0] > mtop[1] ? mtop[0] : mtop[1]);
            stop[0] = stop[1] = half_max_u32(stop[0] > stop[1] ? stop[0] : stop[1]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float mt = __uint_as_float(mtop[q] > kFloorBits ? mtop[q] : kFloorBits);
            const float st = __uint_as_float(stop[q] > kFloorBits ? stop[q] : kFloorBits);
            const float mu = kCodeMax / mt, su = kCodeMax / st;
            const uint32_t pair = (uint32_t)(at[q] >> 1) + a.seed;
            const uint32_t rnd[2] = {mix(pair), mix(pair + 1u)};
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = s[q][e] * su;
                y = y > kCodeMax ? kCodeMax : y;
                y = s[q][e] > 0.f && y < 0x1p-6f ? 0x1p-6f : y;
                // 3 mantissa bits stay: 16 random bits, centred, on top of the 20 that go
                const uint32_t r = e & 1 ? rnd[e >> 1] >> 16 : rnd[e >> 1] & 0xffffu;
                x[e] = __uint_as_float((__float_as_uint(y) + ((r << 4) | 8u)) & 0xfff00000u);
            }
            int cv = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
            cv = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], cv, true);
            int cm = __builtin_amdgcn_cvt_pk_fp8_f32(m[q][0] * mu, m[q][1] * mu, 0, false);
            cm = __builtin_amdgcn_cvt_pk_fp8_f32(m[q][2] * mu, m[q][3] * mu, cm, true);
            if (at[q] < n_coded) {
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + at[q]) = (uint32_t)cm;
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + at[q]) = (uint32_t)cv;
                if (at[q] % GA_STATE_BLOCK == 0) {
                    a.m_scale[at[q] / GA_STATE_BLOCK] = mt * (1.f / kCodeMax);
                    a.v_scale[at[q] / GA_STATE_BLOCK] = st * (1.f / kCodeMax);
                }
            }
        }
    }
}

template <int T, int BITS>
hipError_t adamw_launch(const Adamw& o, const uint64_t* layer_ptrs, const StepArgs& a, hipStream_t s) {
    const GradArgs g = grad_args(o, layer_ptrs);
    const unsigned blocks = (unsigned)((o.n_tiles + kThreads / 64 - 1) / (kThreads / 64));
    return with_levels(o.W, [&](auto lev) {
        hipLaunchKernelGGL((k_adamw<T, BITS, decltype(lev)::value, false>), dim3(blocks), dim3(kThreads), 0, s, g, a,
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
