// Group norm with an activation over images, channels last (ga_groupnorm_forward,
// ga_groupnorm_backward): the plainest form.  A workgroup takes a group of a
// sample and reads it in each of its passes.
#include "elements.h"
#include "layers.h"

namespace ga {

namespace {

constexpr int kThreads = 256;

template <int P>
__device__ __forceinline__ float param(const void* p, int64_t c, float fill) {
    return p ? load_one<P>(reinterpret_cast<uint64_t>(p) + (uint64_t)c * kSize<P>) : fill;
}

__device__ __forceinline__ float block_sum(float x) {
    __shared__ float part[kThreads / 64];
    x = lanes_sum_f32<64>(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    return ((part[0] + part[1]) + part[2]) + part[3];
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

template <int X>
__device__ __forceinline__ uint64_t at(const Images& m, int64_t n, int64_t s, int64_t c) {
    return reinterpret_cast<uint64_t>(m.data) + (uint64_t)(n * m.sample + s * m.ld + c * kSize<X>);
}

template <int X, int P>
__global__ __launch_bounds__(kThreads) void k_gn_fwd(GnArgs a, int32_t C, int32_t G, int32_t act) {
    const int32_t cg = C / G;
    for (int64_t b = blockIdx.x; b < a.N * G; b += gridDim.x) {
        const int64_t n = b / G, c0 = b % G * cg, count = a.S * cg;
        auto value = [&](int64_t i) { return load_one<X>(at<X>(a.x, n, i / cg, c0 + i % cg)); };
        const float first = value(0);
        float s = 0.f, q = 0.f;
        for (int64_t i = threadIdx.x; i < count; i += kThreads) s += value(i) - first;
        const float mean = first + block_sum(s) / (float)count;
        float off = 0.f;
        for (int64_t i = threadIdx.x; i < count; i += kThreads) {
            const float d = value(i) - mean;
            q = fmaf(d, d, q);
            off += d;
        }
        off = block_sum(off) / (float)count;
        const float var = fmaxf(block_sum(q) / (float)count - off * off, 0.f), rstd = 1.f / sqrtf(var + a.eps);
        for (int64_t i = threadIdx.x; i < count; i += kThreads) {
            const int64_t c = c0 + i % cg;
            float z = fmaf((value(i) - mean - off) * rstd, param<P>(a.gamma, c, 1.f), param<P>(a.beta, c, 0.f));
            if (act == GA_ACT_RELU) z = z < 0.f ? 0.f : z;
            else if (act == GA_ACT_SILU) z = z * sigmoid(z);
            store_one<X>(at<X>(a.y, n, i / cg, c), z);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[b] = mean + off;
            if (a.rstd) a.rstd[b] = rstd;
        }
    }
}

// dz of one element, from xh.
__device__ __forceinline__ float before_act(float dy, float xh, float gamma, float beta, int32_t act) {
    if (act == GA_ACT_NONE) return dy;
    const float z = fmaf(xh, gamma, beta);
    if (act == GA_ACT_RELU) return z <= 0.f ? 0.f : dy;
    const float s = sigmoid(z);
    return dy * (s * fmaf(z, 1.f - s, 1.f));
}

template <int X, int P>
__global__ __launch_bounds__(kThreads) void k_gn_dx(GnArgs a, int32_t C, int32_t G, int32_t act) {
    const int32_t cg = C / G;
    for (int64_t b = blockIdx.x; b < a.N * G; b += gridDim.x) {
        const int64_t n = b / G, c0 = b % G * cg, count = a.S * cg;
        const float mean = a.mean[b], rstd = a.rstd[b];
        auto value = [&](int64_t i, float& xh) {
            const int64_t s = i / cg, c = c0 + i % cg;
            const float gamma = param<P>(a.gamma, c, 1.f);
            xh = (load_one<X>(at<X>(a.x, n, s, c)) - mean) * rstd;
            return before_act(load_one<X>(at<X>(a.dy, n, s, c)), xh, gamma, param<P>(a.beta, c, 0.f), act) * gamma;
        };
        float s1 = 0.f, s2 = 0.f, xh;
        for (int64_t i = threadIdx.x; i < count; i += kThreads) {
            const float h = value(i, xh);
            s1 += h;
            s2 = fmaf(h, xh, s2);
        }
        s1 = block_sum(s1) / (float)count;
        s2 = block_sum(s2) / (float)count;
        for (int64_t i = threadIdx.x; i < count; i += kThreads) {
            const float h = value(i, xh);
            store_one<X>(at<X>(a.y, n, i / cg, c0 + i % cg), rstd * (h - fmaf(xh, s2, s1)));
        }
    }
}

template <int X, int P>
__global__ __launch_bounds__(64) void k_gn_params(GnArgs a, int32_t C, int32_t G, int32_t act) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x, w = blockIdx.y;
    if (c >= C) return;
    const float gamma = param<P>(a.gamma, c, 1.f), beta = param<P>(a.beta, c, 0.f);
    double dg = 0.0, db = 0.0;
    for (int64_t n = w * a.per_worker; n < (w + 1) * a.per_worker; ++n) {
        const int64_t b = n * G + c / (C / G);
        for (int64_t s = 0; s < a.S; ++s) {
            const float xh = (load_one<X>(at<X>(a.x, n, s, c)) - a.mean[b]) * a.rstd[b];
            const float dz = before_act(load_one<X>(at<X>(a.dy, n, s, c)), xh, gamma, beta, act);
            dg += (double)(dz * xh);
            db += (double)dz;
        }
    }
    auto put = [&](void* out, float x) {
        if (a.dp_dtype == kF32) static_cast<float*>(out)[w * C + c] = x;
        else if (a.dp_dtype == kF16) store_one<kF16>(reinterpret_cast<uint64_t>(out) + (uint64_t)(w * C + c) * 2, x);
        else store_one<kB16>(reinterpret_cast<uint64_t>(out) + (uint64_t)(w * C + c) * 2, x);
    };
    put(a.dgamma, (float)dg);
    put(a.dbeta, (float)db);
}

template <int X, int P>
hipError_t gn_fwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    const int64_t want = a.N * n.G;
    hipLaunchKernelGGL((k_gn_fwd<X, P>), dim3((unsigned)(want < 65536 ? want : 65536)), dim3(kThreads), 0, s, a, n.C, n.G,
                       n.act);
    return hipGetLastError();
}

template <int X, int P>
hipError_t gn_bwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    if (a.dgamma) {
        hipLaunchKernelGGL((k_gn_params<X, P>), dim3((unsigned)((n.C + 63) / 64), (unsigned)a.workers), dim3(64), 0, s, a,
                           n.C, n.G, n.act);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.N == 0) return e;
    }
    const int64_t want = a.N * n.G;
    hipLaunchKernelGGL((k_gn_dx<X, P>), dim3((unsigned)(want < 65536 ? want : 65536)), dim3(kThreads), 0, s, a, n.C, n.G,
                       n.act);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gn_fwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    if (n.x_dtype == GA_FP32) return gn_fwd<kF32, kF32>(n, a, s);
    if (n.x_dtype == GA_FP16) return n.p_dtype == GA_FP32 ? gn_fwd<kF16, kF32>(n, a, s) : gn_fwd<kF16, kF16>(n, a, s);
    return n.p_dtype == GA_FP32 ? gn_fwd<kB16, kF32>(n, a, s) : gn_fwd<kB16, kB16>(n, a, s);
}

hipError_t launch_gn_bwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    if (n.x_dtype == GA_FP32) return gn_bwd<kF32, kF32>(n, a, s);
    if (n.x_dtype == GA_FP16) return n.p_dtype == GA_FP32 ? gn_bwd<kF16, kF32>(n, a, s) : gn_bwd<kF16, kF16>(n, a, s);
    return n.p_dtype == GA_FP32 ? gn_bwd<kB16, kF32>(n, a, s) : gn_bwd<kB16, kB16>(n, a, s);
}

}  // namespace ga
