// Router of a mixture of experts with its counts and balance loss
// (ga_router_forward, ga_router_backward): the plainest form.  A wavefront takes a
// token, up to 16 experts to a lane.
#include "elements.h"
#include "layers.h"

namespace ga {

namespace {

constexpr int kMost = GA_MAX_EXPERTS / 64;

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, 64));
    return x;
}

__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x = min(x, __shfl_xor(x, off, 64));
    return x;
}

// Softmax and selection of one token.
template <int X>
__global__ __launch_bounds__(64) void k_route(RouteArgs a, int32_t E, int32_t k, int32_t normalize) {
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const uint64_t row = reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx);
        const bool masked = a.mask && !a.mask[t];
        float l[kMost], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int e = i * 64 + lane;
            l[i] = e < E && !masked ? load_one<X>(row + (uint64_t)e * kSize<X>) : -INFINITY;
            top = fmaxf(top, l[i]);
        }
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < kMost; ++i) sum += l[i] == -INFINITY ? 0.f : expf(l[i] - top);
        sum = lanes_sum_f32<64>(sum);
        const bool absent = sum == 0.f;
        const float lse = absent ? 0.f : top + logf(sum);
        float mine = 0.f, chosen = 0.f;     // lane j: exp(logit - top) of slot j
        for (int j = 0; j < k; ++j) {
            int at = -1;
            if (!a.select) {
                const int e = a.r.experts[t * k + j];
                at = e >= 0 && e < E ? e : -1;
            } else if (!absent) {
                float best = -INFINITY;
#pragma unroll
                for (int i = 0; i < kMost; ++i) best = fmaxf(best, l[i]);
                best = wave_max(best);
                int first = 1 << 30;
#pragma unroll
                for (int i = kMost - 1; i >= 0; --i)
                    if (l[i] == best) first = i * 64 + lane;
                first = wave_min(first);
                if (best > -INFINITY) at = first;
#pragma unroll
                for (int i = 0; i < kMost; ++i)
                    if (i * 64 + lane == at) l[i] = -INFINITY;
            }
            float g = 0.f;
            if (at >= 0 && !absent) {
                const float x = load_one<X>(row + (uint64_t)at * kSize<X>);
                g = x == -INFINITY ? 0.f : expf(x - top);
            }
            chosen += g;
            if (lane == j) {
                mine = g;
                if (a.select) a.r.experts[t * k + j] = at;
            }
        }
        float by = normalize ? chosen : sum;
        if (sum != sum) by = sum;
        if (a.r.gates && lane < k) a.r.gates[t * k + lane] = by == 0.f ? 0.f : mine / by;
        if (a.r.lse && lane == 0) a.r.lse[t] = lse;
    }
}

// The load of worker blockIdx.x, from the logits and the experts.
template <int X>
__global__ __launch_bounds__(256) void k_load(RouteArgs a, int32_t E, int32_t k, double* __restrict__ out) {
    __shared__ int count[GA_MAX_EXPERTS];
    __shared__ float top_of, sum_of;
    __shared__ double squares;
    const int64_t w = blockIdx.x;
    double p[GA_MAX_EXPERTS / 256] = {};
    int n = 0;
    for (int e = threadIdx.x; e < GA_MAX_EXPERTS; e += 256) count[e] = 0;
    if (threadIdx.x == 0) squares = 0.0;
    for (int64_t t = w * a.per_worker; t < (w + 1) * a.per_worker; ++t) {
        if (a.mask && !a.mask[t]) continue;
        const uint64_t row = reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx);
        __syncthreads();
        if (threadIdx.x < 64) {
            float top = -INFINITY, sum = 0.f;
            for (int e = threadIdx.x; e < E; e += 64) top = fmaxf(top, load_one<X>(row + (uint64_t)e * kSize<X>));
            top = wave_max(top);
            for (int e = threadIdx.x; e < E; e += 64) {
                const float l = load_one<X>(row + (uint64_t)e * kSize<X>);
                sum += l == -INFINITY ? 0.f : expf(l - top);
            }
            sum = lanes_sum_f32<64>(sum);
            if (threadIdx.x == 0) {
                top_of = top;
                sum_of = sum;
                if (sum != 0.f) {
                    const double lse = (double)top + log((double)sum);
                    squares += lse * lse;
                }
            }
        }
        __syncthreads();
        if (sum_of == 0.f) continue;
        ++n;
        for (int i = 0; i < GA_MAX_EXPERTS / 256; ++i) {
            const int e = i * 256 + threadIdx.x;
            if (e < E) {
                const float l = load_one<X>(row + (uint64_t)e * kSize<X>);
                p[i] += l == -INFINITY && sum_of == sum_of ? 0.0 : (double)(expf(l - top_of) / sum_of);
            }
        }
        if (threadIdx.x < k) {
            const int e = a.r.experts[t * k + threadIdx.x];
            if (e >= 0 && e < E) atomicAdd(&count[e], 1);
        }
    }
    __syncthreads();
    for (int i = 0; i < GA_MAX_EXPERTS / 256; ++i) {
        const int e = i * 256 + threadIdx.x;
        if (e < E) {
            a.load.counts[w * E + e] = count[e];
            a.load.probs[w * E + e] = (float)p[i];
        }
    }
    if (threadIdx.x == 0) {
        a.load.tokens[w] = n;
        out[w] = squares;
    }
}

__global__ __launch_bounds__(64) void k_loss(RouteArgs a, int32_t E, int32_t k, int32_t W, int32_t scope,
                                             const double* __restrict__ squares) {
    if (threadIdx.x != 0) return;
    double loss = 0.0, z = 0.0, all = 0.0;
    for (int w = 0; w < W; ++w) all += a.load.tokens[w];
    const int S = scope == GA_BALANCE_ALL ? 1 : W;
    for (int s = 0; s < S; ++s) {
        const double n = S == 1 ? all : a.load.tokens[s], share = n > 0 ? 1.0 / n / S : 0.0;
        for (int e = 0; e < E; ++e) {
            double F = 0.0, P = 0.0;
            for (int w = S == 1 ? 0 : s; w < (S == 1 ? W : s + 1); ++w) {
                F += a.load.counts[(int64_t)w * E + e];
                P += a.load.probs[(int64_t)w * E + e];
            }
            const double slope = n > 0 ? F * E / k / n * share : 0.0;
            a.load.slope[(int64_t)s * (E + 1) + e] = (float)slope;
            loss += slope * P;
        }
        a.load.slope[(int64_t)s * (E + 1) + E] = (float)(2.0 * share);
        for (int w = S == 1 ? 0 : s; w < (S == 1 ? W : s + 1); ++w) z += squares[w] * share;
    }
    a.load.loss[0] = (float)loss;
    a.load.loss[1] = (float)z;
}

template <int X>
__global__ __launch_bounds__(64) void k_route_bwd(RouteArgs a, int32_t E, int32_t k, int32_t normalize, int32_t S,
                                                  int64_t per_slope) {
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const uint64_t row = reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx);
        const uint64_t out = reinterpret_cast<uint64_t>(a.dx) + (uint64_t)(t * a.ldd);
        float p[kMost], h[kMost], direct[kMost], lse = a.r.lse[t];
        float any = -INFINITY;
        const bool masked = a.mask && !a.mask[t];
        const float* slope = a.slope ? a.slope + t / per_slope * (E + 1) : nullptr;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int e = i * 64 + lane;
            const float l = e < E && !masked ? load_one<X>(row + (uint64_t)e * kSize<X>) : -INFINITY;
            any = l != l ? INFINITY : fmaxf(any, l);
            p[i] = l == -INFINITY && lse == lse ? 0.f : expf(l - lse);
            h[i] = slope && e < E ? a.balance * slope[e] : 0.f;
            direct[i] = 0.f;
        }
        const bool absent = wave_max(any) == -INFINITY;
        float inner = 0.f;
        if (a.dgates && !absent) {
            if (normalize)
                for (int j = 0; j < k; ++j) inner = fmaf(a.r.gates[t * k + j], a.dgates[t * k + j], inner);
            for (int j = 0; j < k; ++j) {
                const int at = a.r.experts[t * k + j];
#pragma unroll
                for (int i = 0; i < kMost; ++i) {
                    if (i * 64 + lane != at) continue;
                    if (normalize) direct[i] = fmaf(a.r.gates[t * k + j], a.dgates[t * k + j] - inner, direct[i]);
                    else h[i] += a.dgates[t * k + j];
                }
            }
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (i * 64 + lane < E) dot = fmaf(h[i], p[i], dot);
        dot = lanes_sum_f32<64>(dot);
        const float shift = (slope ? a.z * slope[E] * lse : 0.f) - dot;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int e = i * 64 + lane;
            if (e < E) store_one<X>(out + (uint64_t)e * kSize<X>, absent ? 0.f : fmaf(p[i], h[i] + shift, direct[i]));
        }
    }
}

template <int X>
hipError_t router_fwd(const Router& r, const RouteArgs& a, hipStream_t s) {
    if (a.T > 0) {
        hipLaunchKernelGGL(k_route<X>, dim3((unsigned)(a.T < 65536 ? a.T : 65536)), dim3(64), 0, s, a, r.E, r.k, r.normalize);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.with_load) return hipSuccess;
    hipLaunchKernelGGL(k_load<X>, dim3((unsigned)r.W), dim3(256), 0, s, a, r.E, r.k, r.d_squares);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_loss, dim3(1), dim3(64), 0, s, a, r.E, r.k, r.W, r.scope, r.d_squares);
    return hipGetLastError();
}

template <int X>
hipError_t router_bwd(const Router& r, const RouteArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_route_bwd<X>, dim3((unsigned)(a.T < 65536 ? a.T : 65536)), dim3(64), 0, s, a, r.E, r.k, r.normalize,
                       r.scope == GA_BALANCE_ALL ? 1 : r.W, r.scope == GA_BALANCE_ALL ? a.T : a.per_worker);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_router_fwd(const Router& r, const RouteArgs& a, hipStream_t s) {
    if (r.x_dtype == GA_FP32) return router_fwd<kF32>(r, a, s);
    if (r.x_dtype == GA_FP16) return router_fwd<kF16>(r, a, s);
    return router_fwd<kB16>(r, a, s);
}

hipError_t launch_router_bwd(const Router& r, const RouteArgs& a, hipStream_t s) {
    if (r.x_dtype == GA_FP32) return router_bwd<kF32>(r, a, s);
    if (r.x_dtype == GA_FP16) return router_bwd<kF16>(r, a, s);
    return router_bwd<kB16>(r, a, s);
}

}  // namespace ga
