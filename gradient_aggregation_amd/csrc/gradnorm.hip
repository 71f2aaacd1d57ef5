// L2 norm of the mean gradient over all layers (ga_grad_norm).
//
// k_grad_norm reads each gradient once (grads.h) and leaves one binary64 sum
// of squares per workgroup (each square is exact in binary64); k_grad_norm_end
// adds them in a fixed order and forms the clip record.  Bound by memory: W * b
// bytes per element, 4 more where the mean gradient is kept.
#include "grads.h"

namespace ga {

namespace {

constexpr int kThreads = 256;
constexpr int kEndThreads = 1024;

template <int T, int LEV>
__global__ __launch_bounds__(kThreads) void k_grad_norm(GradArgs a, int64_t n_tiles, float* __restrict__ grad,
                                                        double* __restrict__ partials) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    double acc0 = 0.0, acc1 = 0.0;
    for (int64_t tile = (int64_t)blockIdx.x * (kThreads / 64) + wave; tile < n_tiles;
         tile += (int64_t)gridDim.x * (kThreads / 64)) {
        const TileRec rec = a.tiles[tile];
        float g[8];
        uint32_t dmask;
        if (rec.flags & kTileWhole) mean_grad_whole<T, LEV>(a, tile, rec, lane, g);
        else mean_grad_part<T, LEV>(a, tile, rec, lane, g, dmask);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            acc0 = fma((double)g[e], (double)g[e], acc0);
            acc1 = fma((double)g[e + 1], (double)g[e + 1], acc1);
        }
        if (grad) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t i = group_at(tile, lane, q);
                if (i + 4 <= a.P) {
                    __builtin_nontemporal_store(f32x4{g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]},
                                                reinterpret_cast<f32x4*>(grad + i));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i + e < a.P) grad[i + e] = g[4 * q + e];
                }
            }
        }
    }
    const double t = wave_sum_f64(acc0 + acc1);
    __shared__ double part[kThreads / 64];
    if (lane == 0) part[wave] = t;
    __syncthreads();
    if (threadIdx.x == 0) partials[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(kEndThreads) void k_grad_norm_end(const double* __restrict__ partials, int32_t n,
                                                               float max_norm, ga_clip* __restrict__ clip) {
    double t = 0.0;
    for (int32_t i = threadIdx.x; i < n; i += kEndThreads) t += partials[i];
    t = wave_sum_f64(t);
    __shared__ double part[kEndThreads / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x != 0) return;
    t = 0.0;
    for (int j = 0; j < kEndThreads / 64; ++j) t += part[j];
    const float norm = (float)sqrt(t);
    const float scale = max_norm / norm;
    clip->norm = norm;
    clip->scale = scale > 1.f ? 1.f : scale;
    clip->skip = norm < __builtin_inff() ? 0 : 1;   // infinite or NaN
    clip->unused = 0;
}

template <int T>
hipError_t norm_launch(const Adamw& o, const uint64_t* layer_ptrs, float max_norm, float* grad, ga_clip* clip,
                       hipStream_t s) {
    const GradArgs g = grad_args(o, layer_ptrs);
    const int64_t want = (o.n_tiles + kThreads / 64 - 1) / (kThreads / 64);
    const int32_t blocks = (int32_t)(want < kNormBlocks ? want : kNormBlocks);
    const hipError_t e = with_levels(o.W, [&](auto lev) {
        hipLaunchKernelGGL((k_grad_norm<T, decltype(lev)::value>), dim3(blocks), dim3(kThreads), 0, s, g,
                           o.n_tiles, grad, o.d_partials);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_grad_norm_end, dim3(1), dim3(kEndThreads), 0, s, o.d_partials, blocks, max_norm, clip);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad_norm(const Adamw& o, const uint64_t* layer_ptrs, float max_norm, float* grad, ga_clip* clip,
                            hipStream_t s) {
    if (o.dtype == GA_FP32) return norm_launch<kF32>(o, layer_ptrs, max_norm, grad, clip, s);
    if (o.dtype == GA_FP16) return norm_launch<kF16>(o, layer_ptrs, max_norm, grad, clip, s);
    return norm_launch<kB16>(o, layer_ptrs, max_norm, grad, clip, s);
}

}  // namespace ga
