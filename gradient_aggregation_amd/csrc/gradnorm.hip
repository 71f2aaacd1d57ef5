// L2 norm of the mean gradient over all layers (ga_grad_norm).
//
// k_grad_norm reads each gradient once (grads.h) and leaves one binary64 sum
// of squares per workgroup (each square is exact in binary64); they are added
// in a fixed order, which forms the clip record.  Bound by memory: W * b bytes
// per element, 4 more where the mean gradient is kept.  122 MB of bf16 gradients
// take 22 us (5.5 TB/s) and the second kernel 4 us; 20M of 16 binary16 workers
// 128 us with it (172 when the tiles that straddle layers came in turn).  A wavefront takes one tile
// at a time: 2, 4 or 8 read together took 23 to 34 us, on 512 to 16384
// workgroups, next to each other or a grid apart.
#include "grads.h"

namespace ga {

namespace {

constexpr int kThreads = 256;
constexpr int kWavesPer = kThreads / 64;
constexpr int kEndThreads = 1024;

// Up to this many workgroups the one that ends last adds the partial sums
// itself; above, a second kernel does, which costs a launch but not a release
// of each workgroup's sum to the other XCDs and an addition to one counter: 7.1
// against 9.6 us a call with 16 to 128 workgroups, 8.6 against 9.7 with 256,
// 12.0 against 9.8 with 512.
constexpr int kOneLaunch = 256;

// Sum over the wavefronts of a workgroup, in order (the result is thread 0's).
template <int THREADS>
__device__ __forceinline__ double block_sum(double wave) {
    __shared__ double part[THREADS / 64];
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = wave;
    __syncthreads();
    double t = part[0];
    for (int j = 1; j < THREADS / 64; ++j) t += part[j];
    return t;
}

__device__ __forceinline__ void write_clip(double squares, float max_norm, ga_clip* clip) {
    const float norm = (float)sqrt(squares);
    const float scale = max_norm / norm;
    clip->norm = norm;
    clip->scale = scale > 1.f ? 1.f : scale;
    clip->skip = norm < __builtin_inff() ? 0 : 1;   // infinite or NaN
    clip->unused = 0;
}

template <int T, int LEV, bool ONE>
__global__ __launch_bounds__(kThreads) void k_grad_norm(GradArgs a, int64_t n_tiles, float* __restrict__ grad,
                                                        double* __restrict__ partials, uint32_t* __restrict__ done,
                                                        float max_norm, ga_clip* __restrict__ clip) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    double acc0 = 0.0, acc1 = 0.0;
    for (int64_t slot = (int64_t)blockIdx.x * kWavesPer + wave; slot < n_tiles;
         slot += (int64_t)gridDim.x * kWavesPer) {
        const TileRec rec = a.tiles[slot];
        const int64_t tile = rec.tile;
        float g[8];
        uint32_t dmask;
        if (rec.flags & kTileWhole) mean_grad_whole<T, LEV>(a, tile, rec, lane, g);
        else mean_grad_part<T, LEV>(a, tile, rec, lane, g, dmask);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            acc0 = fma((double)g[e], (double)g[e], acc0);
            acc1 = fma((double)g[e + 1], (double)g[e + 1], acc1);
        }
        if (!grad) continue;
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
    const double t = block_sum<kThreads>(wave_sum_f64(acc0 + acc1));
    if constexpr (!ONE) {
        if (threadIdx.x == 0) partials[blockIdx.x] = t;
    } else {
        __shared__ uint32_t last;
        if (threadIdx.x == 0) {
            __hip_atomic_store(partials + blockIdx.x, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x;
        }
        __syncthreads();
        if (!last) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        double all = 0.0;
        for (uint32_t i = threadIdx.x; i < gridDim.x; i += kThreads)
            all += __hip_atomic_load(partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        all = block_sum<kThreads>(wave_sum_f64(all));
        if (threadIdx.x != 0) return;
        write_clip(all, max_norm, clip);
        __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
    }
}

__global__ __launch_bounds__(kEndThreads) void k_grad_norm_end(const double* __restrict__ partials, int32_t n,
                                                               float max_norm, ga_clip* __restrict__ clip) {
    double t = 0.0;
    for (int32_t i = threadIdx.x; i < n; i += kEndThreads) t += partials[i];
    t = block_sum<kEndThreads>(wave_sum_f64(t));
    if (threadIdx.x == 0) write_clip(t, max_norm, clip);
}

template <int T>
hipError_t norm_launch(const Adamw& o, const uint64_t* layer_ptrs, float max_norm, float* grad, ga_clip* clip,
                       hipStream_t s) {
    const GradArgs g = grad_args(o, layer_ptrs);
    const int64_t want = (o.n_tiles + kWavesPer - 1) / kWavesPer;
    const int32_t blocks = (int32_t)(want < kNormBlocks ? want : kNormBlocks);
    return with_levels(o.W, [&](auto lev) {
        constexpr int LEV = decltype(lev)::value;
        if (blocks <= kOneLaunch) {
            hipLaunchKernelGGL((k_grad_norm<T, LEV, true>), dim3(blocks), dim3(kThreads), 0, s, g, o.n_tiles, grad,
                               o.d_partials, o.d_done, max_norm, clip);
            return hipGetLastError();
        }
        hipLaunchKernelGGL((k_grad_norm<T, LEV, false>), dim3(blocks), dim3(kThreads), 0, s, g, o.n_tiles, grad,
                           o.d_partials, o.d_done, max_norm, clip);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_grad_norm_end, dim3(1), dim3(kEndThreads), 0, s, o.d_partials, blocks, max_norm, clip);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_grad_norm(const Adamw& o, const uint64_t* layer_ptrs, float max_norm, float* grad, ga_clip* clip,
                            hipStream_t s) {
    if (o.dtype == GA_FP32) return norm_launch<kF32>(o, layer_ptrs, max_norm, grad, clip, s);
    if (o.dtype == GA_FP16) return norm_launch<kF16>(o, layer_ptrs, max_norm, grad, clip, s);
    return norm_launch<kB16>(o, layer_ptrs, max_norm, grad, clip, s);
}

}  // namespace ga
