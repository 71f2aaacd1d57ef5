// Layer norm over rows, forward and backward (ga_layernorm_forward,
// ga_layernorm_backward).
//
// Forward: a row is read once and stays in registers, spread over T threads as
// V vectors of 16 bytes each; its mean and then the sum of squared deviations
// from that mean are reduced across the threads.  A mean of n values is off by
// several roundings of their size, which matters where that is many times the
// row's deviation: there the deviations are summed as well, and their mean
// corrects the first one (constant binary32 rows near 10000, 1001 wide, came out
// up to 0.68 from their bias).  Such rows take 6% to 15% longer (16384 x 4096,
// 4096 x 12288 bf16), those past 16384 elements 21%; the others do not.
//
// Backward: one pass over the rows as well; each thread keeps the weight and the
// two weight-gradient sums of its columns in registers over all the rows its
// workgroup takes, and the workgroup writes them as one partial row at the end.
// The partial rows of each group are added in a fixed order.
//
// Bound by memory: b * (2 to 4) bytes per element forward, b * (3 to 4)
// backward, against some 15 to 25 instructions.  16384 x 4096 bf16 rows, one
// pass after the other: 93 to 99 us forward with the residual (5.8 to 5.4 TB/s: it
// differs between cards, not between runs on one), 95 us backward with it (5.6
// TB/s).
// The backward pass takes one workgroup of 1024 threads per CU: with two of 512
// as many rows are on their way, but twice the partial rows are written and
// read (105 us), with two of 256 the chip waits for memory (110 us).
//
// Loads and stores carry the streaming hint where that was faster: all of the
// outputs forward (30000 x 512 binary32: 24.5 -> 19.5 us), the inputs forward
// where there is a residual (4096 x 5120 binary32: 60.4 -> 57.8 us; without one
// 16384 x 1024 bf16 rows took 14.5 us with it, 12.7 without), the inputs
// backward (16384 x 4096 bf16: 103 -> 92 us) but not dx (8192 x 8192 binary16:
// 87 us, 89 with it).
#include <type_traits>

#include "elements.h"
#include "training.h"

namespace ga {

namespace {

template <int X>
constexpr int kVec = 16 / kSize<X>;     // elements of a 128-bit vector

// Rows wider than this do not stay in registers: they are read again in each
// pass (from the caches, at these lengths).
constexpr int64_t kInRegisters = 16384;
constexpr int kLongThreads = 1024;
constexpr int kBwdThreads = 1024;

// Elements [c, c + N) of a row that ends at dim; those past it are 0.
template <int X, int N, bool NT = false>
__device__ __forceinline__ void load_part(Raw<X, N>& r, uint64_t row, int64_t c, int64_t dim) {
    const uint64_t at = row + (uint64_t)c * kSize<X>;
    if (c + N <= dim) {
        r.template load<NT>(at);
        return;
    }
    float f[N];
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = 0.f;
    if (c < dim) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + e < dim) f[e] = load_one<X>(at + e * kSize<X>);
    }
    r.narrow(f);
}

// The same in two steps, for rows read ahead: the load itself, in which the
// vector that would pass the end is read from where it ends there instead (a
// load per element would have to be waited for at once), and the shift that
// moves its elements into place and fills up with zeros.
template <int X, int N, bool NT>
__device__ __forceinline__ void load_ahead(Raw<X, N>& r, uint64_t row, int32_t c, int32_t dim) {
    if (dim < N) {
        load_part(r, row, c, dim);
    } else if (c < dim) {
        r.template load<NT>(row + (uint64_t)((c < dim - N ? c : dim - N) * kSize<X>));
    } else {
#pragma unroll
        for (int j = 0; j < Raw<X, N>::WORDS; ++j) r.w[j] = 0u;
    }
}

template <int X, int N>
__device__ __forceinline__ void into_place(Raw<X, N>& r, int32_t c, int32_t dim) {
    static_assert(Raw<X, N>::WORDS == 4, "a 128-bit vector");
    if (dim < N || dim % N == 0) return;
    const int past = c + N - dim;
    const uint32_t s = past > 0 && past < N ? past : 0;   // elements to drop
    const uint32_t words = s * kSize<X> / 4;
    if (words & 2u) {
        r.w[0] = r.w[2];
        r.w[1] = r.w[3];
        r.w[2] = r.w[3] = 0u;
    }
    if (words & 1u) {
        r.w[0] = r.w[1];
        r.w[1] = r.w[2];
        r.w[2] = r.w[3];
        r.w[3] = 0u;
    }
    if (kSize<X> == 2 && (s & 1u)) {
        r.w[0] = __builtin_amdgcn_alignbit(r.w[1], r.w[0], 16);
        r.w[1] = __builtin_amdgcn_alignbit(r.w[2], r.w[1], 16);
        r.w[2] = __builtin_amdgcn_alignbit(r.w[3], r.w[2], 16);
        r.w[3] >>= 16;
    }
}

template <int X, bool NT = false, int N>
__device__ __forceinline__ void store_part(const float (&f)[N], uint64_t row, int64_t c, int64_t dim) {
    const uint64_t at = row + (uint64_t)c * kSize<X>;
    if (c + N <= dim) {
        Raw<X, N> r;
        r.narrow(f);
        r.template store<NT>(at);
    } else if (c < dim) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + e < dim) store_one<X>(at + e * kSize<X>, f[e]);
    }
}

// N elements of a weight vector from column c (fill where it is not given or
// past dim).
template <int P, int N>
__device__ __forceinline__ void load_param(float (&f)[N], const void* p, int64_t c, int64_t dim, float fill) {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = fill;
    if (!p || c >= dim) return;
    const uint64_t at = reinterpret_cast<uint64_t>(p) + (uint64_t)c * kSize<P>;
    if (c + N <= dim) {
        Raw<P, N> r;
        r.load(at);
        r.widen(f);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + e < dim) f[e] = load_one<P>(at + e * kSize<P>);
    }
}

// T threads take a row.  Teams of up to a wavefront share a workgroup of 256;
// a larger team is a workgroup.
template <int T>
constexpr int kTeamRows = T <= 64 ? 256 / T : 1;
template <int T>
constexpr int kTeamThreads = T <= 64 ? 256 : T;
template <int T>
constexpr int kTeamWaves = T <= 64 ? 1 : T / 64;

// Sum over a team (of more than a wavefront through LDS: buf holds a value per
// wavefront and must not be written again before the next barrier).
template <int T>
__device__ __forceinline__ float team_sum(float x, float* buf) {
    x = lanes_sum_f32<T < 64 ? T : 64>(x);
    if constexpr (T <= 64) return x;
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    float t = buf[0];
#pragma unroll
    for (int j = 1; j < T / 64; ++j) t += buf[j];
    return t;
}

// Whether a row's mean, as it was first rounded, has to be corrected: past four
// deviations.  Up to there the error that it leaves in y is at most four times
// that of a row about zero.  The same for all threads of a team, whose sums have
// the same bits; false where the row holds an infinity or NaN.
__device__ __forceinline__ bool far_from_zero(float mean, float var, float eps) {
    return mean * mean > 16.f * (var + eps);
}

// The correction: off is the deviations' mean, var their mean square.
__device__ __forceinline__ void correct(float& mean, float& var, float off) {
    mean += off;
    var = var > off * off ? var - off * off : 0.f;
}

template <int X, int P, int T, int V>
__global__ __launch_bounds__(kTeamThreads<T>) void k_ln_fwd(LnFwd a, int32_t dim) {
    constexpr int N = kVec<X>, R = kTeamRows<T>;
    __shared__ float red[3][kTeamWaves<T>];
    const int t = threadIdx.x % T;
    float gamma[V][N], beta[V][N];
    int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / T;
    Raw<X, N> x[V], r[V];
    auto load_row = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * N;
            const uint64_t at = reinterpret_cast<uint64_t>(a.x) + (uint64_t)(row * a.ldx);
            if (a.res) {
                load_ahead<X, N, true>(x[v], at, c, dim);
                load_ahead<X, N, true>(r[v], reinterpret_cast<uint64_t>(a.res) + (uint64_t)(row * a.ldr), c, dim);
            } else {
                load_ahead<X, N, false>(x[v], at, c, dim);
            }
        }
    };
    if (row < a.rows) load_row(row);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        load_param<P>(gamma[v], a.gamma, (v * T + t) * N, dim, 1.f);
        load_param<P>(beta[v], a.beta, (v * T + t) * N, dim, 0.f);
    }
    const float inv_dim = (float)(1.0 / (double)dim);
    for (; row < a.rows; row += (int64_t)gridDim.x * R) {
        float f[V][N];
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            into_place(x[v], (v * T + t) * N, dim);
            x[v].widen(f[v]);
            if (a.res) {
                float h[N];
                into_place(r[v], (v * T + t) * N, dim);
                r[v].widen(h);
                // the sum is rounded to x's type, as it is stored, before it is normalised
#pragma unroll
                for (int e = 0; e < N; ++e) f[v][e] = f[v][e] + h[e];
                Raw<X, N> s;
                s.narrow(f[v]);
                s.widen(f[v]);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) sum += f[v][e];
        }
        const int64_t next = row + (int64_t)gridDim.x * R;
        if (next < a.rows) load_row(next);
        float mean = team_sum<T>(sum, red[0]) * inv_dim;
        // only now has the whole team read the row, which the sum may overwrite
        if (a.sum) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                store_part<X, true>(f[v], reinterpret_cast<uint64_t>(a.sum) + (uint64_t)(row * a.lds), (v * T + t) * N,
                                    dim);
        }
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int left = dim - (v * T + t) * N;
#pragma unroll
            for (int e = 0; e < N; ++e) f[v][e] -= mean;
            if (left >= N) {
#pragma unroll
                for (int e = 0; e < N; ++e) sq = fmaf(f[v][e], f[v][e], sq);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (e < left) sq = fmaf(f[v][e], f[v][e], sq);
            }
        }
        float var = team_sum<T>(sq, red[1]) * inv_dim, off = 0.f;
        if (far_from_zero(mean, var, a.eps)) {
            float sd = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int left = dim - (v * T + t) * N;
#pragma unroll
                for (int e = 0; e < N; ++e) sd += e < left ? f[v][e] : 0.f;
            }
            off = team_sum<T>(sd, red[2]) * inv_dim;
            correct(mean, var, off);
        }
        const float rstd = 1.f / sqrtf(var + a.eps);
        const float shift = -off * rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int e = 0; e < N; ++e) f[v][e] = fmaf(fmaf(f[v][e], rstd, shift), gamma[v][e], beta[v][e]);
            store_part<X, true>(f[v], reinterpret_cast<uint64_t>(a.y) + (uint64_t)(row * a.ldy), (v * T + t) * N, dim);
        }
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Rows that do not stay in registers: a workgroup per row, three passes.
template <int X, int P>
__global__ __launch_bounds__(kLongThreads) void k_ln_fwd_long(LnFwd a, int64_t dim) {
    constexpr int N = kVec<X>, T = kLongThreads;
    __shared__ float red[3][T / 64];
    const float inv_dim = (float)(1.0 / (double)dim);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const uint64_t xr = reinterpret_cast<uint64_t>(a.x) + (uint64_t)(row * a.ldx);
        const uint64_t rr = reinterpret_cast<uint64_t>(a.res) + (uint64_t)(row * a.ldr);
        const uint64_t sr = reinterpret_cast<uint64_t>(a.sum) + (uint64_t)(row * a.lds);
        const uint64_t yr = reinterpret_cast<uint64_t>(a.y) + (uint64_t)(row * a.ldy);
        auto value = [&](int64_t c, float (&f)[N]) {
            Raw<X, N> x;
            load_part(x, xr, c, dim);
            x.widen(f);
            if (a.res) {
                float h[N];
                load_part(x, rr, c, dim);
                x.widen(h);
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] = rounded<X>(f[e] + h[e]);
            }
        };
        // y or sum may be x or the residual: the later passes read the sum
        // where it was stored, else form it again (y is written last)
        auto again = [&](int64_t c, float (&f)[N]) {
            if (a.res && a.sum) {
                Raw<X, N> x;
                load_part(x, sr, c, dim);
                x.widen(f);
            } else {
                value(c, f);
            }
        };
        float sum = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * N; c < dim; c += T * N) {
            float f[N];
            value(c, f);
            if (a.res && a.sum) store_part<X>(f, sr, c, dim);
#pragma unroll
            for (int e = 0; e < N; ++e) sum += f[e];
        }
        const float first = team_sum<T>(sum, red[0]) * inv_dim;
        float sq = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * N; c < dim; c += T * N) {
            float f[N];
            again(c, f);
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (c + e < dim) sq = fmaf(f[e] - first, f[e] - first, sq);
        }
        float mean = first, var = team_sum<T>(sq, red[1]) * inv_dim, off = 0.f;
        if (far_from_zero(mean, var, a.eps)) {
            float sd = 0.f;
            for (int64_t c = (int64_t)threadIdx.x * N; c < dim; c += T * N) {
                float f[N];
                again(c, f);
#pragma unroll
                for (int e = 0; e < N; ++e) sd += c + e < dim ? f[e] - first : 0.f;
            }
            off = team_sum<T>(sd, red[2]) * inv_dim;
            correct(mean, var, off);
        }
        const float rstd = 1.f / sqrtf(var + a.eps);
        const float shift = -off * rstd;
        for (int64_t c = (int64_t)threadIdx.x * N; c < dim; c += T * N) {
            float f[N], gamma[N], beta[N];
            again(c, f);
            load_param<P>(gamma, a.gamma, c, dim, 1.f);
            load_param<P>(beta, a.beta, c, dim, 0.f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = fmaf(fmaf(f[e] - first, rstd, shift), gamma[e], beta[e]);
            store_part<X>(f, yr, c, dim);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Where a workgroup's weight-gradient sums go: straight to the result when its
// group has one part, else to its partial row.
__device__ __forceinline__ void store_param(void* out, int32_t dtype, int64_t i, float x) {
    if (dtype == kF32) static_cast<float*>(out)[i] = x;
    else if (dtype == kF16) store_one<kF16>(reinterpret_cast<uint64_t>(out) + (uint64_t)i * 2, x);
    else store_one<kB16>(reinterpret_cast<uint64_t>(out) + (uint64_t)i * 2, x);
}

// Workgroup blockIdx.x = group * parts + part takes rows part * R, (part +
// parts) * R, ... of its group, R at a time, a team of T threads each.  A row is
// kept as it was read and widened again for dx, after the two sums: half the
// registers of its binary32 values.
template <int X, int P, int T, int V>
__global__ __launch_bounds__(kBwdThreads) void k_ln_bwd(LnBwd a, int32_t dim, int64_t ldp, int32_t parts,
                                                        float* out, uint32_t* done) {
    constexpr int N = kVec<X>, R = kBwdThreads / T, WAVES = T <= 64 ? 1 : T / 64;
    // 128 registers hold the next row beside one of 8 elements per thread.  Of 16 per thread, a wavefront's row
    // keeps the weight (60000 x 768 bf16 rows: 72 us; 92 reading it again), the widest rows not even that.
    constexpr bool AHEAD = V * N <= 8, HOLD = AHEAD || T == 64;
    __shared__ float red[2][2][kBwdThreads / 64];
    const int t = threadIdx.x % T;
    // one number for a whole wavefront where none holds two teams, so that its row's addresses are scalar
    const int team = T >= 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / T) : threadIdx.x / T;
    const int32_t group = (int32_t)(blockIdx.x / (uint32_t)parts), part = (int32_t)(blockIdx.x % (uint32_t)parts);
    const int64_t row1 = (int64_t)(group + 1) * a.group_rows;
    const int64_t step = (int64_t)parts * R;
    int64_t first = (int64_t)group * a.group_rows + (int64_t)part * R;   // the first team's row

    struct Row {
        Raw<X, N> x[V], dy[V], ds[V];
        float mean, rstd;
    };
    auto load_row = [&](Row& r, int64_t row) {
        r.mean = a.mean[row];
        r.rstd = a.rstd[row];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * N;
            load_ahead<X, N, true>(r.x[v], reinterpret_cast<uint64_t>(a.x) + (uint64_t)(row * a.ldx), c, dim);
            load_ahead<X, N, true>(r.dy[v], reinterpret_cast<uint64_t>(a.dy) + (uint64_t)(row * a.ldy), c, dim);
            if (a.dsum)
                load_ahead<X, N, true>(r.ds[v], reinterpret_cast<uint64_t>(a.dsum) + (uint64_t)(row * a.lds), c, dim);
        }
    };
    Row next;
    if (AHEAD && first + team < row1) load_row(next, first + team);
    float held[V][N], dg[V][N], db[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (HOLD) load_param<P>(held[v], a.gamma, (v * T + t) * N, dim, 1.f);
#pragma unroll
        for (int e = 0; e < N; ++e) dg[v][e] = db[v][e] = 0.f;
    }
    const float inv_dim = (float)(1.0 / (double)dim);
    int parity = 0;
    for (; first < row1; first += step) {
        const int64_t row = first + team;
        const bool mine = row < row1;
        Row now;
        if constexpr (AHEAD) {
            now = next;
            if (row + step < row1) load_row(next, row + step);
        } else if (mine) {
            load_row(now, row);
        }
        float s1 = 0.f, s2 = 0.f;
        if (mine) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float x[N], dy[N], gamma[N];
                into_place(now.x[v], (v * T + t) * N, dim);
                into_place(now.dy[v], (v * T + t) * N, dim);
                if (a.dsum) into_place(now.ds[v], (v * T + t) * N, dim);
                now.x[v].widen(x);
                now.dy[v].widen(dy);
                if constexpr (!HOLD) load_param<P>(gamma, a.gamma, (v * T + t) * N, dim, 1.f);
                // columns past dim hold dy = 0 and add nothing anywhere
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float xh = (x[e] - now.mean) * now.rstd, h = dy[e] * (HOLD ? held[v][e] : gamma[e]);
                    dg[v][e] = fmaf(dy[e], xh, dg[v][e]);
                    db[v][e] += dy[e];
                    s1 += h;
                    s2 = fmaf(h, xh, s2);
                }
            }
        }
        s1 = lanes_sum_f32<T < 64 ? T : 64>(s1);
        s2 = lanes_sum_f32<T < 64 ? T : 64>(s2);
        if constexpr (T > 64) {
            if ((threadIdx.x & 63) == 0) {
                red[parity][0][threadIdx.x >> 6] = s1;
                red[parity][1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            s1 = red[parity][0][team * WAVES];
            s2 = red[parity][1][team * WAVES];
#pragma unroll
            for (int j = 1; j < WAVES; ++j) {
                s1 += red[parity][0][team * WAVES + j];
                s2 += red[parity][1][team * WAVES + j];
            }
            parity ^= 1;
        }
        if (!mine) continue;
        s1 *= inv_dim;
        s2 *= inv_dim;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float x[N], dy[N], ds[N], gamma[N];
            now.x[v].widen(x);
            now.dy[v].widen(dy);
            if constexpr (!HOLD) load_param<P>(gamma, a.gamma, (v * T + t) * N, dim, 1.f);
            if (a.dsum) {
                now.ds[v].widen(ds);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) ds[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float xh = (x[e] - now.mean) * now.rstd, h = dy[e] * (HOLD ? held[v][e] : gamma[e]);
                ds[e] = fmaf(now.rstd, h - fmaf(xh, s2, s1), ds[e]);
            }
            store_part<X>(ds, reinterpret_cast<uint64_t>(a.dx) + (uint64_t)(row * a.ldd), (v * T + t) * N, dim);
        }
    }
    if (!a.dgamma) return;
    float* pg = out + (int64_t)blockIdx.x * 2 * ldp;
    auto put = [&](int which, int c, float s) {
        if (parts == 1) store_param(which ? a.dbeta : a.dgamma, a.dp_dtype, (int64_t)group * dim + c, s);
        else pg[which * ldp + c] = s;
    };
    if constexpr (R > 1) {
        // the teams' sums, added in order
        __shared__ float cols[R][V * T * N];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) cols[team][(v * T + t) * N + e] = which ? db[v][e] : dg[v][e];
            __syncthreads();
            for (int c = threadIdx.x; c < dim; c += kBwdThreads) {
                float s = cols[0][c];
#pragma unroll 8
                for (int j = 1; j < R; ++j) s += cols[j][c];
                put(which, c, s);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = (v * T + t) * N + e;
                if (c >= dim) continue;
                put(0, c, dg[v][e]);
                put(1, c, db[v][e]);
            }
        }
    }
    if (!done) return;
    // few partial rows: the group's workgroup that ends last adds them, in their order.  Each wavefront waits for its
    // own stores: the barrier does not, and the release, thread 0's, writes back to memory what the cache holds then.
    __shared__ uint32_t last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(done + group, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
               (uint32_t)parts;
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    if (threadIdx.x == 0) __hip_atomic_store(done + group, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const float* p = out + (int64_t)group * parts * 2 * ldp;
    for (int c = threadIdx.x * 4; c < 2 * (int)ldp; c += kBwdThreads * 4) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        for (int32_t k0 = 0; k0 < parts; k0 += 8) {
            f32x4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = *reinterpret_cast<const f32x4*>(p + (int64_t)(k0 + k < parts ? k0 + k : parts - 1) * 2 * ldp + c);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k0 + k < parts) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] += x[k][e];
                }
            }
        }
        // ldp is a multiple of 4: the four columns are all of one gradient
        void* g = c < (int)ldp ? a.dgamma : a.dbeta;
        const int col = c < (int)ldp ? c : c - (int)ldp;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < dim) store_param(g, a.dp_dtype, (int64_t)group * dim + col + e, s[e]);
    }
}

// Rows that do not stay in registers: dx with two passes over the row ...
template <int X, int P>
__global__ __launch_bounds__(kLongThreads) void k_ln_dx_long(LnBwd a, int64_t dim) {
    constexpr int N = kVec<X>, T = kLongThreads;
    __shared__ float red[2][T / 64];
    const float inv_dim = (float)(1.0 / (double)dim);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = a.mean[row], rs = a.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        auto parts = [&](int64_t c, float (&xh)[N], float (&h)[N]) {
            Raw<X, N> r;
            float gamma[N];
            load_part(r, reinterpret_cast<uint64_t>(a.x) + (uint64_t)(row * a.ldx), c, dim);
            r.widen(xh);
            load_part(r, reinterpret_cast<uint64_t>(a.dy) + (uint64_t)(row * a.ldy), c, dim);
            r.widen(h);
            load_param<P>(gamma, a.gamma, c, dim, 1.f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                xh[e] = (xh[e] - mean) * rs;
                h[e] *= gamma[e];
            }
        };
        for (int64_t c = (int64_t)threadIdx.x * N; c < dim; c += T * N) {
            float xh[N], h[N];
            parts(c, xh, h);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                s1 += h[e];
                s2 = fmaf(h[e], xh[e], s2);
            }
        }
        __syncthreads();   // the previous row's sums are read
        s1 = team_sum<T>(s1, red[0]) * inv_dim;
        s2 = team_sum<T>(s2, red[1]) * inv_dim;
        for (int64_t c = (int64_t)threadIdx.x * N; c < dim; c += T * N) {
            float xh[N], h[N], ds[N];
            parts(c, xh, h);
#pragma unroll
            for (int e = 0; e < N; ++e) ds[e] = 0.f;
            if (a.dsum) {
                Raw<X, N> r;
                load_part(r, reinterpret_cast<uint64_t>(a.dsum) + (uint64_t)(row * a.lds), c, dim);
                r.widen(ds);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) h[e] = fmaf(rs, h[e] - fmaf(xh[e], s2, s1), ds[e]);
            store_part<X>(h, reinterpret_cast<uint64_t>(a.dx) + (uint64_t)(row * a.ldd), c, dim);
        }
    }
}

// ... and the weight gradients with a thread per column, over the rows of part
// blockIdx.y of its group.
template <int X>
__global__ __launch_bounds__(256) void k_ln_params_long(LnBwd a, int64_t dim, int64_t ldp, int32_t parts,
                                                        float* __restrict__ out) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= dim) return;
    const int32_t group = (int32_t)(blockIdx.y / (uint32_t)parts), part = (int32_t)(blockIdx.y % (uint32_t)parts);
    const int64_t row1 = (int64_t)(group + 1) * a.group_rows;
    float dg = 0.f, db = 0.f;
    for (int64_t row = (int64_t)group * a.group_rows + part; row < row1; row += parts) {
        const float x = load_one<X>(reinterpret_cast<uint64_t>(a.x) + (uint64_t)(row * a.ldx + c * kSize<X>));
        const float dy = load_one<X>(reinterpret_cast<uint64_t>(a.dy) + (uint64_t)(row * a.ldy + c * kSize<X>));
        dg = fmaf(dy, (x - a.mean[row]) * a.rstd[row], dg);
        db += dy;
    }
    if (parts == 1) {
        store_param(a.dgamma, a.dp_dtype, (int64_t)group * dim + c, dg);
        store_param(a.dbeta, a.dp_dtype, (int64_t)group * dim + c, db);
    } else {
        out[(int64_t)blockIdx.y * 2 * ldp + c] = dg;
        out[((int64_t)blockIdx.y * 2 + 1) * ldp + c] = db;
    }
}

// Adds the `parts` partial rows of group blockIdx.y in a fixed order: 16
// threads take every 16th part of 64 columns, then the 16 sums are added.
// parts = 0 writes zeros.
__global__ __launch_bounds__(256) void k_ln_params_end(const float* __restrict__ in, int64_t dim, int64_t ldp,
                                                       int32_t parts, void* dgamma, void* dbeta, int32_t dp_dtype) {
    __shared__ f32x4 sums[16][16];
    const int quad = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int64_t c4 = ((int64_t)blockIdx.x * 16 + quad) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (c4 < 2 * ldp) {
        const float* p = in + (int64_t)blockIdx.y * parts * 2 * ldp + c4;
#pragma unroll 4
        for (int32_t k = slice; k < parts; k += 16) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(p + (int64_t)k * 2 * ldp);
            s.x += x.x;
            s.y += x.y;
            s.z += x.z;
            s.w += x.w;
        }
    }
    sums[slice][quad] = s;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= 2 * ldp) return;
    const float* f = reinterpret_cast<const float*>(sums);
    float t = f[threadIdx.x];
    for (int k = 1; k < 16; ++k) t += f[k * 64 + threadIdx.x];
    const int64_t col = c < ldp ? c : c - ldp;
    if (col >= dim) return;
    store_param(c < ldp ? dgamma : dbeta, dp_dtype, (int64_t)blockIdx.y * dim + col, t);
}

// Calls f<T, V> with the team that holds a row of dim elements.  Forward: 16
// elements per thread of a workgroup of 256 where that is enough (16384 x 4096
// bf16 rows with a residual, on one card: 94 us; 98 with 8 per thread of 512), and no more
// threads than a narrow row needs (60000 x 64 rows: 10 us with 16 threads, 27
// with 64).
#define GA_TEAM(T, V) \
    if (dim <= T * V * kVec<X>) return f(std::integral_constant<int, T>{}, std::integral_constant<int, V>{})
template <int X, typename F>
hipError_t with_fwd_team(int64_t dim, F f) {
    GA_TEAM(16, 1);
    GA_TEAM(32, 1);
    GA_TEAM(64, 1);
    GA_TEAM(64, 2);
    if constexpr (X == kF32) {
        GA_TEAM(64, 4);
        GA_TEAM(256, 2);
        GA_TEAM(256, 4);
        GA_TEAM(512, 4);
        GA_TEAM(1024, 4);
    } else {
        GA_TEAM(256, 1);
        GA_TEAM(256, 2);
        GA_TEAM(512, 2);
        GA_TEAM(1024, 2);
    }
    return hipErrorInvalidValue;
}

// Backward: 8 elements (4 binary32) per thread up to the workgroup's width, but
// one wavefront for a 16-bit row of up to 1024 elements, which then needs no
// barrier: 60000 x 768 bf16 rows 72 us against 100 with 128 threads each,
// 16384 x 1024 rows 24.5 against 23.2.
template <int X, typename F>
hipError_t with_bwd_team(int64_t dim, F f) {
    GA_TEAM(16, 1);
    GA_TEAM(32, 1);
    GA_TEAM(64, 1);
    if constexpr (X == kF32) {
        GA_TEAM(128, 1);
        GA_TEAM(256, 1);
    } else {
        GA_TEAM(64, 2);
        GA_TEAM(256, 1);
    }
    GA_TEAM(512, 1);
    GA_TEAM(1024, 1);
    GA_TEAM(1024, 2);
    if constexpr (X == kF32) GA_TEAM(1024, 4);
    return hipErrorInvalidValue;
}
#undef GA_TEAM

constexpr int64_t kFwdBlocks = 2048;   // workgroups of 256 threads that fill the chip

template <int X, int P>
hipError_t ln_fwd(const LayerNorm& n, const LnFwd& a, hipStream_t s) {
    if (n.dim > kInRegisters) {
        const unsigned blocks = (unsigned)(a.rows < 1024 ? a.rows : 1024);
        hipLaunchKernelGGL((k_ln_fwd_long<X, P>), dim3(blocks), dim3(kLongThreads), 0, s, a, n.dim);
        return hipGetLastError();
    }
    return with_fwd_team<X>(n.dim, [&](auto t, auto v) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value;
        const int64_t want = (a.rows + kTeamRows<T> - 1) / kTeamRows<T>;
        const int64_t most = kFwdBlocks * 256 / kTeamThreads<T>;
        hipLaunchKernelGGL((k_ln_fwd<X, P, T, V>), dim3((unsigned)(want < most ? want : most)),
                           dim3(kTeamThreads<T>), 0, s, a, (int32_t)n.dim);
        return hipGetLastError();
    });
}

// Parts of each group: a workgroup for each CU, at most one per row-set and
// kLnParts in all.
inline int32_t parts_of(const LnBwd& a, int rows_at_once) {
    int64_t p = (a.group_rows + rows_at_once - 1) / rows_at_once;
    if (p > kLnParts / a.groups) p = kLnParts / a.groups;
    return p < 1 ? 1 : (int32_t)p;
}

// Up to this many elements in a group's partial rows of one gradient, its
// workgroup that ends last adds them itself; above, a second kernel does, which
// costs a launch but spreads the sums over the chip.  Calls one after the other:
// 8.4 against 10.4 us at 8192 (128 x 512 binary32 rows), 10.8 both ways at 12288
// (256 x 768 bf16), 13.0 against 10.8 at 32768 (512 x 512).
constexpr int64_t kOneLaunch = 12288;

template <int X, int P>
hipError_t ln_bwd(const LayerNorm& n, const LnBwd& a, hipStream_t s) {
    int32_t parts = 0;
    bool one = false;
    hipError_t e = hipSuccess;
    if (a.rows > 0 && n.dim > kInRegisters) {
        if (a.dgamma) {
            parts = parts_of(a, 64);
            hipLaunchKernelGGL((k_ln_params_long<X>), dim3((unsigned)((n.dim + 255) / 256), (unsigned)(a.groups * parts)),
                               dim3(256), 0, s, a, n.dim, n.ldp, parts, n.d_parts);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        const unsigned blocks = (unsigned)(a.rows < 1024 ? a.rows : 1024);
        hipLaunchKernelGGL((k_ln_dx_long<X, P>), dim3(blocks), dim3(kLongThreads), 0, s, a, n.dim);
        e = hipGetLastError();
    } else if (a.rows > 0) {
        e = with_bwd_team<X>(n.dim, [&](auto t, auto v) {
            constexpr int T = decltype(t)::value, V = decltype(v)::value;
            parts = parts_of(a, kBwdThreads / T);
            one = parts > 1 && parts * n.dim <= kOneLaunch;
            hipLaunchKernelGGL((k_ln_bwd<X, P, T, V>), dim3((unsigned)(a.groups * parts)), dim3(kBwdThreads), 0, s,
                               a, (int32_t)n.dim, n.ldp, parts, n.d_parts, one ? n.d_done : nullptr);
            return hipGetLastError();
        });
    }
    if (e != hipSuccess || !a.dgamma || parts == 1 || one) return e;
    hipLaunchKernelGGL(k_ln_params_end, dim3((unsigned)((2 * n.ldp + 63) / 64), (unsigned)a.groups), dim3(256), 0, s,
                       n.d_parts, n.dim, n.ldp, parts, a.dgamma, a.dbeta, a.dp_dtype);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ln_fwd(const LayerNorm& n, const LnFwd& a, hipStream_t s) {
    if (n.x_dtype == GA_FP32) return ln_fwd<kF32, kF32>(n, a, s);
    if (n.x_dtype == GA_FP16)
        return n.p_dtype == GA_FP32 ? ln_fwd<kF16, kF32>(n, a, s) : ln_fwd<kF16, kF16>(n, a, s);
    return n.p_dtype == GA_FP32 ? ln_fwd<kB16, kF32>(n, a, s) : ln_fwd<kB16, kB16>(n, a, s);
}

hipError_t launch_ln_bwd(const LayerNorm& n, const LnBwd& a, hipStream_t s) {
    if (n.x_dtype == GA_FP32) return ln_bwd<kF32, kF32>(n, a, s);
    if (n.x_dtype == GA_FP16)
        return n.p_dtype == GA_FP32 ? ln_bwd<kF16, kF32>(n, a, s) : ln_bwd<kF16, kF16>(n, a, s);
    return n.p_dtype == GA_FP32 ? ln_bwd<kB16, kF32>(n, a, s) : ln_bwd<kB16, kB16>(n, a, s);
}

}  // namespace ga
