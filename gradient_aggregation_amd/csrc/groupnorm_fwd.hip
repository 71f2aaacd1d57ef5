// Group norm forward, with its activation (ga_groupnorm_forward).
//
// The statistics of a group take one pass: each thread sums the deviations from a
// value of its own (shift: it reads that value first, so that an outlier there is
// among its squares too) and their squares as its vectors arrive.  The sums of all
// threads give the mean m; with d = m - shift a thread's squares about m are
// s2 - 2 d s1 + count d^2, and its deviations from m, s1 - count d, add up to what
// m's roundings left, which corrects it.
#include "groupnorm.h"

namespace ga {

namespace {

template <bool WHOLE, int N>
struct Moments {
    static constexpr int M = WHOLE ? 1 : N;    // a sum of the vector, or one for each channel
    float shift[M], s1[M], s2[M];
    int rows;

    __device__ __forceinline__ Moments() : rows(0) {
#pragma unroll
        for (int e = 0; e < M; ++e) shift[e] = s1[e] = s2[e] = 0.f;
    }

    __device__ __forceinline__ void add(float (&f)[N], const Place<WHOLE, N>& p) {
        const bool full = p.left >= N;
        if (rows++ == 0) {
            if constexpr (!WHOLE) {
#pragma unroll
                for (int e = 0; e < N; ++e) shift[e] = f[e];
            } else {
                float t = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) t += full || e < p.left ? f[e] : 0.f;
                shift[0] = t * (full ? 1.f / N : 1.f / (float)p.left);
            }
        }
        if (WHOLE && !full) {
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = e < p.left ? f[e] : shift[0];
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int k = WHOLE ? 0 : e;
            const float d = f[e] - shift[k];
            s1[k] += d;
            s2[k] = fmaf(d, d, s2[k]);
        }
    }
};

// What a thread's groups have over all of a workgroup's values: m, the mean as first rounded; off, the mean of the
// deviations from it; sq, the sum of their squares (not yet less count * off^2).  base: a value of the group, or one
// that its threads share; constant groups add up exactly about it.
template <bool WHOLE, int N, int T>
__device__ __forceinline__ void statistics(const Moments<WHOLE, N>& t, float base, float inv, float (&m)[WHOLE ? 1 : N],
                                           float (&off)[WHOLE ? 1 : N], float (&sq)[WHOLE ? 1 : N], float* tile, float* res,
                                           const GnShape& h, const Place<WHOLE, N>& p) {
    constexpr int M = WHOLE ? 1 : N;
    const int all = h.Q * h.sg;
    const float count = (float)t.rows * (float)(!WHOLE ? 1 : p.left >= N ? N : p.left > 0 ? p.left : 0);
    int at[M];
    float first[1][M], d1[1][M], d2[1][M];
#pragma unroll
    for (int e = 0; e < M; ++e) {
        at[e] = p.here ? p.q * h.sg + p.group(h, e) : 0;
        first[0][e] = t.rows ? fmaf(count, t.shift[e] - base, t.s1[e]) : 0.f;
    }
    sum_groups<WHOLE, N, T, 1>(first, tile, res, h, p);
#pragma unroll
    for (int e = 0; e < M; ++e) {
        m[e] = fmaf(res[at[e]], inv, base);
        const float d = m[e] - t.shift[e];
        d1[0][e] = t.rows ? fmaf(-count, d, t.s1[e]) : 0.f;
        d2[0][e] = t.rows ? fmaf(-d, t.s1[e] + d1[0][e], t.s2[e]) : 0.f;
    }
    if constexpr (WHOLE) {
        const float both[2][1] = {{d1[0][0]}, {d2[0][0]}};
        sum_groups<WHOLE, N, T, 2>(both, tile, res + all, h, p);
    } else {
        sum_groups<WHOLE, N, T, 1>(d1, tile, res + all, h, p);
        sum_groups<WHOLE, N, T, 1>(d2, tile, res + 2 * all, h, p);
    }
#pragma unroll
    for (int e = 0; e < M; ++e) {
        off[e] = res[all + at[e]] * inv;
        sq[e] = res[2 * all + at[e]];
    }
}

// The first value of the group (WHOLE) or of the slab; it may be another group's, and then not finite.
template <int X, bool WHOLE, int N>
__device__ __forceinline__ float base_value(uint64_t image, const GnShape& h, const Place<WHOLE, N>& p) {
    const float b = load_one<X>(image + (uint64_t)((p.g0 + (WHOLE ? p.group(h, 0) : 0)) * h.cg) * kSize<X>);
    return fabsf(b) < INFINITY ? b : 0.f;
}

// y of one vector: (x - m) * scale + bias, activated.
template <int X, bool WHOLE, int N>
__device__ __forceinline__ void put_vector(const Raw<X, N>& x, const float (&m)[WHOLE ? 1 : N], const float (&scale)[N],
                                           const float (&bias)[N], uint64_t row, const Place<WHOLE, N>& p, int32_t act) {
    float f[N];
    x.widen(f);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = fmaf(f[e] - m[WHOLE ? 0 : e], scale[e], bias[e]);
    activate(f, act);
    store_part<X, true>(f, row, p.c, p.c + (p.left < N ? p.left : N));
}

// A sample's slab that stays in registers, V vectors to a thread.
template <int X, bool WHOLE, int T, int V>
__global__ __launch_bounds__(T) void k_gn_fwd(GnArgs a, GnShape h) {
    constexpr int N = kVec<X>, M = WHOLE ? 1 : N;
    extern __shared__ float lds[];
    const uint32_t id = xcd_block();
    const Place<WHOLE, N> p(h, (int)(id % (uint32_t)h.slabs));
    const int64_t n = (int64_t)(id / (uint32_t)h.slabs) * h.Q + p.q;
    const bool in = p.here && n < a.N && p.left > 0;
    const int rows = in ? (h.S - p.r + h.R - 1) / h.R : 0;
    const uint64_t xr = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(n * a.x.sample);
    Raw<X, N> x[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < rows) load_ahead<X, N, false>(x[i], xr + (uint64_t)((p.r + i * h.R) * a.x.ld), p.c, h.C);
    const float base = in ? base_value<X>(xr, h, p) : 0.f;
    float scale[N], bias[N];
    load_weight<X>(scale, a.gamma, h, p.c, 1.f);
    load_weight<X>(bias, a.beta, h, p.c, 0.f);
    Moments<WHOLE, N> t;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i >= rows) continue;
        float f[N];
        if (p.past) drop_front(x[i], p.past);
        x[i].widen(f);
        t.add(f, p);
    }
    float m[M], off[M], sq[M];
    statistics<WHOLE, N, T>(t, base, h.inv_n, m, off, sq, lds, lds + h.res_at, h, p);
    if (!in) return;
#pragma unroll
    for (int e = 0; e < M; ++e) {
        const float var = fmaf(-off[e], off[e], sq[e] * h.inv_n);
        const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);
        const int g = p.group(h, e);
        if (p.r == 0 && e < p.left && p.v * N + e == g * h.cg) {
            if (a.mean) a.mean[n * h.G + p.g0 + g] = m[e] + off[e];
            if (a.rstd) a.rstd[n * h.G + p.g0 + g] = rstd;
        }
        sq[e] = rstd;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        scale[e] *= sq[WHOLE ? 0 : e];
        bias[e] = fmaf(-off[WHOLE ? 0 : e], scale[e], bias[e]);
    }
    const uint64_t yr = reinterpret_cast<uint64_t>(a.y.data) + (uint64_t)(n * a.y.sample);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < rows) put_vector<X>(x[i], m, scale, bias, yr + (uint64_t)((p.r + i * h.R) * a.y.ld), p, h.act);
}

// ---- images that do not stay in registers ------------------------------------
// Two kernels with the same workgroups on the same parts of the images: the statistics of each part, then y.

// Of a part (and piece) of a group: the mean m + off and the sum of squares about it.
typedef f32x4 GnRecord;

template <int X, bool WHOLE, int T>
__global__ __launch_bounds__(T) void k_gn_stats(GnArgs a, GnShape h, GnRecord* __restrict__ records) {
    constexpr int N = kVec<X>, M = WHOLE ? 1 : N;
    extern __shared__ float lds[];
    const PartOf o(h, xcd_block());
    const Place<WHOLE, N> p(h, o.slab);
    const uint64_t xr = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(o.n * a.x.sample);
    const bool in = p.here && p.left > 0;
    const float base = in ? base_value<X>(xr, h, p) : 0.f;
    Moments<WHOLE, N> t;
    if (in) {
        const int64_t step = h.R * a.x.ld;
        uint64_t row = xr + (uint64_t)((int64_t)(o.s0 + p.r) * a.x.ld);
        for (int64_t s = (int64_t)o.s0 + p.r; s < o.s1; s += kAhead * h.R, row += kAhead * step) {
            Raw<X, N> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (s + (int64_t)i * h.R < o.s1) load_ahead<X, N, false>(x[i], row + i * step, p.c, h.C);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (s + (int64_t)i * h.R >= o.s1) continue;
                float f[N];
                if (p.past) drop_front(x[i], p.past);
                x[i].widen(f);
                t.add(f, p);
            }
        }
    }
    // of the groups' values in this part and slab
    const float count = (float)(o.s1 - o.s0) * (float)(h.pieces == 1 ? h.cg : p.channels), inv = 1.f / count;
    float m[M], off[M], sq[M];
    statistics<WHOLE, N, T>(t, base, inv, m, off, sq, lds, lds + h.res_at, h, p);
    if (!in || p.r != 0) return;
    const int K = h.parts * h.pieces, k = o.part * h.pieces + (h.pieces == 1 ? 0 : o.slab % h.pieces);
#pragma unroll
    for (int e = 0; e < M; ++e) {
        const int g = p.group(h, e);
        if (e < p.left && p.v * N + e == g * h.cg) {
            const float about = fmaf(-off[e] * count, off[e], sq[e]);
            records[(o.n * K + k) * h.G + p.g0 + g] = GnRecord{m[e], off[e], about < 0.f ? 0.f : about, 0.f};
        }
    }
}

template <int X, bool WHOLE, int T>
__global__ __launch_bounds__(T) void k_gn_apply(GnArgs a, GnShape h, const GnRecord* __restrict__ records) {
    constexpr int N = kVec<X>, M = WHOLE ? 1 : N;
    extern __shared__ float lds[];        // m, what its rounding left, 1/deviation of the slab's groups
    const PartOf o(h, xcd_block());
    const Place<WHOLE, N> p(h, o.slab);
    const uint64_t xr = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(o.n * a.x.sample);
    const uint64_t yr = reinterpret_cast<uint64_t>(a.y.data) + (uint64_t)(o.n * a.y.sample);
    const bool in = p.here && p.left > 0;
    const int64_t step = h.R * a.x.ld;
    uint64_t row = xr + (uint64_t)((int64_t)(o.s0 + p.r) * a.x.ld);
    int64_t s = (int64_t)o.s0 + p.r;
    Raw<X, N> x[kAhead];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (in && s + (int64_t)i * h.R < o.s1) load_ahead<X, N, false>(x[i], row + i * step, p.c, h.C);
    };
    load();
    float scale[N], bias[N];
    load_weight<X>(scale, a.gamma, h, p.c, 1.f);
    load_weight<X>(bias, a.beta, h, p.c, 0.f);
    const int K = h.parts * h.pieces, j = threadIdx.x & (h.lanes - 1);
    for (int g = threadIdx.x / h.lanes; g < h.sg; g += T / h.lanes) {
        const int group = p.g0 + g < h.G ? p.g0 + g : h.G - 1;
        const GnRecord* of = records + o.n * K * h.G + group;
        auto count = [&](int k) {
            const int part = k / h.pieces, first = (k - part * h.pieces) * h.nv * N;
            const int rows = h.S - part * h.span < h.span ? h.S - part * h.span : h.span;
            return (double)rows * (h.pieces == 1 ? h.cg : h.nv * N < h.cg - first ? h.nv * N : h.cg - first);
        };
        const double inv = 1.0 / ((double)h.S * h.cg);
        double sum = 0.0, sq = 0.0;
        for (int k = j; k < K; k += h.lanes) {
            const GnRecord r = of[(int64_t)k * h.G];
            sum += count(k) * ((double)r.x + (double)r.y);
        }
        for (int b = h.lanes >> 1; b; b >>= 1) sum += __shfl_xor(sum, b, 64);
        const double mean = sum * inv;
        for (int k = j; k < K; k += h.lanes) {
            const GnRecord r = of[(int64_t)k * h.G];
            const double d = (double)r.x + (double)r.y - mean;
            sq += (double)r.z + count(k) * d * d;
        }
        for (int b = h.lanes >> 1; b; b >>= 1) sq += __shfl_xor(sq, b, 64);
        if (j == 0) {
            const float m = (float)mean, rstd = 1.f / sqrtf((float)(sq * inv) + a.eps);
            lds[3 * g] = m;
            lds[3 * g + 1] = (float)(mean - (double)m);
            lds[3 * g + 2] = rstd;
            if (o.part == 0 && p.g0 + g < h.G && (h.pieces == 1 || o.slab % h.pieces == 0)) {
                if (a.mean) a.mean[o.n * h.G + group] = m;
                if (a.rstd) a.rstd[o.n * h.G + group] = rstd;
            }
        }
    }
    __syncthreads();
    if (!in) return;
    float m[M];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int g = p.group(h, e);
        if (e < M) m[e] = lds[3 * g];
        scale[e] *= lds[3 * g + 2];
        bias[e] = fmaf(-lds[3 * g + 1], scale[e], bias[e]);
    }
    for (; s < o.s1; ) {
        const int64_t now = s;
        Raw<X, N> y[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) y[i] = x[i];
        s += kAhead * h.R;
        row += kAhead * step;
        load();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (now + (int64_t)i * h.R >= o.s1) continue;
            if (p.past) drop_front(y[i], p.past);
            put_vector<X>(y[i], m, scale, bias, yr + (uint64_t)((now + (int64_t)i * h.R) * a.y.ld), p, h.act);
        }
    }
}

// ---- on the host -------------------------------------------------------------

constexpr TeamSize kTeams[] = {{256, 1}, {256, 2}, {256, 4}, {512, 4}, {512, 8}, {1024, 8}, {1024, 16}};

// Calls f with the team's sizes as constants.
template <typename F>
hipError_t with_team(int k, F f) {
#define GA_TEAM(K)     if (k == K) return f(std::integral_constant<int, kTeams[K].T>{}, std::integral_constant<int, kTeams[K].V>{})
    GA_TEAM(0);
    GA_TEAM(1);
    GA_TEAM(2);
    GA_TEAM(3);
    GA_TEAM(4);
    GA_TEAM(5);
    GA_TEAM(6);
#undef GA_TEAM
    return hipErrorInvalidValue;
}

constexpr int kWideThreads = 512;

// The arguments of samples [n0, n0 + count).
GnArgs samples_of(const GnArgs& all, int32_t G, int64_t n0, int64_t count) {
    GnArgs a = all;
    a.N = count;
    a.x.data += n0 * a.x.sample;
    a.y.data += n0 * a.y.sample;
    if (a.mean) a.mean += n0 * G;
    if (a.rstd) a.rstd += n0 * G;
    return a;
}

template <int X>
hipError_t gn_fwd(const GroupNorm& n, const GnArgs& all, hipStream_t s) {
    constexpr int N = kVec<X>;
    GnShape h = shape_of(n, all.S);
    const int k = choose(h, N, kTeams, all.N);
    if (k >= 0) {
        const bool whole = whole_vectors(h, N);
        h.res_at = (int32_t)lds_of_groups(h, N, kTeams[k].T, whole ? 2 : 1);
        const size_t bytes = sizeof(float) * ((size_t)h.res_at + 3 * (size_t)h.Q * h.sg);
        const int64_t step = kMostBlocks / h.slabs * h.Q;
        for (int64_t n0 = 0; n0 < all.N; n0 += step) {
            const GnArgs a = samples_of(all, n.G, n0, all.N - n0 < step ? all.N - n0 : step);
            const unsigned blocks = (unsigned)(ceil_div(a.N, h.Q) * h.slabs);
            const hipError_t e = with_team(k, [&](auto t, auto v) {
                constexpr int T = decltype(t)::value, V = decltype(v)::value;
                if (whole) hipLaunchKernelGGL((k_gn_fwd<X, true, T, V>), dim3(blocks), dim3(T), bytes, s, a, h);
                else hipLaunchKernelGGL((k_gn_fwd<X, false, T, V>), dim3(blocks), dim3(T), bytes, s, a, h);
                return hipGetLastError();
            });
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    constexpr int T = kWideThreads;
    lay_wide(h, N, T, all.N, 1024);
    const bool whole = whole_vectors(h, N);
    h.res_at = (int32_t)lds_of_groups(h, N, T, whole ? 2 : 1);
    const size_t bytes = sizeof(float) * ((size_t)h.res_at + 3 * (size_t)h.sg);
    // as many samples at once as the records have room for
    const int64_t per = (int64_t)h.parts * h.pieces * n.G;
    int64_t step = kGnRecords / per;
    if (step > kMostBlocks / ((int64_t)h.parts * h.slabs)) step = kMostBlocks / ((int64_t)h.parts * h.slabs);
    if (step < 1) return hipErrorInvalidValue;
    for (int64_t n0 = 0; n0 < all.N; n0 += step) {
        const GnArgs a = samples_of(all, n.G, n0, all.N - n0 < step ? all.N - n0 : step);
        const unsigned blocks = (unsigned)(a.N * h.parts * h.slabs);
        GnRecord* records = reinterpret_cast<GnRecord*>(n.d_records);
        if (whole) {
            hipLaunchKernelGGL((k_gn_stats<X, true, T>), dim3(blocks), dim3(T), bytes, s, a, h, records);
            hipLaunchKernelGGL((k_gn_apply<X, true, T>), dim3(blocks), dim3(T), bytes, s, a, h, records);
        } else {
            hipLaunchKernelGGL((k_gn_stats<X, false, T>), dim3(blocks), dim3(T), bytes, s, a, h, records);
            hipLaunchKernelGGL((k_gn_apply<X, false, T>), dim3(blocks), dim3(T), bytes, s, a, h, records);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_gn_fwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    if (n.x_dtype == GA_FP32) return gn_fwd<kF32>(n, a, s);
    return n.x_dtype == GA_FP16 ? gn_fwd<kF16>(n, a, s) : gn_fwd<kB16>(n, a, s);
}

}  // namespace ga
