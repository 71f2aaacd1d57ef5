// Group norm forward, with its activation (ga_groupnorm_forward).
//
// The statistics of a group take one pass: each thread sums the deviations from a
// value of its own (shift, the mean of its first vector: an outlier there is among
// its squares too) and their squares as its vectors arrive.  The sums of all
// threads give the mean m; with d = m - shift a thread's squares about m are
// s2 - 2 d s1 + count d^2, and its deviations from m, s1 - count d, add up to what
// m's roundings left, which corrects it.  A thread of many rows moves its sums to
// their own mean after 8, 16, 32, ... of them: a shift that is an outlier, A from
// the rest, would add A^2 with every row, and so take the others' bits.
//
// What bounds it, on bf16 with silu: small images (1 x 64 x 1280: 6.2 us of one kernel) the chain load, exchange, store; large
// ones (4 x 65536 x 256) two readings and one writing, 25 us at 5.4 TB/s for the statistics and 42 us at 6.4 TB/s for y,
// whose vector instructions take 70% of that time.
#include "groupnorm.h"

namespace ga {

namespace {

template <int MODE, int N>
struct Moments {
    static constexpr int M = MODE == kWhole ? 1 : N;    // a sum of the vector, or one for each channel
    float shift[M], s1[M], s2[M];
    float past[M];         // squares of the rows before the last move, about shift
    int rows;

    __device__ __forceinline__ Moments() : rows(0) {
#pragma unroll
        for (int e = 0; e < M; ++e) shift[e] = s1[e] = s2[e] = past[e] = 0.f;
    }

    template <bool RAGGED>
    __device__ __forceinline__ void start(const float (&f)[N], const Place<MODE, N>& p) {
        if constexpr (MODE == kWhole) {
            const bool full = !RAGGED || p.left >= N;
            float t = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) t += full || e < p.left ? f[e] : 0.f;
            shift[0] = t * (full ? 1.f / N : 1.f / (float)p.left);
        } else if constexpr (MODE == kSpan) {
            // of the vector's two groups each its own
            const int left = RAGGED && p.left < N ? p.left : N, border = p.border < left ? p.border : left;
            float first = 0.f, second = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                first += e < border ? f[e] : 0.f;
                second += e >= border && e < left ? f[e] : 0.f;
            }
            first *= 1.f / (float)border;
            second *= left > border ? 1.f / (float)(left - border) : 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) shift[e] = e < border ? first : second;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) shift[e] = f[e];
        }
    }

    template <bool RAGGED>
    __device__ __forceinline__ void add(float (&f)[N], const Place<MODE, N>& p) {
        ++rows;
        if (MODE == kWhole && RAGGED && p.left < N) {
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = e < p.left ? f[e] : shift[0];
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int k = MODE == kWhole ? 0 : e;
            const float d = f[e] - shift[k];
            s1[k] += d;
            s2[k] = fmaf(d, d, s2[k]);
        }
    }

    // Moves sum k of `count` values by about `by`, in roundings of the deviations' size only.
    __device__ __forceinline__ void move(int k, float by, float count) {
        const float to = shift[k] + by, d = to - shift[k], left = fmaf(-count, d, s1[k]);
        past[k] += fmaf(-d, s1[k] + left, s2[k]);             // s2 - 2 d s1 + count d^2
        shift[k] = to;
        s1[k] = left;
        s2[k] = 0.f;
    }

    // The sums to the mean of what they hold (a reciprocal's ulp off, which the sums then have).
    template <bool RAGGED>
    __device__ __forceinline__ void recentre(const Place<MODE, N>& p) {
        const int left = RAGGED && p.left < N ? p.left : N;
        if constexpr (MODE == kWhole) {
            const float count = (float)(rows * left);
            move(0, s1[0] * __builtin_amdgcn_rcpf(count), count);
        } else {
            const float count = (float)rows, inv = __builtin_amdgcn_rcpf(count);
            const int border = MODE == kSpan ? p.border < left ? p.border : left : 0;
            float first = 0.f, second = 0.f;
            if constexpr (MODE == kSpan) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    first += e < border ? s1[e] : 0.f;
                    second += e >= border && e < left ? s1[e] : 0.f;
                }
                first *= inv * __builtin_amdgcn_rcpf((float)border);
                second *= left > border ? inv * __builtin_amdgcn_rcpf((float)(left - border)) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < N; ++e) move(e, MODE == kMany ? s1[e] * inv : e < border ? first : second, count);
        }
    }

    __device__ __forceinline__ void end() {
#pragma unroll
        for (int e = 0; e < M; ++e) s2[e] += past[e];
    }
};

// What a thread's groups have over all of a workgroup's values: m, the mean as first rounded; off, the mean of the
// deviations from it; sq, the sum of their squares (not yet less count * off^2).  Constant groups add up exactly.
template <int MODE, int N, int T>
__device__ __forceinline__ void statistics(const Moments<MODE, N>& t, const float (&base)[Moments<MODE, N>::M], float inv,
                                           float (&m)[Moments<MODE, N>::M], float (&off)[Moments<MODE, N>::M],
                                           float (&sq)[Moments<MODE, N>::M], float* lds, const GnShape& h, const Place<MODE, N>& p) {
    constexpr int M = Moments<MODE, N>::M, SEGMENTS = MODE == kSpan ? 2 : 1;
    const int all = h.Q * h.sg;
    if constexpr (MODE != kMany) {
        // s1, s2, shift and count of each thread and group; a group's teams of threads read them twice
        f32x4* tile = reinterpret_cast<f32x4*>(lds);
        float* res = lds + SEGMENTS * 4 * T;
        if constexpr (MODE == kWhole) {
            const int mine = p.left >= N ? N : p.left > 0 ? p.left : 0;
            tile[threadIdx.x] = f32x4{t.s1[0], t.s2[0], t.shift[0], (float)t.rows * (float)mine};
        } else {
            f32x4 first = {0.f, 0.f, t.shift[0], 0.f}, second = {0.f, 0.f, t.shift[N - 1], 0.f};
            const int left = p.left < N ? p.left : N, border = p.border < left ? p.border : left;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                first.x += e < border ? t.s1[e] : 0.f;
                first.y += e < border ? t.s2[e] : 0.f;
                second.x += e >= border && e < left ? t.s1[e] : 0.f;
                second.y += e >= border && e < left ? t.s2[e] : 0.f;
            }
            first.w = (float)t.rows * (float)(border > 0 ? border : 0);
            second.w = (float)t.rows * (float)(left > border ? left - border : 0);
            tile[threadIdx.x] = first;
            tile[T + threadIdx.x] = second;
        }
        __syncthreads();
        const int j = threadIdx.x & (h.lanes - 1), jv = j & (h.spread - 1), jr = j / h.spread, rows = h.lanes / h.spread;
        for (int vg = threadIdx.x / h.lanes; vg < all; vg += T / h.lanes) {
            const int q = h.Q == 1 ? 0 : vg / h.sg, g = vg - q * h.sg, c0 = g * h.cg;
            const int v0 = h.sg == 1 ? 0 : c0 / N, v1 = h.sg == 1 ? h.nv - 1 : (c0 + h.cg - 1) / N;
            // vectors that start before the group have it as their second
            const f32x4* of = tile + q * h.R * h.nv;
            auto entry = [&](int r, int v) { return of[(MODE == kSpan && v * N < c0 ? T : 0) + r * h.nv + v]; };
            const float about = entry(0, v0).z;
            float s[1] = {0.f}, u[2] = {0.f, 0.f};
            for (int r = jr; r < h.R; r += rows) {
                for (int v = v0 + jv; v <= v1; v += h.spread) {
                    const f32x4 a = entry(r, v);
                    s[0] += fmaf(a.w, a.z - about, a.x);
                }
            }
            sum_lanes(s, h.lanes);
            const float mean = fmaf(s[0], inv, about);
            for (int r = jr; r < h.R; r += rows) {
                for (int v = v0 + jv; v <= v1; v += h.spread) {
                    const f32x4 a = entry(r, v);
                    const float d = mean - a.z, dev = fmaf(-a.w, d, a.x);
                    u[0] += dev;
                    u[1] += fmaf(-d, a.x + dev, a.y);         // s2 - 2 d s1 + count d^2
                }
            }
            sum_lanes(u, h.lanes);
            if (j == 0) {
                res[vg] = mean;
                res[all + vg] = u[0] * inv;
                res[2 * all + vg] = u[1];
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const int at = p.here ? p.q * h.sg + p.group(h, e) : 0;
            m[e] = res[at];
            off[e] = res[all + at];
            sq[e] = res[2 * all + at];
        }
    } else {
        float *tile = lds, *res = lds + T * N + h.slices * h.Q * h.nv * N;
        const float count = (float)t.rows;
        float x[1][M];
#pragma unroll
        for (int e = 0; e < M; ++e) x[0][e] = t.rows ? fmaf(count, t.shift[e] - base[e], t.s1[e]) : 0.f;
        sum_groups<N, T>(x, tile, res, h, p);
#pragma unroll
        for (int e = 0; e < M; ++e) {
            m[e] = fmaf(res[p.here ? p.q * h.sg + p.group(h, e) : 0], inv, base[e]);
            x[0][e] = t.rows ? fmaf(-count, m[e] - t.shift[e], t.s1[e]) : 0.f;
        }
        sum_groups<N, T>(x, tile, res + all, h, p);
#pragma unroll
        for (int e = 0; e < M; ++e) {
            off[e] = res[all + (p.here ? p.q * h.sg + p.group(h, e) : 0)] * inv;
            x[0][e] = t.rows ? fmaf(t.shift[e] - m[e], t.s1[e] + x[0][e], t.s2[e]) : 0.f;
        }
        sum_groups<N, T>(x, tile, res + 2 * all, h, p);
#pragma unroll
        for (int e = 0; e < M; ++e) sq[e] = res[2 * all + (p.here ? p.q * h.sg + p.group(h, e) : 0)];
    }
}

// Bytes of LDS that they take.
size_t lds_of_statistics(GnMode mode, const GnShape& h, int N, int T) {
    const size_t tile = mode == kWhole ? 4 * (size_t)T : mode == kSpan ? 8 * (size_t)T
                                       : (size_t)T * N + (size_t)h.slices * h.Q * h.nv * N;
    return sizeof(float) * (tile + 3 * (size_t)h.Q * h.sg);
}

// Where a vector holds several groups: of each element's group the first value, which the group's threads share.  A value
// of another group would not do: its distance may be any number of deviations.  (Not finite: nor is then the group's mean.)
// They are in the vector itself, but for the first element's.
template <int X, int MODE, bool TINY, int N>
struct Base {
    Raw<X, N> x;
    float before;

    __device__ __forceinline__ Base(uint64_t image, const GnShape& h, const Place<MODE, N>& p) {
        if constexpr (MODE == kMany) {
            const int c = p.c0 + p.group(h, 0) * h.cg;
            load_vector<X, TINY>(x, image, h, p);
            before = load_one<X>(image + (uint64_t)((c < h.C ? c : h.C - 1) * kSize<X>));
        }
    }

    template <int M>
    __device__ __forceinline__ void get(float (&base)[M], const GnShape& h, const Place<MODE, N>& p) {
        if constexpr (MODE == kMany) {
            float f[N];
            into_row<X, true>(x, p.past);
            x.widen(f);
            int g = p.group(h, 0);
            base[0] = before;
#pragma unroll
            for (int e = 1; e < N; ++e) {
                const int last = g;
                g = p.group(h, e);
                base[e] = g != last ? f[e] : base[e - 1];
            }
        }
    }
};

// y of one vector: (x - m) * scale + bias, activated.
template <int X, bool RAGGED, bool STREAM, int MODE, int N>
__device__ __forceinline__ void put_vector(const Raw<X, N>& x, const float (&m)[Moments<MODE, N>::M], const float (&scale)[N],
                                           const float (&bias)[N], uint64_t row, const Place<MODE, N>& p, const GnShape& h) {
    float f[N];
    x.widen(f);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = fmaf(f[e] - m[MODE == kWhole ? 0 : e], scale[e], bias[e]);
    activate(f, h.act);
    store_vector<X, RAGGED, STREAM>(f, row, p);
}

// A sample's slab that stays in registers, V vectors to a thread.
template <int X, int MODE, int T, int V>
__global__ __launch_bounds__(T) void k_gn_fwd(GnArgs a, GnShape h) {
    constexpr int N = kVec<X>, M = MODE == kWhole ? 1 : N;
    extern __shared__ __align__(16) float lds[];
    const uint32_t id = xcd_block(gridDim.x);
    const Place<MODE, N> p(h, (int)(id % (uint32_t)h.slabs));
    const int64_t n = (int64_t)(id / (uint32_t)h.slabs) * h.Q + p.q;
    const bool in = p.here && n < a.N && p.left > 0;
    const int most = (h.S + h.R - 1) / h.R, last = p.r + (most - 1) * h.R;    // rows of a thread; its last row
    const bool fits = last < h.S;
    const uint64_t image = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)((n < a.N ? n : a.N - 1) * a.x.sample);
    const uint64_t xr = image + (uint64_t)(p.r * a.x.ld), xl = image + (uint64_t)((fits ? last : h.S - 1) * a.x.ld);
    const int64_t step = h.R * a.x.ld;
    Raw<X, N> x[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < most) load_vector<X, false>(x[i], i + 1 < most ? xr + (uint64_t)(i * step) : xl, h, p);
    Base<X, MODE, false, N> first(image, h, p);
    float scale[N], bias[N];
    load_weight<X>(scale, a.gamma, h, p.c, 1.f);
    load_weight<X>(bias, a.beta, h, p.c, 0.f);
    Moments<MODE, N> t;
    if (in) {
        if_ragged(p.ragged, [&](auto ragged) {
            constexpr bool RAGGED = decltype(ragged)::value;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (i >= most) continue;
                float f[N];
                into_row<X, RAGGED>(x[i], p.past);
                x[i].widen(f);
                if (i == 0) t.template start<RAGGED>(f, p);
                if (i + 1 < most || fits) t.template add<RAGGED>(f, p);
            }
        });
    }
    float base[M], m[M], off[M], sq[M];
    first.get(base, h, p);
    statistics<MODE, N, T>(t, base, h.inv_n, m, off, sq, lds, h, p);
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
        scale[e] *= sq[MODE == kWhole ? 0 : e];
        bias[e] = fmaf(-off[MODE == kWhole ? 0 : e], scale[e], bias[e]);
    }
    const uint64_t yr = reinterpret_cast<uint64_t>(a.y.data) + (uint64_t)(n * a.y.sample + p.r * a.y.ld);
    const int64_t stepy = h.R * a.y.ld;
    if_ragged(p.ragged, [&](auto ragged) {
        constexpr bool RAGGED = decltype(ragged)::value;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < most && (i + 1 < most || fits))
                put_vector<X, RAGGED, false>(x[i], m, scale, bias, yr + (uint64_t)(i * stepy), p, h);
    });
}

// ---- images that do not stay in registers ------------------------------------
// Two kernels with the same workgroups on the same parts of the images: the statistics of each part, then y.  Images of up
// to about 128 MB are in the last-level cache when the second reads them.

// Of a part (and piece) of a group: the mean m + off and the sum of squares about it.
typedef f32x4 GnRecord;

template <int X, int MODE, bool TINY, int T>
__global__ __launch_bounds__(T) void k_gn_stats(GnArgs a, GnShape h, GnRecord* __restrict__ records) {
    constexpr int N = kVec<X>, M = MODE == kWhole ? 1 : N;
    extern __shared__ __align__(16) float lds[];
    const PartOf o(h, xcd_block(gridDim.x));
    const Place<MODE, N> p(h, o.slab);
    const uint64_t image = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(o.n * a.x.sample);
    const bool in = p.here && p.left > 0;
    Base<X, MODE, TINY, N> first(image, h, p);
    Moments<MODE, N> t;
    const Rows rows(h, o.part, p.r);
    if (in && rows.full + rows.tail > 0) {
        if_ragged(TINY || p.ragged, [&](auto ragged) {
            constexpr bool RAGGED = decltype(ragged)::value;
            const int64_t step = h.R * a.x.ld, stride = (int64_t)h.parts * kAhead * step;
            uint64_t row = image + (uint64_t)(rows.first * a.x.ld);
            Raw<X, N> x[kAhead], y[kAhead];
            auto load = [&](Raw<X, N>(&to)[kAhead], int many) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (i < many) load_vector<X, TINY>(to[i], row + (uint64_t)(i * step), h, p);
                row += (uint64_t)stride;
            };
            auto add = [&](Raw<X, N>(&of)[kAhead], int many, bool first) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (i >= many) continue;
                    float f[N];
                    into_row<X, RAGGED>(of[i], p.past);
                    of[i].widen(f);
                    if (i == 0 && first) t.template start<RAGGED>(f, p);
                    t.template add<RAGGED>(f, p);
                }
            };
            // the next vectors are on their way while these are added
            if (rows.full > 0) {
                load(x, kAhead);
                for (int i = 0; i + 1 < rows.full; ++i) {
                    load(y, kAhead);
                    add(x, kAhead, i == 0);
                    // after 8, 16, 32, ... rows: of an outlier's square in the first of them, 8 at most, each later one adds less
                    if (kAhead * (i + 1) >= 8 && (i & (i + 1)) == 0) t.template recentre<RAGGED>(p);
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) x[k] = y[k];
                }
                if (rows.tail > 0) load(y, rows.tail);
                add(x, kAhead, rows.full == 1);
                if (rows.tail > 0) add(y, rows.tail, false);
            } else {
                load(x, rows.tail);
                add(x, rows.tail, true);
            }
        });
        t.end();
    }
    // of the groups' values in this part and slab
    const float count = (float)positions_of(h, o.part) * (float)(h.pieces == 1 ? h.cg : p.channels), inv = 1.f / count;
    float base[M], m[M], off[M], sq[M];
    first.get(base, h, p);
    statistics<MODE, N, T>(t, base, inv, m, off, sq, lds, h, p);
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

template <int X, int MODE, bool TINY, int T>
__global__ __launch_bounds__(T) void k_gn_apply(GnArgs a, GnShape h, const GnRecord* __restrict__ records) {
    constexpr int N = kVec<X>, M = MODE == kWhole ? 1 : N;
    extern __shared__ __align__(16) float lds[];        // m, what its rounding left, 1/deviation of the slab's groups
    const PartOf o(h, xcd_block(gridDim.x));
    const Place<MODE, N> p(h, o.slab);
    const bool in = p.here && p.left > 0;
    const Rows rows(h, o.part, p.r);
    const int64_t step = h.R * a.x.ld, stepy = h.R * a.y.ld, ahead = (int64_t)h.parts * kAhead;
    uint64_t row = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(o.n * a.x.sample + rows.first * a.x.ld);
    uint64_t yr = reinterpret_cast<uint64_t>(a.y.data) + (uint64_t)(o.n * a.y.sample + rows.first * a.y.ld);
    int full = in ? rows.full : 0;
    const int tail = in ? rows.tail : 0;
    Raw<X, N> x[kAhead];
    auto load = [&]() {     // the next chunk, or the incomplete one
        const int many = full > 0 ? kAhead : tail;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < many) load_vector<X, TINY>(x[i], row + (uint64_t)(i * step), h, p);
        row += (uint64_t)(ahead * step);
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
            const int part = h.pieces == 1 ? k : k / h.pieces, first = (k - part * h.pieces) * h.nv * N;
            return (double)positions_of(h, part) * (h.pieces == 1 ? h.cg : h.nv * N < h.cg - first ? h.nv * N : h.cg - first);
        };
        double sum = 0.0, sq = 0.0;
        for (int k = j; k < K; k += h.lanes) {
            const GnRecord r = of[(int64_t)k * h.G];
            sum += count(k) * ((double)r.x + (double)r.y);
        }
        for (int b = h.lanes >> 1; b; b >>= 1) sum += __shfl_xor(sum, b, 64);
        const double mean = sum * h.inv_count;
        for (int k = j; k < K; k += h.lanes) {
            const GnRecord r = of[(int64_t)k * h.G];
            const double d = (double)r.x + (double)r.y - mean;
            sq += (double)r.z + count(k) * d * d;
        }
        for (int b = h.lanes >> 1; b; b >>= 1) sq += __shfl_xor(sq, b, 64);
        if (j == 0) {
            const float m = (float)mean, rstd = 1.f / sqrtf((float)(sq * h.inv_count) + a.eps);
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
    if (full + tail == 0) return;
    float m[M];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int g = p.group(h, e);
        if (e < M) m[e] = lds[3 * g];
        scale[e] *= lds[3 * g + 2];
        bias[e] = fmaf(-lds[3 * g + 1], scale[e], bias[e]);
    }
    auto all = [&](auto ragged, auto stream) {
        constexpr bool RAGGED = decltype(ragged)::value, STREAM = decltype(stream)::value;
        auto put = [&](Raw<X, N>& v, int i) {
            into_row<X, RAGGED>(v, p.past);
            put_vector<X, RAGGED, STREAM>(v, m, scale, bias, yr + (uint64_t)(i * stepy), p, h);
        };
        while (full > 0) {
            Raw<X, N> now[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) now[i] = x[i];
            --full;
            load();
#pragma unroll
            for (int i = 0; i < kAhead; ++i) put(now[i], i);
            yr += (uint64_t)(ahead * stepy);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < tail) put(x[i], i);
    };
    const std::integral_constant<bool, true> yes;
    const std::integral_constant<bool, false> no;
    if (TINY || p.ragged) all(yes, no);
    else if (h.stream) all(no, yes);
    else all(no, no);
}

// ---- on the host -------------------------------------------------------------

constexpr TeamSize kTeams[] = {{256, 1}, {256, 2}, {256, 4}, {512, 4}, {512, 8}};

// Calls f with the team's sizes as constants.
template <typename F>
hipError_t with_team(int k, F f) {
#define GA_TEAM(K)     if (k == K) return f(std::integral_constant<int, kTeams[K].T>{}, std::integral_constant<int, kTeams[K].V>{})
    GA_TEAM(0);
    GA_TEAM(1);
    GA_TEAM(2);
    GA_TEAM(3);
    GA_TEAM(4);
#undef GA_TEAM
    return hipErrorInvalidValue;
}

constexpr int kWideThreads = 256;

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
    const int k = choose(h, N, kTeams, 4, all.N);
    if (k >= 0) {
        const GnMode mode = mode_of(h, N);
        const size_t bytes = lds_of_statistics(mode, h, N, kTeams[k].T);
        const int64_t step = kMostBlocks / h.slabs * h.Q;
        for (int64_t n0 = 0; n0 < all.N; n0 += step) {
            const GnArgs a = samples_of(all, n.G, n0, all.N - n0 < step ? all.N - n0 : step);
            const unsigned blocks = (unsigned)(ceil_div(a.N, h.Q) * h.slabs);
            const hipError_t e = with_team(k, [&](auto t, auto v) {
                constexpr int T = decltype(t)::value, V = decltype(v)::value;
                with_mode(mode, [&](auto m) {
                    hipLaunchKernelGGL((k_gn_fwd<X, decltype(m)::value, T, V>), dim3(blocks), dim3(T), bytes, s, a, h);
                });
                return hipGetLastError();
            });
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    constexpr int T = kWideThreads;
    lay_wide(h, N, T, all.N);
    h.stream = whole_lines(h, all.y, kSize<X>);
    const bool tiny = h.C < N;
    const GnMode mode = tiny ? kMany : mode_of(h, N);
    const size_t bytes = lds_of_statistics(mode, h, N, T);
    // as many samples at once as the records have room for
    const int64_t per = (int64_t)h.parts * h.pieces * n.G;
    int64_t step = kGnRecords / per;
    if (step > kMostBlocks / ((int64_t)h.parts * h.slabs)) step = kMostBlocks / ((int64_t)h.parts * h.slabs);
    if (step < 1) return hipErrorInvalidValue;
    for (int64_t n0 = 0; n0 < all.N; n0 += step) {
        const GnArgs a = samples_of(all, n.G, n0, all.N - n0 < step ? all.N - n0 : step);
        const unsigned blocks = (unsigned)(a.N * h.parts * h.slabs);
        GnRecord* records = reinterpret_cast<GnRecord*>(n.d_records);
        auto launch = [&](auto m, auto t) {
            constexpr int MODE = decltype(m)::value;
            constexpr bool TINY = decltype(t)::value;
            hipLaunchKernelGGL((k_gn_stats<X, MODE, TINY, T>), dim3(blocks), dim3(T), bytes, s, a, h, records);
            hipLaunchKernelGGL((k_gn_apply<X, MODE, TINY, T>), dim3(blocks), dim3(T), sizeof(float) * 3 * h.sg, s, a, h,
                               records);
        };
        if (tiny) launch(std::integral_constant<int, kMany>{}, std::integral_constant<bool, true>{});
        else with_mode(mode, [&](auto m) { launch(m, std::integral_constant<bool, false>{}); });
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
