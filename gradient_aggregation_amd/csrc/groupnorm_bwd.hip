// Group norm backward, through its activation (ga_groupnorm_backward).
//
// The sums of dz and dz * xh over a sample's positions, for each channel, give both
// what dx needs (a group's means of h = dz * gamma and h * xh are those sums weighted
// by gamma) and the weight gradients (those sums added over the samples).
//
// What bounds it: 16 x 16384 x 128 bf16 with silu, 34 to 36 us for the sums (3.7 TB/s; 20 vector instructions to an element,
// two of them transcendental: 63% of the time of the SIMDs, whose two wavefronts wait for the rest) and 34 us for dx (5.9
// TB/s); 6 x 1443 x 250 binary32 13 and 8.5 us, few rows to a thread and a slab that leaves half of its threads idle;
// 4 x 36 x 1024, held in registers, 6.7 us of one kernel.
#include "groupnorm.h"
#include "training.h"

namespace ga {

namespace {

// What dx and the sums need of a vector's channels.
template <int X, int MODE, int N>
struct Channels {
    static constexpr int M = MODE == kWhole ? 1 : N;
    float gamma[N], beta[N], mean[M], rstd[M];

    __device__ __forceinline__ void weights(const GnArgs& a, const GnShape& h, int c) {
        load_weight<X>(gamma, a.gamma, h, c, 1.f);
        load_weight<X>(beta, a.beta, h, c, 0.f);
    }

    __device__ __forceinline__ void sample(const GnArgs& a, const GnShape& h, int64_t n, const Place<MODE, N>& p, bool in) {
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const int g = p.g0 + p.group(h, e);
            const int64_t at = n * h.G + (g < h.G ? g : h.G - 1);
            mean[e] = in ? a.mean[at] : 0.f;
            rstd[e] = in ? a.rstd[at] : 0.f;
        }
    }

    __device__ __forceinline__ void values(const Raw<X, N>& x, const Raw<X, N>& dy, float (&xh)[N], float (&dz)[N],
                                           int32_t act) const {
        x.widen(xh);
        dy.widen(dz);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int k = MODE == kWhole ? 0 : e;
            xh[e] = (xh[e] - mean[k]) * rstd[k];
        }
        through_activation(dz, xh, gamma, beta, act);
    }

    __device__ __forceinline__ void add(const Raw<X, N>& x, const Raw<X, N>& dy, float (&s)[2][N], int32_t act) const {
        float xh[N], dz[N];
        values(x, dy, xh, dz, act);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            s[0][e] += dz[e];
            s[1][e] = fmaf(dz[e], xh[e], s[1][e]);
        }
    }

    // dx = rstd * (dz * gamma - m1 - xh * m2); m1 and m2 come times -rstd.
    template <bool RAGGED, bool STREAM>
    __device__ __forceinline__ void put(const Raw<X, N>& x, const Raw<X, N>& dy, const float (&m1)[M], const float (&m2)[M],
                                        uint64_t row, const Place<MODE, N>& p, const GnShape& h) const {
        float xh[N], dz[N];
        values(x, dy, xh, dz, h.act);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int k = MODE == kWhole ? 0 : e;
            dz[e] = fmaf(dz[e], gamma[e] * rstd[k], fmaf(xh[e], m2[k], m1[k]));
        }
        store_vector<X, RAGGED, STREAM>(dz, row, p);
    }
};

// From the channels' sums (sum_channels, two values) of `samples` samples: those of the groups, weighted by gamma and
// times `scale`, into res; and the channels' own, added to acc.
template <int X, int N, int T>
__device__ __forceinline__ void share_sums(const GnArgs& a, const GnShape& h, int c0, int channels, int samples,
                                           const float* sums, float* res, float* acc, float scale) {
    const int wide = h.nv * N, pairs = h.Q * wide, plane = h.slices * pairs, all = h.Q * h.sg;
    const int j = threadIdx.x & (h.lanes - 1);
    for (int vg = threadIdx.x / h.lanes; vg < all; vg += T / h.lanes) {
        const int q = h.Q == 1 ? 0 : vg / h.sg, g = vg - q * h.sg;
        float t[2] = {0.f, 0.f};
        for (int i = j; i < h.cg; i += h.lanes) {
            const int c = g * h.cg + i;
            if (c >= channels) break;
            float u[2] = {0.f, 0.f}, weight = 1.f;
            if (a.gamma) {
                const uint64_t at = reinterpret_cast<uint64_t>(a.gamma);
                weight = h.p32 ? load_one<kF32>(at + (uint64_t)(c0 + c) * 4) : load_one<X>(at + (uint64_t)(c0 + c) * kSize<X>);
            }
#pragma unroll 4
            for (int k = 0; k < h.slices; ++k) {
                u[0] += sums[k * pairs + q * wide + c];
                u[1] += sums[plane + k * pairs + q * wide + c];
            }
            t[0] = fmaf(weight, u[0], t[0]);
            t[1] = fmaf(weight, u[1], t[1]);
        }
        sum_lanes(t, h.lanes);
        if (j == 0) {
            res[vg] = t[0] * scale;
            res[all + vg] = t[1] * scale;
        }
    }
    if (!a.dgamma) return;
    for (int c = threadIdx.x; c < channels; c += T) {
        float u[2] = {acc[c], acc[wide + c]};
        for (int q = 0; q < samples; ++q) {
#pragma unroll 4
            for (int k = 0; k < h.slices; ++k) {
                u[0] += sums[k * pairs + q * wide + c];
                u[1] += sums[plane + k * pairs + q * wide + c];
            }
        }
        acc[c] = u[0];
        acc[wide + c] = u[1];
    }
}

// A workgroup's weight gradients: the result itself where the worker has one row of them, else partial row `row`.
template <int T>
__device__ __forceinline__ void put_params(const GnArgs& a, const GnShape& h, int c0, int channels, int wide, int64_t row,
                                           const float* acc, float* __restrict__ rows_out, bool direct) {
    for (int c = threadIdx.x; c < channels; c += T) {
        if (direct) {
            store_param(a.dgamma, a.dp_dtype, row * h.C + c0 + c, acc[wide + c]);
            store_param(a.dbeta, a.dp_dtype, row * h.C + c0 + c, acc[c]);
        } else {
            rows_out[row * 2 * h.ldp + c0 + c] = acc[wide + c];
            rows_out[(row * 2 + 1) * h.ldp + c0 + c] = acc[c];
        }
    }
}

// Samples' slabs that stay in registers, V vectors to a thread: workgroup (worker, row) takes every h.rows-th Q samples
// of the worker (all of them where there are weight gradients).
template <int X, int MODE, int T, int V>
__global__ __launch_bounds__(T) void k_gn_bwd(GnArgs a, GnShape h) {
    constexpr int N = kVec<X>, M = MODE == kWhole ? 1 : N;
    extern __shared__ __align__(16) float lds[];
    const int wide = h.nv * N, all = h.Q * h.sg;
    float *tile = lds, *sums = tile + 2 * T * N, *res = sums + 2 * h.slices * h.Q * wide, *acc = res + 2 * all;
    const uint32_t id = xcd_block(gridDim.x);
    const int row = (int)(id / (uint32_t)h.slabs), w = row / h.rows;
    const Place<MODE, N> p(h, (int)(id % (uint32_t)h.slabs));
    Channels<X, MODE, N> ch;
    ch.weights(a, h, p.c);
    for (int c = threadIdx.x; c < wide; c += T) acc[c] = acc[wide + c] = 0.f;
    const int most = (h.S + h.R - 1) / h.R, last = p.r + (most - 1) * h.R;    // rows of a thread; its last row
    const bool fits = last < h.S;
    for (int64_t b = row - w * h.rows; b * h.Q < a.per_worker; b += h.rows) {
        const int64_t left = a.per_worker - b * h.Q, n = w * a.per_worker + b * h.Q + p.q;
        const bool in = p.here && p.q < left && p.left > 0;
        const int64_t m = p.q < left ? n : n - p.q;       // a thread without a sample reads another's
        const uint64_t xi = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(m * a.x.sample);
        const uint64_t di = reinterpret_cast<uint64_t>(a.dy.data) + (uint64_t)(m * a.dy.sample);
        Raw<X, N> x[V], dy[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= most) continue;
            const int64_t at = i + 1 < most ? p.r + i * h.R : fits ? last : h.S - 1;
            load_vector<X, false>(x[i], xi + (uint64_t)(at * a.x.ld), h, p);
            load_vector<X, false>(dy[i], di + (uint64_t)(at * a.dy.ld), h, p);
        }
        ch.sample(a, h, n, p, in);
        float s[2][N];
#pragma unroll
        for (int e = 0; e < N; ++e) s[0][e] = s[1][e] = 0.f;
        if (in) {
            if_ragged(p.ragged, [&](auto ragged) {
                constexpr bool RAGGED = decltype(ragged)::value;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (i >= most) continue;
                    into_row<X, RAGGED>(x[i], p.past);
                    into_row<X, RAGGED>(dy[i], p.past);
                    if (i + 1 < most || fits) ch.add(x[i], dy[i], s, h.act);
                }
            });
        }
        sum_channels<N, T, 2>(s, tile, sums, h, p);
        share_sums<X, N, T>(a, h, p.c0, p.channels, left < h.Q ? (int)left : h.Q, sums, res, acc, h.inv_n);
        __syncthreads();
        if (!in) continue;
        float m1[M], m2[M];
#pragma unroll
        for (int e = 0; e < M; ++e) {
            m1[e] = -ch.rstd[e] * res[p.q * h.sg + p.group(h, e)];
            m2[e] = -ch.rstd[e] * res[all + p.q * h.sg + p.group(h, e)];
        }
        const uint64_t out = reinterpret_cast<uint64_t>(a.y.data) + (uint64_t)(n * a.y.sample);
        if_ragged(p.ragged, [&](auto ragged) {
            constexpr bool RAGGED = decltype(ragged)::value;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < most && (i + 1 < most || fits))
                    ch.template put<RAGGED, false>(x[i], dy[i], m1, m2, out + (uint64_t)((p.r + i * h.R) * a.y.ld), p, h);
        });
    }
    if (a.dgamma) put_params<T>(a, h, p.c0, p.channels, wide, row, acc, nullptr, true);
}

// ---- images that do not stay in registers ------------------------------------
// The sums first, then dx, each over parts of the samples.  This launch takes `count` samples of each of the workers
// [w0, ...) from each one's sample `skip`; the parts of a worker's samples go to its h.rows workgroups in turn.

struct GnSpan {
    int32_t w0;
    int32_t add;           // the partial rows hold sums already
    int64_t skip, count;
};

// Of a part (and piece) of a group: the sums of h and h * xh.
typedef f32x2 GnSums;

template <int X, int MODE, bool TINY, int T>
__global__ __launch_bounds__(T) void k_gn_sums(GnArgs a, GnShape h, GnSpan span, GnSums* __restrict__ records,
                                               float* __restrict__ rows_out, bool direct) {
    constexpr int N = kVec<X>;
    extern __shared__ __align__(16) float lds[];
    const int wide = h.nv * N;
    float *tile = lds, *sums = tile + 2 * T * N, *res = sums + 2 * h.slices * wide, *acc = res + 2 * h.sg;
    const uint32_t id = xcd_block(gridDim.x);
    const int slab = (int)(id % (uint32_t)h.slabs), row = (int)(id / (uint32_t)h.slabs), w = row / h.rows;
    const Place<MODE, N> p(h, slab);
    const bool in = p.here && p.left > 0;
    const int K = h.parts * h.pieces;
    Channels<X, MODE, N> ch;
    ch.weights(a, h, p.c);
    for (int c = threadIdx.x; c < wide; c += T) {
        const bool old = span.add && a.dgamma && c < p.channels;
        acc[c] = old ? rows_out[((int64_t)row * 2 + 1) * h.ldp + p.c0 + c] : 0.f;
        acc[wide + c] = old ? rows_out[(int64_t)row * 2 * h.ldp + p.c0 + c] : 0.f;
    }
    for (int64_t item = row - w * h.rows; item < span.count * h.parts; item += h.rows) {
        const int64_t i = item / h.parts, n = (span.w0 + w) * a.per_worker + span.skip + i;
        const int part = (int)(item - i * h.parts);
        const Rows rows(h, part, p.r);
        ch.sample(a, h, n, p, in);
        float s[2][N];
#pragma unroll
        for (int e = 0; e < N; ++e) s[0][e] = s[1][e] = 0.f;
        if (in && rows.full + rows.tail > 0) {
            if_ragged(TINY || p.ragged, [&](auto ragged) {
                constexpr bool RAGGED = decltype(ragged)::value;
                const int64_t stepx = h.R * a.x.ld, stepd = h.R * a.dy.ld, ahead = (int64_t)h.parts * kAhead;
                uint64_t xr = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(n * a.x.sample + rows.first * a.x.ld);
                uint64_t dr = reinterpret_cast<uint64_t>(a.dy.data) + (uint64_t)(n * a.dy.sample + rows.first * a.dy.ld);
                Raw<X, N> x[2][kAhead], dy[2][kAhead];
                auto load = [&](int to, int many) {
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        if (k >= many) continue;
                        load_vector<X, TINY>(x[to][k], xr + (uint64_t)(k * stepx), h, p);
                        load_vector<X, TINY>(dy[to][k], dr + (uint64_t)(k * stepd), h, p);
                    }
                    xr += (uint64_t)(ahead * stepx);
                    dr += (uint64_t)(ahead * stepd);
                };
                auto add = [&](int of, int many) {
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        if (k >= many) continue;
                        into_row<X, RAGGED>(x[of][k], p.past);
                        into_row<X, RAGGED>(dy[of][k], p.past);
                        ch.add(x[of][k], dy[of][k], s, h.act);
                    }
                };
                // the next vectors are on their way while these are added
                load(0, rows.full > 0 ? kAhead : rows.tail);
                for (int i = 0; i < rows.full; ++i) {
                    if (i + 1 < rows.full) load(1, kAhead);
                    else load(1, rows.tail);
                    add(0, kAhead);
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        x[0][k] = x[1][k];
                        dy[0][k] = dy[1][k];
                    }
                }
                if (rows.tail > 0) add(0, rows.tail);
            });
        }
        sum_channels<N, T, 2>(s, tile, sums, h, p);
        share_sums<X, N, T>(a, h, p.c0, p.channels, 1, sums, res, acc, 1.f);
        __syncthreads();
        const int64_t r = ((w * span.count + i) * K + part * h.pieces + (h.pieces == 1 ? 0 : slab % h.pieces)) * h.G;
        for (int g = threadIdx.x; g < h.sg; g += T)
            if (p.g0 + g < h.G) records[r + p.g0 + g] = GnSums{res[g], res[h.sg + g]};
    }
    if (a.dgamma) put_params<T>(a, h, p.c0, p.channels, wide, direct ? span.w0 + w : row, acc, rows_out, direct);
}

// Workgroups past the images' add the partial rows of the weight gradients: of worker w0 + i those of 32 channels, which
// eight rows of threads share and then add in order.
template <int T>
__device__ __forceinline__ void end_params(const GnArgs& a, const GnShape& h, int32_t w0, const float* __restrict__ rows_in,
                                           uint32_t job, float* lds) {
    constexpr int SHARE = T / 32;
    const int groups = (h.C + 31) / 32, i = (int)(job / (uint32_t)groups), c = (int)(job % (uint32_t)groups) * 32 + (threadIdx.x & 31);
    const int share = threadIdx.x / 32;
    float dg = 0.f, db = 0.f;
    if (c < h.C) {
        const float* in = rows_in + (int64_t)i * h.rows * 2 * h.ldp + c;
#pragma unroll 4
        for (int r = share; r < h.rows; r += SHARE) {
            dg += in[(int64_t)r * 2 * h.ldp];
            db += in[((int64_t)r * 2 + 1) * h.ldp];
        }
    }
    lds[threadIdx.x] = dg;
    lds[T + threadIdx.x] = db;
    __syncthreads();
    if (share != 0 || c >= h.C) return;
    for (int k = 1; k < SHARE; ++k) {
        dg += lds[k * 32 + threadIdx.x];
        db += lds[T + k * 32 + threadIdx.x];
    }
    store_param(a.dgamma, a.dp_dtype, (int64_t)(w0 + i) * h.C + c, dg);
    store_param(a.dbeta, a.dp_dtype, (int64_t)(w0 + i) * h.C + c, db);
}

template <int X, int MODE, bool TINY, int T>
__global__ __launch_bounds__(T) void k_gn_dx(GnArgs a, GnShape h, GnSpan span, const GnSums* __restrict__ records,
                                             const float* __restrict__ rows_in, uint32_t images) {
    constexpr int N = kVec<X>, M = MODE == kWhole ? 1 : N;
    extern __shared__ __align__(16) float lds[];        // the means of h and h * xh of the slab's groups, 64 at most
    if (blockIdx.x >= images) {
        end_params<T>(a, h, span.w0, rows_in, blockIdx.x - images, lds);
        return;
    }
    const PartOf o(h, xcd_block(images));
    const Place<MODE, N> p(h, o.slab);
    const bool in = p.here && p.left > 0;
    const int64_t w = o.n / span.count, n = (span.w0 + w) * a.per_worker + span.skip + (o.n - w * span.count);
    const Rows rows(h, o.part, p.r);
    const int64_t stepx = h.R * a.x.ld, stepd = h.R * a.dy.ld, stepy = h.R * a.y.ld, ahead = (int64_t)h.parts * kAhead;
    uint64_t xr = reinterpret_cast<uint64_t>(a.x.data) + (uint64_t)(n * a.x.sample + rows.first * a.x.ld);
    uint64_t dr = reinterpret_cast<uint64_t>(a.dy.data) + (uint64_t)(n * a.dy.sample + rows.first * a.dy.ld);
    uint64_t yr = reinterpret_cast<uint64_t>(a.y.data) + (uint64_t)(n * a.y.sample + rows.first * a.y.ld);
    int full = in ? rows.full : 0;
    const int tail = in ? rows.tail : 0;
    Raw<X, N> x[kAhead], dy[kAhead];
    auto load = [&]() {     // the next chunk, or the incomplete one
        const int many = full > 0 ? kAhead : tail;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (k >= many) continue;
            load_vector<X, TINY>(x[k], xr + (uint64_t)(k * stepx), h, p);
            load_vector<X, TINY>(dy[k], dr + (uint64_t)(k * stepd), h, p);
        }
        xr += (uint64_t)(ahead * stepx);
        dr += (uint64_t)(ahead * stepd);
    };
    load();
    Channels<X, MODE, N> ch;
    ch.weights(a, h, p.c);
    ch.sample(a, h, n, p, in);
    const int K = h.parts * h.pieces, j = threadIdx.x & (h.lanes - 1);
    for (int g = threadIdx.x / h.lanes; g < h.sg; g += T / h.lanes) {
        const GnSums* of = records + o.n * K * h.G + (p.g0 + g < h.G ? p.g0 + g : h.G - 1);
        float t[2] = {0.f, 0.f};
        for (int k = j; k < K; k += h.lanes) {
            const GnSums r = of[(int64_t)k * h.G];
            t[0] += r.x;
            t[1] += r.y;
        }
        sum_lanes(t, h.lanes);
        if (j == 0) {
            lds[2 * g] = t[0] * h.inv_n;
            lds[2 * g + 1] = t[1] * h.inv_n;
        }
    }
    __syncthreads();
    if (full + tail == 0) return;
    float m1[M], m2[M];
#pragma unroll
    for (int e = 0; e < M; ++e) {
        m1[e] = -ch.rstd[e] * lds[2 * p.group(h, e)];
        m2[e] = -ch.rstd[e] * lds[2 * p.group(h, e) + 1];
    }
    auto all = [&](auto ragged, auto stream) {
        constexpr bool RAGGED = decltype(ragged)::value, STREAM = decltype(stream)::value;
        auto put = [&](Raw<X, N>& u, Raw<X, N>& v, int k) {
            into_row<X, RAGGED>(u, p.past);
            into_row<X, RAGGED>(v, p.past);
            ch.template put<RAGGED, STREAM>(u, v, m1, m2, yr + (uint64_t)(k * stepy), p, h);
        };
        while (full > 0) {
            Raw<X, N> u[kAhead], v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                u[k] = x[k];
                v[k] = dy[k];
            }
            --full;
            load();
#pragma unroll
            for (int k = 0; k < kAhead; ++k) put(u[k], v[k], k);
            yr += (uint64_t)(ahead * stepy);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k < tail) put(x[k], dy[k], k);
    };
    const std::integral_constant<bool, true> yes;
    const std::integral_constant<bool, false> no;
    if (TINY || p.ragged) all(yes, no);
    else if (h.stream) all(no, yes);
    else all(no, no);
}

// ---- on the host -------------------------------------------------------------

constexpr TeamSize kTeams[] = {{256, 1}, {256, 2}, {256, 4}, {512, 4}};

template <typename F>
hipError_t with_team(int k, F f) {
#define GA_TEAM(K) \
    if (k == K) return f(std::integral_constant<int, kTeams[K].T>{}, std::integral_constant<int, kTeams[K].V>{})
    GA_TEAM(0);
    GA_TEAM(1);
    GA_TEAM(2);
    GA_TEAM(3);
#undef GA_TEAM
    return hipErrorInvalidValue;
}

constexpr int kWideThreads = 256;

size_t lds_bytes(const GnShape& h, int N, int T) {
    return sizeof(float) * (2 * (size_t)T * N + 2 * (size_t)h.slices * h.Q * h.nv * N + 2 * (size_t)h.Q * h.sg +
                            2 * (size_t)h.nv * N);
}

// Workgroups (rows of the weight gradients) of each of `workers` workers for so many items of work.
int32_t rows_of(const GroupNorm& n, const GnArgs& a, int64_t items, int64_t workers) {
    int64_t r = (a.dgamma ? n.rows : kGnRows) / workers;
    if (r > items) r = items;
    return r < 1 ? 1 : (int32_t)r;
}

template <int X>
hipError_t gn_bwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    constexpr int N = kVec<X>;
    if (a.N == 0) return launch_params_end(n.d_rows, n.C, n.ldp, 0, a.workers, a.dgamma, a.dbeta, a.dp_dtype, s);
    GnShape h = shape_of(n, a.S);
    const int k = choose(h, N, kTeams, -1, a.N);
    if (k >= 0) {
        if (h.Q > a.per_worker) {
            h.Q = (int)a.per_worker;
            sharing(h, N, kTeams[k].T);
        }
        const int64_t items = ceil_div(a.per_worker, h.Q);
        // with weight gradients of more than one workgroup a worker, it would take a second kernel to add them: no better
        // than the two below (4 x 64 x 256 bf16: 12.4 us against 12.3, and 9.6 where each sample is a worker's own)
        if (!a.dgamma || items == 1) {
            const int64_t most = kMostBlocks / h.slabs / a.workers;
            h.rows = (int32_t)(items < most ? items : most < 1 ? 1 : most);
            return with_team(k, [&](auto t, auto v) {
                constexpr int T = decltype(t)::value, V = decltype(v)::value;
                const unsigned blocks = (unsigned)((int64_t)a.workers * h.rows * h.slabs);
                with_mode(mode_of(h, N), [&](auto m) {
                    hipLaunchKernelGGL((k_gn_bwd<X, decltype(m)::value, T, V>), dim3(blocks), dim3(T), lds_bytes(h, N, T), s,
                                       a, h);
                });
                return hipGetLastError();
            });
        }
        h = shape_of(n, a.S);
    }
    constexpr int T = kWideThreads;
    lay_wide(h, N, T, a.N);
    h.stream = whole_lines(h, a.y, kSize<X>);
    const size_t bytes = lds_bytes(h, N, T);
    GnSums* records = reinterpret_cast<GnSums*>(n.d_records);
    // as many samples at once as the records have room for: of several workers, or a part of one's
    const int64_t per = (int64_t)h.parts * h.pieces * n.G;
    int64_t room = 2 * kGnRecords / per;
    if (room > kMostBlocks / ((int64_t)h.parts * h.slabs)) room = kMostBlocks / ((int64_t)h.parts * h.slabs);
    if (room < 1) return hipErrorInvalidValue;
    int64_t together = room / a.per_worker, count = a.per_worker;
    if (together < 1) {
        together = 1;
        count = room;
    }
    if (together > a.workers) together = a.workers;
    if (a.dgamma && together > n.rows) together = n.rows;
    h.rows = rows_of(n, a, count * h.parts, together);
    const bool direct = h.rows == 1 && count == a.per_worker;
    for (int64_t w0 = 0; w0 < a.workers; w0 += together) {
        const int64_t here = a.workers - w0 < together ? a.workers - w0 : together;
        for (int64_t skip = 0; skip < a.per_worker; skip += count) {
            const GnSpan span = {(int32_t)w0, skip > 0, skip, a.per_worker - skip < count ? a.per_worker - skip : count};
            const unsigned blocks = (unsigned)(here * h.rows * h.slabs);
            const unsigned images = (unsigned)(here * span.count * h.parts * h.slabs);
            const bool last = skip + span.count == a.per_worker;
            const unsigned ends = a.dgamma && !direct && last ? (unsigned)(here * ceil_div(h.C, 32)) : 0u;
            auto launch = [&](auto m, auto t) {
                constexpr int MODE = decltype(m)::value;
                constexpr bool TINY = decltype(t)::value;
                hipLaunchKernelGGL((k_gn_sums<X, MODE, TINY, T>), dim3(blocks), dim3(T), bytes, s, a, h, span, records,
                                   n.d_rows, direct);
                hipLaunchKernelGGL((k_gn_dx<X, MODE, TINY, T>), dim3(images + ends), dim3(T), sizeof(float) * 2 * T, s, a, h, span, records,
                                   n.d_rows, images);
            };
            if (h.C < N) launch(std::integral_constant<int, kMany>{}, std::integral_constant<bool, true>{});
            else with_mode(mode_of(h, N), [&](auto m) { launch(m, std::integral_constant<bool, false>{}); });
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_gn_bwd(const GroupNorm& n, const GnArgs& a, hipStream_t s) {
    if (n.x_dtype == GA_FP32) return gn_bwd<kF32>(n, a, s);
    return n.x_dtype == GA_FP16 ? gn_bwd<kF16>(n, a, s) : gn_bwd<kB16>(n, a, s);
}

}  // namespace ga
