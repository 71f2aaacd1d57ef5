// What both passes of the group norm share: how workgroups lie on channels-last
// images, the activations, and sums over a group's or a channel's values.
#pragma once

#include <type_traits>

#include "layers.h"
#include "rowvec.h"

namespace ga {

// A workgroup takes a slab: some whole groups (consecutive channels) or a piece of one, R positions at once, a vector
// of N channels to a thread.  Where a sample's slab stays in registers, it may take Q samples at once.
struct GnShape {
    int32_t C, G, cg;      // channels, groups, channels of a group
    int32_t sg, nv;        // groups (1 for a piece) and vectors of a slab; the last one may have fewer
    int32_t slabs, pieces; // slabs of the channels; pieces of a group
    int32_t R, Q;
    int32_t lanes;         // threads that add a group's sums (a power of 2, at most 64)
    int32_t slices;        // threads that share the rows of a channel's sum
    int32_t S;
    int32_t p32, act;      // weights in binary32; activation
    int32_t parts, span;   // images that do not stay in registers: parts of a sample, positions of a part
    int32_t rows;          // backward: partial rows of the weight gradients of a worker
    int32_t ldp;           // their stride
    int32_t res_at;        // where the groups' sums lie in LDS
    float inv_n;           // 1 / (S * cg)
};

// Consecutive workgroups go to the 8 XCDs in turn: those of an XCD take consecutive work, so that slabs beside each
// other, which share cache lines, share a cache.
__device__ __forceinline__ uint32_t xcd_block() {
    const uint32_t b = blockIdx.x, n = gridDim.x, x = b & 7u, per = n >> 3, rest = n & 7u;
    return x * per + (x < rest ? x : rest) + (b >> 3);
}

template <int X, int N>
__device__ __forceinline__ void load_weight(float (&f)[N], const void* p, const GnShape& h, int c, float fill) {
    if (h.p32) load_param<kF32>(f, p, c, h.C, fill);
    else load_param<X>(f, p, c, h.C, fill);
}

// 1 / (1 + exp(-z)): the hardware's base-2 exponential and reciprocal, each within 1 ulp; the exponent's rounding
// adds |z| half ulps.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int32_t act) {
    if (act == GA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < N; ++e) z[e] *= sigmoid(z[e]);
    } else if (act == GA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) z[e] = z[e] < 0.f ? 0.f : z[e];
    }
}

// dy -> dz, z = xh * gamma + beta.
template <int N>
__device__ __forceinline__ void through_activation(float (&dy)[N], const float (&xh)[N], const float (&gamma)[N],
                                                   const float (&beta)[N], int32_t act) {
    if (act == GA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float z = fmaf(xh[e], gamma[e], beta[e]), s = sigmoid(z);
            dy[e] *= s * fmaf(z, 1.f - s, 1.f);
        }
    } else if (act == GA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) dy[e] = fmaf(xh[e], gamma[e], beta[e]) <= 0.f ? 0.f : dy[e];
    }
}

// The slab's channels, and a thread's place: row r of sample q, vector v, whose first channel is c (of all).  WHOLE:
// each vector lies in one group.
template <bool WHOLE, int N>
struct Place {
    int g0, c0, channels;  // first group and channel (of all), channels of the slab
    int q, r, v, c;
    int left;              // elements of the vector within the slab (none: 0 or less)
    uint32_t past;         // elements that its loads are moved to the front by, to end with the row
    bool here;             // the thread has a place

    __device__ __forceinline__ Place(const GnShape& h, int slab) {
        const int t = threadIdx.x, per = h.nv * h.R;
        if (h.pieces == 1) {
            g0 = slab * h.sg;
            c0 = g0 * h.cg;
            channels = (h.sg < h.G - g0 ? h.sg : h.G - g0) * h.cg;
        } else {
            g0 = slab / h.pieces;
            const int first = (slab - g0 * h.pieces) * h.nv * N;
            c0 = g0 * h.cg + first;
            channels = h.nv * N < h.cg - first ? h.nv * N : h.cg - first;
        }
        q = t / per;
        r = (t - q * per) / h.nv;
        v = t - q * per - r * h.nv;
        here = q < h.Q;
        c = c0 + v * N;
        left = channels - v * N;
        past = h.C >= N && c < h.C && c + N > h.C ? c + N - h.C : 0;
    }

    // Group (of the slab) of element e.
    __device__ __forceinline__ int group(const GnShape& h, int e) const {
        const int g = h.sg == 1 ? 0 : (v * N + (WHOLE ? 0 : e)) / h.cg;
        return g < h.sg ? g : h.sg - 1;
    }
};

// Images that do not stay in registers: part `part` of sample n, positions [s0, s1), slab `slab`.
struct PartOf {
    int64_t n;
    int part, slab, s0, s1;

    __device__ __forceinline__ PartOf(const GnShape& h, uint32_t id) {
        slab = (int)(id % (uint32_t)h.slabs);
        const uint32_t rest = id / (uint32_t)h.slabs;
        part = (int)(rest % (uint32_t)h.parts);
        n = rest / (uint32_t)h.parts;
        positions(h);
    }

    __device__ __forceinline__ void positions(const GnShape& h) {
        s0 = part * h.span;
        s1 = h.S - s0 < h.span ? h.S : s0 + h.span;
    }
};

constexpr int kAhead = 4;      // vectors of a thread on their way together there

// Sums over the R rows of each channel, into sums[k][slice][q][channel], still to be added over the slices.
template <int N, int T, int K, typename P>
__device__ __forceinline__ void sum_channels(const float (&s)[K][N], float* tile, float* sums, const GnShape& h, const P& p) {
    const int wide = h.nv * N, pairs = h.Q * wide;
    if (p.here) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) tile[k * T * N + (p.q * h.R + p.r) * wide + p.v * N + e] = s[k][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < h.slices * pairs; i += T) {
        const int j = i / pairs, pair = i - j * pairs, q = pair / wide;
        const int at = q * h.R * wide + (pair - q * wide);
        float t[K] = {};
#pragma unroll 4
        for (int r = j; r < h.R; r += h.slices) {
#pragma unroll
            for (int k = 0; k < K; ++k) t[k] += tile[k * T * N + at + r * wide];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) sums[k * h.slices * pairs + i] = t[k];
    }
    __syncthreads();
}

// A sum over a team of `lanes` consecutive threads (a power of 2), in all of them.
template <int K>
__device__ __forceinline__ void sum_lanes(float (&s)[K], int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] += __shfl_xor(s[k], o, 64);
    }
}

// Sums of K values over each sample's groups, into res[k * Q * sg + q * sg + g].  WHOLE: a thread has one value of its
// vector; otherwise one for each channel of it, which are added over the rows first.
template <bool WHOLE, int N, int T, int K>
__device__ __forceinline__ void sum_groups(const float (&x)[K][WHOLE ? 1 : N], float* tile, float* res, const GnShape& h,
                                           const Place<WHOLE, N>& p) {
    const int j = threadIdx.x & (h.lanes - 1), all = h.Q * h.sg, step = T / h.lanes;
    if constexpr (WHOLE) {
        const int nvg = h.sg == 1 ? h.nv : h.cg / N, length = h.R * nvg;
        if (p.here) {
            const int g = h.sg == 1 ? 0 : p.v / nvg;
#pragma unroll
            for (int k = 0; k < K; ++k) tile[k * T + (p.q * h.sg + g) * length + p.r * nvg + p.v - g * nvg] = x[k][0];
        }
        __syncthreads();
        for (int vg = threadIdx.x / h.lanes; vg < all; vg += step) {
            float s[K] = {};
#pragma unroll 4
            for (int i = j; i < length; i += h.lanes) {
#pragma unroll
                for (int k = 0; k < K; ++k) s[k] += tile[k * T + vg * length + i];
            }
            sum_lanes(s, h.lanes);
            if (j == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) res[k * all + vg] = s[k];
            }
        }
        __syncthreads();
    } else {
        const int wide = h.nv * N, pairs = h.Q * wide, plane = h.slices * pairs;
        float* sums = tile + K * T * N;
        sum_channels<N, T, K>(x, tile, sums, h, p);
        for (int vg = threadIdx.x / h.lanes; vg < all; vg += step) {
            const int q = vg / h.sg, g = vg - q * h.sg;
            float s[K] = {};
            for (int c = j; c < h.cg; c += h.lanes) {
#pragma unroll 4
                for (int i = 0; i < h.slices; ++i) {
#pragma unroll
                    for (int k = 0; k < K; ++k) s[k] += sums[k * plane + i * pairs + q * wide + g * h.cg + c];
                }
            }
            sum_lanes(s, h.lanes);
            if (j == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) res[k * all + vg] = s[k];
            }
        }
        __syncthreads();
    }
}

// ---- on the host -------------------------------------------------------------

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int gcd_of(int a, int b) { return b ? gcd_of(b, a % b) : a; }
inline int pow2_floor(int64_t x) {
    int p = 1;
    while (2 * (int64_t)p <= x) p *= 2;
    return p;
}

constexpr int kMostGroups = 512;     // of a slab; of a workgroup's samples twice that
constexpr int64_t kMostBlocks = 1 << 20;

inline GnShape shape_of(const GroupNorm& n, int64_t S) {
    GnShape h = {};
    h.C = n.C;
    h.G = n.G;
    h.cg = n.C / n.G;
    h.pieces = 1;
    h.Q = 1;
    h.S = (int32_t)S;
    h.p32 = n.p_dtype == GA_FP32;
    h.act = n.act;
    h.inv_n = (float)(1.0 / ((double)S * h.cg));
    h.ldp = n.ldp;
    return h;
}

inline bool whole_vectors(const GnShape& h, int N) { return h.sg == 1 || h.cg % N == 0; }

// The teams that add the sums, of a workgroup of T threads.
inline void sharing(GnShape& h, int N, int T) {
    const int pairs = h.Q * h.nv * N;
    h.lanes = pow2_floor(T / (h.Q * h.sg));
    if (h.lanes > 64) h.lanes = 64;
    h.slices = T / pairs < 1 ? 1 : T / pairs < h.R ? T / pairs : h.R;
}

// Floats of LDS that sum_groups (K values) takes, and sum_channels.
inline size_t lds_of_groups(const GnShape& h, int N, int T, int K) {
    if (whole_vectors(h, N)) return (size_t)K * T;
    return (size_t)K * ((size_t)T * N + (size_t)h.slices * h.Q * h.nv * N);
}

// Slabs of sg whole groups on workgroups of T threads with V vectors each that hold a sample's slab; false if it does
// not fit.
inline bool lay(GnShape& h, int sg, int N, int T, int V, int64_t samples) {
    h.sg = sg;
    h.nv = (int)ceil_div((int64_t)sg * h.cg, N);
    if (h.nv > T) return false;
    h.R = h.S < T / h.nv ? h.S : T / h.nv;
    if (ceil_div(h.S, h.R) > V) return false;
    h.slabs = (int)ceil_div(h.G, sg);
    // several samples at once where one leaves threads idle, as long as the workgroups fill the chip
    int64_t Q = T / (h.nv * h.R);
    if (Q > 2 * kMostGroups / sg) Q = 2 * kMostGroups / sg;
    const int64_t most = samples * h.slabs / 1024;
    if (Q > most) Q = most;
    h.Q = Q < 1 ? 1 : (int)Q;
    sharing(h, N, T);
    return true;
}

struct TeamSize {
    int T, V;
};

// The narrowest team that holds slabs of whole groups: slabs of at least 64 bytes (a cache line's half) where a
// sample's fit, and of whole vectors where that divides the channels.  -1: none does.
template <int K>
inline int choose(GnShape& h, int N, const TeamSize (&teams)[K], int64_t samples) {
    const int unit = N / gcd_of(h.cg, N);
    int64_t sg = unit;
    while (sg * h.cg < 4 * N && sg < h.G) sg += unit;
    if (sg > h.G) sg = h.G;
    for (;;) {
        if (sg <= kMostGroups) {
            for (int k = 0; k < K; ++k)
                if (lay(h, (int)sg, N, teams[k].T, teams[k].V, samples)) return k;
        }
        if (sg <= 1) return -1;
        sg = sg > unit ? (sg - 1) / unit * unit : sg / 2;
    }
}

// Slabs for images that do not stay in registers: whole groups of at least 128 bytes (a cache line) together, or pieces
// of a group that is wider than T vectors.  Parts of a sample so that `want` workgroups of T threads take N samples,
// each of them at least four rows of its threads.
inline void lay_wide(GnShape& h, int N, int T, int64_t samples, int64_t want) {
    const int nvg = (int)ceil_div(h.cg, N);
    if (nvg > T) {
        h.sg = 1;
        h.pieces = (int)ceil_div(nvg, T);
        h.nv = (int)ceil_div(nvg, h.pieces);
        h.slabs = h.G * h.pieces;
    } else {
        const int unit = N / gcd_of(h.cg, N);
        int64_t sg = unit;
        while (sg * h.cg < 8 * N && sg < h.G) sg += unit;
        while (ceil_div(sg * h.cg, N) > T || sg > kMostGroups) sg -= sg > unit ? unit : 1;
        if (sg > h.G) sg = h.G;
        h.sg = (int)sg;
        h.slabs = (int)ceil_div(h.G, sg);
        h.nv = (int)ceil_div(sg * h.cg, N);
    }
    h.R = h.S < T / h.nv ? h.S : T / h.nv;
    sharing(h, N, T);
    int64_t parts = ceil_div(want, samples * h.slabs);
    const int64_t most = ceil_div(h.S, 4 * (int64_t)h.R), least = ceil_div(h.S, 256 * (int64_t)h.R);
    if (parts > most) parts = most;
    if (parts < least) parts = least;    // a thread adds up at most 256 rows, whose roundings add up too
    h.span = (int)ceil_div(h.S, parts);
    h.parts = (int)ceil_div(h.S, h.span);
}

}  // namespace ga
