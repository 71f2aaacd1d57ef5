// What both passes of the group norm share: how workgroups lie on channels-last
// images, the activations, and sums over a group's or a channel's values.
#pragma once

#include <type_traits>

#include "layers.h"
#include "rowvec.h"

namespace ga {

// Division of numbers below 2^16 by one of them, by multiplication: x * ceil(2^32 / d) is off by less than x.
struct Divisor {
    uint32_t m;            // 0: by 1

    __device__ __forceinline__ int of(int x) const { return m ? (int)__umulhi((uint32_t)x, m) : x; }
};

// How groups lie on vectors: each vector in one group; over the border of at most two (groups of N channels or more);
// or in more.
enum GnMode { kWhole = 0, kSpan = 1, kMany = 2 };

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
    int32_t stream;        // stores pass the caches by
    int32_t parts;         // images that do not stay in registers: parts of a sample, each of `chunks` whole chunks (see
    int32_t chunks, more;  // PartOf), the first `more` of them one more, the next one `rest` positions more
    int32_t rest;
    int32_t spread;        // of the threads that add a group's sums, those that share a row (a power of 2)
    int32_t rows;          // backward: partial rows of the weight gradients of a worker
    int32_t ldp;           // their stride
    float inv_n;           // 1 / (S * cg)
    double inv_count;      // the same
    Divisor by_cg, by_nv, by_place, by_pairs, by_wide, by_R;     // by cg, nv, nv * R, Q * nv * N, nv * N, R
};

// Consecutive workgroups go to the 8 XCDs in turn: those of an XCD take consecutive work, so that slabs beside each
// other, which share cache lines, share a cache.
__device__ __forceinline__ uint32_t xcd_block(uint32_t n) {
    const uint32_t b = blockIdx.x, x = b & 7u, per = n >> 3, rest = n & 7u;
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

// dy -> dz, z = xh * gamma + beta.  silu's derivative: s + z s (1 - s).
template <int N>
__device__ __forceinline__ void through_activation(float (&dy)[N], const float (&xh)[N], const float (&gamma)[N],
                                                   const float (&beta)[N], int32_t act) {
    if (act == GA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float z = fmaf(xh[e], gamma[e], beta[e]), s = sigmoid(z);
            dy[e] *= fmaf(z, fmaf(-s, s, s), s);
        }
    } else if (act == GA_ACT_RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) dy[e] = fmaf(xh[e], gamma[e], beta[e]) <= 0.f ? 0.f : dy[e];
    }
}

// The slab's channels, and a thread's place: row r of sample q, vector v, whose first channel is c (of all).
template <int MODE, int N>
struct Place {
    int g0, c0, channels;  // first group and channel (of all), channels of the slab
    bool ragged;           // some vector of the workgroup ends within the slab's last vector
    int q, r, v, c;
    int left;              // elements of the vector within the slab (none: 0 or less)
    uint32_t past;         // elements that its loads are moved to the front by, to end with the row
    int from;              // the channel that they start at
    bool here;             // the thread has a place
    int g, border;         // group (of the slab) of the first element; elements of the vector in it

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
        ragged = channels % N != 0;
        q = h.by_place.of(t);
        r = h.by_nv.of(t - q * per);
        v = t - q * per - r * h.nv;
        here = q < h.Q;
        c = c0 + v * N;
        left = channels - v * N;
        from = c + N > h.C && h.C >= N ? h.C - N : c;
        past = c < h.C ? (uint32_t)(c - from) : 0u;
        g = h.sg == 1 ? 0 : h.by_cg.of(v * N);
        g = g < h.sg ? g : h.sg - 1;
        border = MODE == kWhole || g == h.sg - 1 ? N : (g + 1) * h.cg - v * N;
    }

    // Group (of the slab) of element e.
    __device__ __forceinline__ int group(const GnShape& h, int e) const {
        if (MODE == kWhole) return g;
        if (MODE == kSpan) return g + (e >= border ? 1 : 0);
        const int of = h.by_cg.of(v * N + e);
        return of < h.sg ? of : h.sg - 1;
    }
};

// A vector of the row at `row`.  TINY: rows shorter than a vector, element by element.  Otherwise every thread reads
// within the row, and one that has no place, or only a part of a vector, some elements too many.
template <int X, bool TINY, int MODE, int N>
__device__ __forceinline__ void load_vector(Raw<X, N>& r, uint64_t row, const GnShape& h, const Place<MODE, N>& p) {
    if constexpr (TINY) load_part(r, row, p.c, h.C);
    else r.load(row + (uint64_t)(p.from * kSize<X>));
}

template <int X, bool RAGGED, int N>
__device__ __forceinline__ void into_row(Raw<X, N>& r, uint32_t past) {
    if (RAGGED && past) drop_front(r, past);
}

template <int X, bool RAGGED, bool STREAM, int MODE, int N>
__device__ __forceinline__ void store_vector(const float (&f)[N], uint64_t row, const Place<MODE, N>& p) {
    if constexpr (RAGGED) {
        store_part<X>(f, row, p.c, p.c + (p.left < N ? p.left : N));
    } else {
        Raw<X, N> r;
        r.narrow(f);
        r.template store<STREAM>(row + (uint64_t)p.c * kSize<X>);
    }
}

// Calls f(std::bool_constant) with whether the workgroup's slab is ragged.
template <typename F>
__device__ __forceinline__ void if_ragged(bool ragged, F f) {
    if (ragged) f(std::integral_constant<bool, true>{});
    else f(std::integral_constant<bool, false>{});
}

constexpr int kAhead = 2;      // vectors of a thread on their way together where images do not stay in registers

// There, part `part` of sample n takes every h.parts-th chunk of kAhead * R positions, so that the workgroups go over
// the images side by side.
struct PartOf {
    int64_t n;
    int part, slab;

    __device__ __forceinline__ PartOf(const GnShape& h, uint32_t id) {
        slab = (int)(id % (uint32_t)h.slabs);
        const uint32_t rest = id / (uint32_t)h.slabs;
        part = (int)(rest % (uint32_t)h.parts);
        n = rest / (uint32_t)h.parts;
    }
};

// Positions of a part, and a row's: `full` chunks of kAhead, then `tail` of an incomplete one.
__device__ __forceinline__ int positions_of(const GnShape& h, int part) {
    return (h.chunks + (part < h.more ? 1 : 0)) * kAhead * h.R + (part == h.more ? h.rest : 0);
}

struct Rows {
    int64_t first;
    int full, tail;

    __device__ __forceinline__ Rows(const GnShape& h, int part, int r) {
        first = (int64_t)part * kAhead * h.R + r;
        full = h.chunks + (part < h.more ? 1 : 0);
        tail = part == h.more && r < h.rest ? h.by_R.of(h.rest - r + h.R - 1) : 0;
    }
};

// Sums over the R rows of each channel, into sums[k][slice][q][channel], still to be added over the slices.
template <int N, int T, int K, typename P>
__device__ __forceinline__ void sum_channels(const float (&s)[K][N], float* tile, float* sums, const GnShape& h, const P& p) {
    const int wide = h.nv * N, pairs = h.Q * wide;
    if (p.here) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f32x4* to = reinterpret_cast<f32x4*>(tile + k * T * N + (p.q * h.R + p.r) * wide + p.v * N);
#pragma unroll
            for (int e = 0; e < N; e += 4) to[e / 4] = f32x4{s[k][e], s[k][e + 1], s[k][e + 2], s[k][e + 3]};
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < h.slices * pairs; i += T) {
        const int j = h.by_pairs.of(i), pair = i - j * pairs, q = h.by_wide.of(pair);
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
    const auto add = [](float x, uint32_t y) { return x + __uint_as_float(y); };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float x = s[k];
        if (lanes >= 2) x = add(x, lane_move<0xb1>(__float_as_uint(x)));      // xor 1
        if (lanes >= 4) x = add(x, lane_move<0x4e>(__float_as_uint(x)));      // xor 2
        if (lanes >= 8) x = add(x, lane_move<0x141>(__float_as_uint(x)));     // mirror within 8
        if (lanes >= 16) x = add(x, lane_move<0x140>(__float_as_uint(x)));    // mirror within 16
        if (lanes >= 32) {
            const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
            x = add(__uint_as_float(r[0]), r[1]);
        }
        if (lanes >= 64) {
            const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
            x = add(__uint_as_float(r[0]), r[1]);
        }
        s[k] = x;
    }
}

// Sums over each sample's groups, of a value for each channel of a thread's vector, into res[q * sg + g].
template <int N, int T, typename P>
__device__ __forceinline__ void sum_groups(const float (&x)[1][N], float* tile, float* res, const GnShape& h, const P& p) {
    const int j = threadIdx.x & (h.lanes - 1), all = h.Q * h.sg, wide = h.nv * N, pairs = h.Q * wide;
    float* sums = tile + T * N;
    sum_channels<N, T, 1>(x, tile, sums, h, p);
    for (int vg = threadIdx.x / h.lanes; vg < all; vg += T / h.lanes) {
        const int q = h.Q == 1 ? 0 : vg / h.sg, g = vg - q * h.sg;
        float s[1] = {0.f};
        for (int c = j; c < h.cg; c += h.lanes) {
#pragma unroll 4
            for (int i = 0; i < h.slices; ++i) s[0] += sums[i * pairs + q * wide + g * h.cg + c];
        }
        sum_lanes(s, h.lanes);
        if (j == 0) res[vg] = s[0];
    }
    __syncthreads();
}

// ---- on the host -------------------------------------------------------------

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int gcd_of(int a, int b) { return b ? gcd_of(b, a % b) : a; }
inline int pow2_floor(int64_t x) {
    int p = 1;
    while (2 * (int64_t)p <= x) p *= 2;
    return p;
}

constexpr int kMostSums = 1024;       // groups of a workgroup's samples together; a slab has 64 at most (see choose, lay_wide)
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
    h.inv_count = 1.0 / ((double)S * h.cg);
    h.inv_n = (float)h.inv_count;
    h.ldp = n.ldp;
    return h;
}

inline GnMode mode_of(const GnShape& h, int N) {
    return h.sg == 1 || h.cg % N == 0 ? kWhole : h.cg >= N ? kSpan : kMany;
}

// Calls f with the mode as a constant.
template <typename F>
void with_mode(GnMode m, F f) {
    if (m == kWhole) f(std::integral_constant<int, kWhole>{});
    else if (m == kSpan) f(std::integral_constant<int, kSpan>{});
    else f(std::integral_constant<int, kMany>{});
}

inline Divisor divisor(int64_t d) { return {d > 1 ? (uint32_t)((((uint64_t)1 << 32) + (uint64_t)d - 1) / (uint64_t)d) : 0u}; }

// The teams that add the sums, of a workgroup of T threads.
inline void sharing(GnShape& h, int N, int T) {
    const int pairs = h.Q * h.nv * N;
    h.by_cg = divisor(h.cg);
    h.by_nv = divisor(h.nv);
    h.by_place = divisor((int64_t)h.nv * h.R);
    h.by_pairs = divisor(pairs);
    h.by_wide = divisor(h.nv * N);
    h.by_R = divisor(h.R);
    h.lanes = pow2_floor(T / (h.Q * h.sg));
    if (h.lanes > 64) h.lanes = 64;
    const int64_t vectors = h.sg == 1 ? h.nv : h.cg / N + 2;      // of a group at most
    h.spread = 1;
    while (h.spread < h.lanes && h.spread < vectors) h.spread *= 2;
    h.slices = T / pairs < 1 ? 1 : T / pairs < h.R ? T / pairs : h.R;
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
    if (Q > kMostSums / sg) Q = kMostSums / sg;
    const int64_t most = samples * h.slabs / 1024;
    if (Q > most) Q = most;
    h.Q = Q < 1 ? 1 : (int)Q;
    sharing(h, N, T);
    return true;
}

struct TeamSize {
    int T, V;
};

// The narrowest team that holds slabs of whole groups of at least 64 bytes (half a cache line), of whole vectors where
// that divides the channels; -1 where none does, or where two kernels over wide slabs are faster.  One after the other,
// bf16, 32 groups, us, held in registers against not: 16 x 256 x 256 forward 8.3, 11.3 and backward 12.7, 15.5; 16 x 1024 x
// 256 10.4, 11.1 and 22.4, 19.4; 16 x 1024 x 320 (slabs of 80 bytes) 17.3, 14.2 and 34.9, 26.5; 64 x 256 x 640 21.9, 17.0
// and 46.4, 34.0.  So the last team, `half`, takes slabs of whole half lines only, and large batches of others go the
// other way.
template <int K>
inline int choose(GnShape& h, int N, const TeamSize (&teams)[K], int half, int64_t samples) {
    if (h.C < N) return -1;
    const int unit = N / gcd_of(h.cg, N);
    int64_t sg = unit;
    while (sg * h.cg < 4 * N && sg < h.G) sg += unit;
    if (sg > h.G) sg = h.G;
    const bool halves = sg * h.cg % (4 * N) == 0;
    if (!halves && samples * h.S * h.C > (int64_t)(8 << 20) / 16 * N) return -1;
    for (int k = 0; k < K; ++k)
        if ((k != half || halves) && lay(h, (int)sg, N, teams[k].T, teams[k].V, samples)) return k;
    return -1;
}

// Slabs for images that do not stay in registers: pieces of a group that is wider than T vectors; else groups that
// together are a multiple of a cache line of 128 bytes, where that is less than eight of them, else all of a short row, else
// at least a line.  Parts of a sample so that 512 workgroups take all samples, each at least a chunk.
inline void lay_wide(GnShape& h, int N, int T, int64_t samples) {
    const int nvg = (int)ceil_div(h.cg, N), line = 8 * N;
    if (nvg > T) {
        h.sg = 1;
        h.pieces = (int)ceil_div(nvg, T);
        h.nv = (int)ceil_div(nvg, h.pieces);
        h.slabs = h.G * h.pieces;
    } else {
        int64_t sg = line / gcd_of(h.cg, line);
        if (sg > h.G || sg * h.cg > 8 * line) {
            const int unit = N / gcd_of(h.cg, N);
            sg = h.C <= 4 * line ? h.G : unit;
            while (sg * h.cg < line && sg < h.G) sg += unit;
            while (ceil_div(sg * h.cg, N) > T) sg -= sg > unit ? unit : 1;
        }
        if (sg > h.G) sg = h.G;
        h.sg = (int)sg;
        h.slabs = (int)ceil_div(h.G, sg);
        h.nv = (int)ceil_div(sg * h.cg, N);
    }
    h.R = h.S < T / h.nv ? h.S : T / h.nv;
    sharing(h, N, T);
    // 512 workgroups of 256 threads: with 1024 the prologues cost more than they hide (4 x 65536 x 256 bf16 forward: 68 us,
    // 71), with 256 too little is on its way (87); of 512 or 1024 threads 77
    int64_t parts = ceil_div(512, samples * h.slabs);
    const int64_t most = ceil_div(h.S, kAhead * (int64_t)h.R), least = ceil_div(h.S, 256 * (int64_t)h.R);
    if (parts > most) parts = most;
    // a thread adds up at most some 256 rows, whose roundings add up too, unless so many groups leave no room to (images of
    // 17 GB and more)
    if (parts < least) parts = least;
    const int64_t room = kGnRecords / ((int64_t)h.pieces * h.G);
    if (parts > room) parts = room;
    h.parts = (int)parts;
    const int64_t chunk = kAhead * (int64_t)h.R, all = h.S / chunk;
    h.chunks = (int)(all / parts);
    h.more = (int)(all % parts);
    h.rest = (int)(h.S - all * chunk);
}

// Whether a workgroup writes whole cache lines of 128 bytes, so that its stores may pass the caches by: slabs of whole
// lines, or whole rows that follow one another.
inline bool whole_lines(const GnShape& h, const Images& m, int64_t size) {
    if (h.pieces != 1) return false;
    if (h.slabs == 1 && m.ld == h.C * size) return true;
    return h.sg * h.cg * size % 128 == 0 && h.C * size % 128 == 0 && m.ld % 128 == 0 && m.sample % 128 == 0 &&
           (reinterpret_cast<uintptr_t>(m.data) & 127) == 0;
}

}  // namespace ga
