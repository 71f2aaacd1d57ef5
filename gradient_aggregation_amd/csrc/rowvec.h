// Vectors of consecutive elements of a row (128 bits), at any alignment and past
// neither end of the row, as the normalisations read, shift and write them.
#pragma once

#include "elements.h"

namespace ga {

template <int X>
constexpr int kVec = 16 / kSize<X>;     // elements of a 128-bit vector

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

// Drops the first s elements of a vector: the others move to its front, zeros follow them.
template <int X, int N>
__device__ __forceinline__ void drop_front(Raw<X, N>& r, uint32_t s) {
    static_assert(Raw<X, N>::WORDS == 4, "a 128-bit vector");
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

// Where all vectors start at multiples of N.
template <int X, int N>
__device__ __forceinline__ void into_place(Raw<X, N>& r, int32_t c, int32_t dim) {
    if (dim < N || dim % N == 0) return;
    const int past = c + N - dim;
    drop_front(r, past > 0 && past < N ? (uint32_t)past : 0u);   // elements to drop
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

// An element of a weight gradient, rounded to its type.
__device__ __forceinline__ void store_param(void* out, int32_t dtype, int64_t i, float x) {
    if (dtype == kF32) static_cast<float*>(out)[i] = x;
    else if (dtype == kF16) store_one<kF16>(reinterpret_cast<uint64_t>(out) + (uint64_t)i * 2, x);
    else store_one<kB16>(reinterpret_cast<uint64_t>(out) + (uint64_t)i * 2, x);
}

}  // namespace ga
