// The mean gradient of a tile of the fused row, read straight from the
// workers' per-layer tensors: the leaves of the fixed tree (tree.h), 512
// consecutive elements per wavefront, 8 per lane.
#pragma once

#include <type_traits>

#include "elements.h"
#include "training.h"
#include "tree.h"

namespace ga {

struct GradArgs {
    const uint64_t* __restrict__ ptrs;      // [W][L] tensor addresses
    const TileRec* __restrict__ tiles;
    const int64_t* __restrict__ offsets;    // [L+1]
    const uint8_t* __restrict__ decay;      // [L]
    int32_t L, W;
    int64_t P;
    float inv_w;
};

// A lane's 8 elements are two groups of 4, 256 elements apart: each of a
// wavefront's accesses, to a gradient as to a binary32 vector, is one run with
// no gaps.  (With the groups side by side a wavefront's binary32 access is
// every other 16 bytes of its run, each 128-byte line is asked for twice, and
// streaming hints make the second time a miss: the update of 7.6M parameters
// took 94 us that way.)
__device__ __forceinline__ int64_t group_at(int64_t tile, int lane, int q) { return tile * kTile + q * 256 + lane * 4; }

// Workers whose leaves a lane has in flight (W < 2^LEV).  61M parameters of 16
// workers: 573 us with 4, 582 with 8 at the same occupancy, 788 with 16, whose
// registers leave room for fewer wavefronts.
template <int LEV>
constexpr int kInFlight = LEV == 1 ? 1 : 4;

template <int T>
struct Leaf {
    Raw<T, 4> q0, q1;
    __device__ __forceinline__ void load(uint64_t base, uint32_t at) {
        q0.template load<true>(base + at);
        q1.template load<true>(base + at + 256 * kSize<T>);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        float a[4], b[4];
        q0.widen(a);
        q1.widen(b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = a[e];
            f[4 + e] = b[e];
        }
    }
};

// g[4q + e] = the mean gradient of element group_at(q) + e of a tile that lies
// in one layer.  All 64 lanes take part; tile and rec are the wavefront's.
template <int T, int LEV>
__device__ __forceinline__ void mean_grad_whole(const GradArgs& a, int64_t tile, const TileRec& rec, int lane,
                                                float (&g)[8]) {
    const uint64_t in_layer = (uint64_t)(tile * kTile - rec.start) * kSize<T>;
    const uint32_t at = (uint32_t)lane * 4 * kSize<T>;
    if constexpr (LEV == 1) {
        Leaf<T> x;
        x.load(a.ptrs[rec.layer] + in_layer, at);
        x.widen(g);
    } else {
        constexpr int U = kInFlight<LEV>;
        TreeAcc<LEV, 8> tree;
        uint32_t cnt = 0;
        for (int32_t g0 = 0; g0 < a.W; g0 += 64) {
            // lane l holds worker (g0 + l)'s address, read out lane by lane
            const int32_t gn = a.W - g0 < 64 ? a.W - g0 : 64;
            const uint64_t mine = lane < gn ? a.ptrs[(int64_t)(g0 + lane) * a.L + rec.layer] : 0ull;
            const int lo = (int)(uint32_t)mine, hi = (int)(uint32_t)(mine >> 32);
            for (int32_t u0 = 0; u0 < gn; u0 += U) {
                Leaf<T> x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u0 + u < gn) {
                        const uint64_t base = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, u0 + u) << 32) |
                                              (uint32_t)__builtin_amdgcn_readlane(lo, u0 + u);
                        x[u].load(base + in_layer, at);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u0 + u < gn) {
                        float f[8];
                        x[u].widen(f);
                        tree.push(f, cnt);
                        ++cnt;
                    }
                }
            }
        }
        float s[8];
        tree.result((uint32_t)a.W, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = s[e] * a.inv_w;
    }
}

// The same of a tile that straddles a layer boundary or holds the tail (0 past
// P); bit 4q + e of dmask: the element's layer decays.  Each group of 4 resolves
// its own layer, between those of the tile's first and last element; one whose
// elements lie in one layer is a vector load, of the others each element's
// place is found once, before the workers' loop.
template <int T, int LEV>
__device__ __forceinline__ void mean_grad_part(const GradArgs& a, int64_t tile, const TileRec& rec, int lane,
                                               float (&g)[8], uint32_t& dmask) {
    constexpr int SZ = kSize<T>;
    constexpr int V = kInFlight<LEV>;
    dmask = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t i = group_at(tile, lane, q);
        int32_t lo = (int32_t)rec.layer, hi = lo + (int32_t)(rec.flags >> kTileSpanShift);
        while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (a.offsets[mid + 1] <= i) lo = mid + 1;
            else hi = mid;
        }
        const int64_t start = a.offsets[lo];
        const bool vec = i + 4 <= a.offsets[lo + 1], part = !vec && i < a.P;
        int32_t layer[4];
        uint64_t at[4];
        if (vec) {
            dmask |= a.decay[lo] ? 0xfu << (4 * q) : 0u;
        } else if (part) {
            int32_t l = lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (i + e < a.P) {
                    while (a.offsets[l + 1] <= i + e) ++l;
                    dmask |= a.decay[l] ? 1u << (4 * q + e) : 0u;
                }
                // past P: the last element again, set to 0 below
                const int64_t in = i + e < a.P ? i + e : a.P - 1;
                layer[e] = l;
                at[e] = (uint64_t)((in - a.offsets[l]) * SZ);
            }
        }
        TreeAcc<LEV, 4> tree;
        uint32_t cnt = 0;
        for (int32_t w0 = 0; w0 < a.W; w0 += V) {
            float f[V][4];
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) f[u][e] = 0.f;
            // workers past W are read as the last one and not added
            if (vec) {
                uint64_t base[V];
                Raw<T, 4> x[V];
#pragma unroll
                for (int u = 0; u < V; ++u) base[u] = a.ptrs[(int64_t)(w0 + u < a.W ? w0 + u : a.W - 1) * a.L + lo];
#pragma unroll
                for (int u = 0; u < V; ++u) x[u].load(base[u] + (uint64_t)((i - start) * SZ));
#pragma unroll
                for (int u = 0; u < V; ++u) x[u].widen(f[u]);
            } else if (part) {
                uint64_t base[V][4];
#pragma unroll
                for (int u = 0; u < V; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        base[u][e] = a.ptrs[(int64_t)(w0 + u < a.W ? w0 + u : a.W - 1) * a.L + layer[e]];
#pragma unroll
                for (int u = 0; u < V; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[u][e] = load_one<T>(base[u][e] + at[e]);
#pragma unroll
                for (int u = 0; u < V; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[u][e] = i + e < a.P ? f[u][e] : 0.f;
            }
            if constexpr (LEV == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) g[4 * q + e] = f[0][e];
            } else {
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    if (w0 + u < a.W) {
                        tree.push(f[u], cnt);
                        ++cnt;
                    }
                }
            }
        }
        if constexpr (LEV > 1) {
            float s[4];
            tree.result((uint32_t)a.W, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[4 * q + e] = s[e] * a.inv_w;
        }
    }
}

// Calls f with the tree depth that serves W workers, as a constant.
template <typename F>
hipError_t with_levels(int32_t W, F f) {
    if (W == 1) return f(std::integral_constant<int, 1>{});
    if (W < 8) return f(std::integral_constant<int, 3>{});
    if (W < 32) return f(std::integral_constant<int, 5>{});
    if (W < 256) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 11>{});
}

inline GradArgs grad_args(const Adamw& o, const uint64_t* layer_ptrs) {
    GradArgs a;
    a.ptrs = layer_ptrs;
    a.tiles = o.d_tiles;
    a.offsets = o.d_offsets;
    a.decay = o.d_decay;
    a.L = o.L;
    a.W = o.W;
    a.P = o.P;
    a.inv_w = (float)(1.0 / (double)o.W);
    return a;
}

}  // namespace ga
