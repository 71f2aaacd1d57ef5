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

// A lane's 8 elements are two groups of 4: with SPLIT the groups lie 256
// elements apart, so that a wavefront's 128-bit accesses to binary32 vectors
// are one contiguous run; without it they are neighbours, so that 8 16-bit
// elements are one 128-bit access.
template <bool SPLIT>
__device__ __forceinline__ int64_t group_at(int64_t tile, int lane, int q) {
    return tile * kTile + (SPLIT ? q * 256 + lane * 4 : lane * 8 + q * 4);
}

template <int T, bool SPLIT>
__device__ __forceinline__ void load_leaf8(Raw<T, 8>& x, uint64_t addr) {
    if constexpr (SPLIT) {
        Raw<T, 4> a, b;
        a.template load<true>(addr);
        b.template load<true>(addr + 256 * kSize<T>);
#pragma unroll
        for (int j = 0; j < Raw<T, 4>::WORDS; ++j) {
            x.w[j] = a.w[j];
            x.w[Raw<T, 4>::WORDS + j] = b.w[j];
        }
    } else {
        x.template load<true>(addr);
    }
}

// Leaves in flight per lane and levels of the tree for W workers, W < 2^LEV.
template <int LEV>
constexpr int kInFlight = LEV <= 1 ? 1 : LEV <= 3 ? 4 : LEV <= 8 ? 8 : 4;

// g[4q + e] = the mean gradient of element group_at(q) + e (0 past P); bit
// 4q + e of dmask: the element's layer decays.  All 64 lanes take part.
template <int T, int LEV, bool SPLIT>
__device__ __forceinline__ void mean_grad(const GradArgs& a, int64_t tile, const TileRec& rec, int lane, float (&g)[8],
                                          uint32_t& dmask) {
    constexpr int SZ = kSize<T>;
    constexpr int U = kInFlight<LEV>;
    TreeAcc<LEV, 8> tree;
    uint32_t cnt = 0;
    if (rec.flags & kTileWhole) {
        dmask = rec.flags & kTileDecay ? 0xffu : 0u;
        const uint64_t at = (uint64_t)((group_at<SPLIT>(tile, lane, 0) - rec.start) * SZ);
        if constexpr (LEV == 1) {
            Raw<T, 8> x;
            load_leaf8<T, SPLIT>(x, a.ptrs[rec.layer] + at);
            x.widen(g);
            return;
        } else {
            for (int32_t g0 = 0; g0 < a.W; g0 += 64) {
                // lane l holds worker (g0 + l)'s address, read out lane by lane
                const int32_t gn = a.W - g0 < 64 ? a.W - g0 : 64;
                const uint64_t mine = lane < gn ? a.ptrs[(int64_t)(g0 + lane) * a.L + rec.layer] : 0ull;
                const int lo = (int)(uint32_t)mine, hi = (int)(uint32_t)(mine >> 32);
                for (int32_t u0 = 0; u0 < gn; u0 += U) {
                    Raw<T, 8> x[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (u0 + u < gn) {
                            const uint64_t base = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, u0 + u) << 32) |
                                                  (uint32_t)__builtin_amdgcn_readlane(lo, u0 + u);
                            load_leaf8<T, SPLIT>(x[u], base + at);
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
        }
    } else {
        // The tile straddles a layer boundary or holds the tail: each group
        // resolves its own layer; one whose 4 elements lie in one layer is a
        // vector load, the others go element by element.
        constexpr int V = U < 4 ? U : 4;
        int64_t i[2], start[2];
        int32_t layer[2];
        bool vec[2], part[2];
        dmask = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            i[q] = group_at<SPLIT>(tile, lane, q);
            int32_t lo = (int32_t)rec.layer, hi = a.L - 1;
            while (lo < hi) {
                const int32_t mid = (lo + hi) >> 1;
                if (a.offsets[mid + 1] <= i[q]) lo = mid + 1;
                else hi = mid;
            }
            layer[q] = lo;
            start[q] = a.offsets[lo];
            vec[q] = i[q] + 4 <= a.offsets[lo + 1];
            part[q] = !vec[q] && i[q] < a.P;
            if (vec[q]) {
                dmask |= a.decay[lo] ? 0xfu << (4 * q) : 0u;
            } else if (part[q]) {
                int32_t l = lo;
                for (int e = 0; e < 4 && i[q] + e < a.P; ++e) {
                    while (a.offsets[l + 1] <= i[q] + e) ++l;
                    dmask |= a.decay[l] ? 1u << (4 * q + e) : 0u;
                }
            }
        }
        for (int32_t w0 = 0; w0 < a.W; w0 += V) {
            float f[V][8];
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[u][e] = 0.f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (vec[q]) {
                    uint64_t base[V];
                    Raw<T, 4> x[V];
#pragma unroll
                    for (int u = 0; u < V; ++u)
                        base[u] = a.ptrs[(int64_t)(w0 + u < a.W ? w0 + u : a.W - 1) * a.L + layer[q]];
#pragma unroll
                    for (int u = 0; u < V; ++u) x[u].load(base[u] + (uint64_t)((i[q] - start[q]) * SZ));
#pragma unroll
                    for (int u = 0; u < V; ++u) {
                        float h[4];
                        x[u].widen(h);
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[u][4 * q + e] = h[e];
                    }
                } else if (part[q]) {
                    int32_t l = layer[q];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (i[q] + e < a.P) {
                            while (a.offsets[l + 1] <= i[q] + e) ++l;
                            const uint64_t at = (uint64_t)((i[q] + e - a.offsets[l]) * SZ);
#pragma unroll
                            for (int u = 0; u < V; ++u)
                                f[u][4 * q + e] =
                                    load_one<T>(a.ptrs[(int64_t)(w0 + u < a.W ? w0 + u : a.W - 1) * a.L + l] + at);
                        }
                    }
                }
            }
            if constexpr (LEV == 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = f[0][e];
                return;
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
    }
    if constexpr (LEV > 1) {
        float s[8];
        tree.result((uint32_t)a.W, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = s[e] * a.inv_w;
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
