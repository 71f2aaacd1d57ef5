// Internal host-side declarations of the training-step operators: the AdamW
// and layer-norm handles and their kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gradagg.h"

namespace ga {

// A wavefront takes kTile consecutive elements of the fused row.
constexpr int kTile = 512;

// A tile and where its gradients are: the layer its first element lies in, and
// that layer's start in the fused row.  The table holds the tiles that are not
// whole first, the others in order: those few take several times as long and
// would end last.
struct TileRec {
    int64_t tile;       // elements [tile * kTile, (tile + 1) * kTile) of the fused row
    int64_t start;      // first element of the layer
    uint32_t layer;
    uint32_t flags;     // kTileWhole | kTileDecay | layers after this one in the tile << kTileSpanShift
};
constexpr uint32_t kTileWhole = 1u;   // all kTile elements exist and lie in this layer
constexpr uint32_t kTileDecay = 2u;   // the layer's weights decay
constexpr int kTileSpanShift = 16;    // a tile of 512 elements holds at most 512 layers

// Workgroups of the norm pass at most: its partial sums are one binary64 each.
constexpr int kNormBlocks = 2048;

struct Adamw {
    int32_t W, L, dtype, bits;
    int64_t P, n_tiles;
    int device;
    // one allocation: tiles [n_tiles], offsets [L+1], decay flags [L]
    TileRec* d_tiles;
    int64_t* d_offsets;
    uint8_t* d_decay;
    double* d_partials;   // [kNormBlocks], then d_done
    uint32_t* d_done;     // workgroups of a norm call that have ended; 0 between calls
};

struct StepArgs {
    float lr_t, beta1, beta2, c1, c2, eps, rbc2, keep;   // see k_adamw
    uint32_t seed;
    int32_t m_rounding;   // of 8-bit codes: a ga_rounding
    float* w;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    const ga_clip* clip;
    void* copy;
    int32_t copy_dtype;
};

hipError_t launch_grad_norm(const Adamw& o, const uint64_t* layer_ptrs, float max_norm, float* grad, ga_clip* clip,
                            hipStream_t s);
hipError_t launch_adamw(const Adamw& o, const uint64_t* layer_ptrs, const StepArgs& a, hipStream_t s);

// Partial rows of the weight gradients at most (all groups together).
constexpr int kLnParts = 256;

struct LayerNorm {
    int64_t dim, ldp;      // ldp: stride of a partial row (dim rounded up to 4)
    int32_t x_dtype, p_dtype;
    int device;
    float* d_parts;        // [kLnParts][2][ldp], then d_done; or nullptr
    uint32_t* d_done;      // [kLnParts] a group's workgroups that have ended; 0 between calls
};

struct LnFwd {
    const char *x, *res;
    char *y, *sum;
    int64_t ldx, ldr, ldy, lds;   // bytes
    const void *gamma, *beta;
    float *mean, *rstd;
    float eps;
    int64_t rows;
};

struct LnBwd {
    const char *dy, *x, *dsum;
    char* dx;
    int64_t ldy, ldx, lds, ldd;   // bytes
    const void* gamma;
    const float *mean, *rstd;
    int64_t rows, group_rows;
    int32_t groups;
    void *dgamma, *dbeta;
    int32_t dp_dtype;
};

hipError_t launch_ln_fwd(const LayerNorm& n, const LnFwd& a, hipStream_t s);
hipError_t launch_ln_bwd(const LayerNorm& n, const LnBwd& a, hipStream_t s);
// Adds each group's `parts` partial rows of two weight gradients, [groups][parts][2][ldp], in a fixed order; parts = 0
// writes zeros.
hipError_t launch_params_end(const float* in, int64_t dim, int64_t ldp, int32_t parts, int32_t groups, void* dgamma,
                             void* dbeta, int32_t dp_dtype, hipStream_t s);

}  // namespace ga
