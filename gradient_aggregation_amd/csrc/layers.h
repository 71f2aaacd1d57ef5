// Internal host-side declarations of the layer operators: the group-norm and
// router handles and their kernel launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gradagg.h"

namespace ga {

struct GroupNorm {
    int32_t C, G;
    int32_t x_dtype, p_dtype, act;
    int device;
    int32_t backward;
    int32_t ldp;           // stride of a partial row (channels rounded up to 4)
    int32_t rows;          // partial rows of the weight gradients
    float* d_rows;         // [rows][2][ldp], or nullptr
    void* d_records;       // kGnRecords of 16 bytes: partial sums of groups
};

// Partial rows at most, and their bytes.
constexpr int kGnRows = 512;
constexpr int64_t kGnRowBytes = (int64_t)16 << 20;
constexpr int64_t kGnRecords = (int64_t)1 << 20;

struct Images {
    const char* data;
    int64_t ld, sample;    // bytes
};

struct GnArgs {
    int64_t N, S;
    Images x, y;           // y: the output (dx)
    const void *gamma, *beta;
    float* mean;
    float* rstd;
    float eps;
    // backward
    Images dy;
    int32_t workers;
    int64_t per_worker;    // samples of a worker
    void *dgamma, *dbeta;
    int32_t dp_dtype;
};

hipError_t launch_gn_fwd(const GroupNorm& n, const GnArgs& a, hipStream_t s);
hipError_t launch_gn_bwd(const GroupNorm& n, const GnArgs& a, hipStream_t s);

struct Router {
    int32_t E, k, W;
    int32_t x_dtype, normalize, scope;
    int device;
    int32_t rows;          // partial loads: kRouterRows, or a row for each worker
    // one allocation
    double* d_squares;     // [rows] sums of lse^2
    double* d_dots;        // [GA_MAX_EXPERTS] parts of the balance loss
    float* d_probs;        // [rows][E]
    int32_t* d_counts;     // [rows][E]
    int32_t* d_tokens;     // [rows]
    uint32_t* d_done;      // [2] counts of workgroups that have ended; 0 between calls
};

constexpr int kRouterRows = 256;

struct RouteArgs {
    int64_t T, per_worker;    // tokens, tokens of a worker
    const char* x;
    int64_t ldx;              // bytes
    const uint8_t* mask;
    int32_t select;
    ga_routing r;
    ga_load load;
    int32_t with_load;
    // backward
    char* dx;
    int64_t ldd;
    const float *slope, *dgates;
    float balance, z;
};

hipError_t launch_router_fwd(const Router& r, const RouteArgs& a, hipStream_t s);
hipError_t launch_router_bwd(const Router& r, const RouteArgs& a, hipStream_t s);

}  // namespace ga
