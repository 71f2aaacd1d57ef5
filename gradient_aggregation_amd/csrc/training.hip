// C ABI of the training-step operators: handles, argument validation and
// launches.  The operations are specified in include/gradagg.h.
#include "training.h"

#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "plan.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

ga_status invalid(const char* msg) { return ga::api_fail(GA_ERR_INVALID, msg); }
ga_status misaligned(const char* msg) { return ga::api_fail(GA_ERR_ALIGN, msg); }

ga_status launched(hipError_t e) {
    return e == hipSuccess ? ga::api_ok() : ga::api_fail(GA_ERR_DEVICE, hipGetErrorString(e));
}

// The calling thread's current device must be the handle's.
ga_status on_device(int device) {
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return ga::api_fail(GA_ERR_DEVICE, hipGetErrorString(e));
    return dev == device ? GA_OK : invalid("the current device is not the handle's device");
}

bool known(ga_dtype t) { return t == GA_FP32 || t == GA_FP16 || t == GA_BF16; }
int64_t size_of(ga_dtype t) { return t == GA_FP32 ? 4 : 2; }

ga::Adamw* as_adamw(const ga_adamw* o) { return reinterpret_cast<ga::Adamw*>(const_cast<ga_adamw*>(o)); }
const ga::LayerNorm* as_ln(const ga_layernorm* n) { return reinterpret_cast<const ga::LayerNorm*>(n); }

bool finite_at_least(float x, float least) { return x >= least && x < INFINITY; }

// Rows of dim elements of `size` bytes, as the kernels take them.
ga_status check_rows(const ga_rows* r, int64_t rows, int64_t dim, int64_t size, const char** data, int64_t* ld) {
    *data = nullptr;
    *ld = 0;
    if (!r || !r->data) return GA_OK;
    if (rows > 1 && r->ld < dim) return invalid("a row stride is shorter than a row");
    if (!aligned(r->data, (uintptr_t)size)) return misaligned("a tensor is not aligned to its element");
    *data = static_cast<const char*>(r->data);
    *ld = r->ld * size;
    return GA_OK;
}

}  // namespace

extern "C" {

int32_t ga_training_version(void) { return GA_TRAINING_VERSION; }

ga_status ga_adamw_create(int32_t W, int32_t n_layers, const int64_t* layer_numel, ga_dtype grad_dtype,
                          int32_t state_bits, const uint8_t* decay, ga_adamw** out) {
    if (!out) return invalid("out is NULL");
    *out = nullptr;
    if (!known(grad_dtype)) return invalid("unknown gradient type");
    if (state_bits != 32 && state_bits != 8) return invalid("state_bits must be 32 or 8");
    ga_plan_info info;
    const ga_status st = ga_plan_compute_info(W, n_layers, layer_numel, GA_FP32, 0, 0.0, &info);
    if (st != GA_OK) return st;
    ga::Adamw* o = new (std::nothrow) ga::Adamw();
    if (!o) return ga::api_fail(GA_ERR_DEVICE, "out of host memory");
    o->W = W;
    o->L = n_layers;
    o->dtype = (int32_t)grad_dtype;
    o->bits = state_bits;
    o->P = info.P;
    o->n_tiles = (info.P + ga::kTile - 1) / ga::kTile;
    o->d_tiles = nullptr;
    o->d_partials = nullptr;
    const size_t tiles_b = sizeof(ga::TileRec) * (size_t)o->n_tiles;
    const size_t offs_b = sizeof(int64_t) * (size_t)(n_layers + 1);
    const size_t all_b = tiles_b + offs_b + (size_t)n_layers;
    char* h = (char*)malloc(all_b);
    if (!h) {
        delete o;
        return ga::api_fail(GA_ERR_DEVICE, "out of host memory");
    }
    ga::TileRec* tiles = reinterpret_cast<ga::TileRec*>(h);
    int64_t* offs = reinterpret_cast<int64_t*>(h + tiles_b);
    uint8_t* flags = reinterpret_cast<uint8_t*>(h + tiles_b + offs_b);
    offs[0] = 0;
    for (int32_t l = 0; l < n_layers; ++l) {
        offs[l + 1] = offs[l] + layer_numel[l];
        flags[l] = decay ? decay[l] != 0 : 1;
    }
    ga::TileRec* next = tiles;
    for (const bool whole : {false, true}) {
        int32_t l = 0;
        for (int64_t t = 0; t < o->n_tiles; ++t) {
            const int64_t e0 = t * ga::kTile;
            while (offs[l + 1] <= e0) ++l;
            if ((offs[l + 1] >= e0 + ga::kTile) != whole) continue;
            const int64_t last = (e0 + ga::kTile < info.P ? e0 + ga::kTile : info.P) - 1;
            int32_t end = l;
            while (offs[end + 1] <= last) ++end;
            next->tile = t;
            next->start = offs[l];
            next->layer = (uint32_t)l;
            next->flags = (whole ? ga::kTileWhole : 0u) | (flags[l] ? ga::kTileDecay : 0u) |
                          ((uint32_t)(end - l) << ga::kTileSpanShift);
            ++next;
        }
    }
    char* d = nullptr;
    hipError_t e = hipGetDevice(&o->device);
    if (e == hipSuccess) e = hipMalloc((void**)&d, all_b);
    if (e == hipSuccess) e = hipMemcpy(d, h, all_b, hipMemcpyHostToDevice);
    const size_t parts_b = sizeof(double) * ga::kNormBlocks;
    const uint64_t zero = 0;
    if (e == hipSuccess) e = hipMalloc((void**)&o->d_partials, parts_b + sizeof zero);
    if (e == hipSuccess) e = hipMemcpy(o->d_partials + ga::kNormBlocks, &zero, sizeof zero, hipMemcpyHostToDevice);
    o->d_done = reinterpret_cast<uint32_t*>(o->d_partials + ga::kNormBlocks);
    free(h);
    o->d_tiles = reinterpret_cast<ga::TileRec*>(d);
    if (e != hipSuccess) {
        const ga_status bad = ga::api_fail(GA_ERR_DEVICE, hipGetErrorString(e));
        (void)hipGetLastError();
        ga_adamw_destroy(reinterpret_cast<ga_adamw*>(o));
        return bad;
    }
    o->d_offsets = reinterpret_cast<int64_t*>(d + tiles_b);
    o->d_decay = reinterpret_cast<uint8_t*>(d + tiles_b + offs_b);
    *out = reinterpret_cast<ga_adamw*>(o);
    return ga::api_ok();
}

void ga_adamw_destroy(ga_adamw* opt) {
    if (!opt) return;
    ga::Adamw* o = as_adamw(opt);
    if (o->d_tiles) (void)hipFree(o->d_tiles);
    if (o->d_partials) (void)hipFree(o->d_partials);
    delete o;
}

ga_status ga_grad_norm(const ga_adamw* opt, const uint64_t* d_layer_ptrs, float max_norm, float* d_grad,
                       ga_clip* d_clip, hipStream_t stream) {
    if (!opt || !d_layer_ptrs || !d_clip) return invalid("NULL argument");
    if (!(max_norm > 0.f)) return invalid("max_norm must be positive");
    if (!aligned(d_layer_ptrs, 8) || !aligned(d_clip, 16) || (d_grad && !aligned(d_grad, 16)))
        return misaligned("misaligned device buffer");
    const ga::Adamw* o = as_adamw(opt);
    const ga_status st = on_device(o->device);
    if (st != GA_OK) return st;
    return launched(ga::launch_grad_norm(*o, d_layer_ptrs, max_norm, d_grad, d_clip, stream));
}

ga_status ga_adamw_step(const ga_adamw* opt, const uint64_t* d_layer_ptrs, const ga_adamw_params* params, float* d_w,
                        const ga_adamw_state* state, const ga_clip* d_clip, void* d_copy, ga_dtype copy_dtype,
                        hipStream_t stream) {
    if (!opt || !d_layer_ptrs || !params || !d_w || !state || !state->m || !state->v) return invalid("NULL argument");
    const ga::Adamw* o = as_adamw(opt);
    if (o->bits == 8 && (!state->m_scale || !state->v_scale)) return invalid("8-bit states need their scales");
    if (params->t < 1) return invalid("t counts steps from 1");
    if (!finite_at_least(params->beta1, 0.f) || !(params->beta1 < 1.f) || !finite_at_least(params->beta2, 0.f) ||
        !(params->beta2 < 1.f))
        return invalid("beta1 and beta2 must be in [0, 1)");
    if (!finite_at_least(params->lr, 0.f) || !finite_at_least(params->eps, 0.f) ||
        !finite_at_least(params->weight_decay, 0.f))
        return invalid("lr, eps and weight_decay must be finite and not negative");
    if (o->bits == 8 && params->m_rounding != GA_ROUND_RANDOM && params->m_rounding != GA_ROUND_NEAREST)
        return invalid("unknown m_rounding");
    if (d_copy && copy_dtype != GA_FP16 && copy_dtype != GA_BF16) return invalid("the copy is GA_FP16 or GA_BF16");
    if (!aligned(d_layer_ptrs, 8) || !aligned(d_w, 16) || !aligned(state->m, 16) || !aligned(state->v, 16) ||
        (d_copy && !aligned(d_copy, 16)) || (d_clip && !aligned(d_clip, 16)) ||
        (o->bits == 8 && (!aligned(state->m_scale, 4) || !aligned(state->v_scale, 4))))
        return misaligned("misaligned device buffer");
    const ga_status st = on_device(o->device);
    if (st != GA_OK) return st;
    // the factors that depend on t, formed in binary64 and rounded once
    const double b1 = params->beta1, b2 = params->beta2, lr = params->lr;
    ga::StepArgs a;
    a.lr_t = (float)(lr / (1.0 - pow(b1, (double)params->t)));
    a.beta1 = params->beta1;
    a.beta2 = params->beta2;
    a.c1 = (float)(1.0 - b1);
    a.c2 = (float)(1.0 - b2);
    // a denormal eps would have no reciprocal in the kernel's hardware instruction
    a.eps = params->eps > 0.f && params->eps < 0x1p-126f ? 0x1p-126f : params->eps;
    a.rbc2 = (float)(1.0 / sqrt(1.0 - pow(b2, (double)params->t)));
    // nor has the hardware's reciprocal a denormal result: the quotient's denominator and lr's factor are scaled alike
    if (a.eps >= 0x1p125f) {
        a.eps *= 0x1p-4f;
        a.rbc2 *= 0x1p-4f;
        a.lr_t *= 0x1p-4f;
    }
    a.keep = (float)(1.0 - lr * (double)params->weight_decay);
    a.seed = (uint32_t)((uint64_t)params->t * 0x9E3779B9u + 0x7F4A7C15u);
    a.m_rounding = params->m_rounding;
    a.w = d_w;
    a.m = state->m;
    a.v = state->v;
    a.m_scale = state->m_scale;
    a.v_scale = state->v_scale;
    a.clip = d_clip;
    a.copy = d_copy;
    a.copy_dtype = (int32_t)copy_dtype;
    return launched(ga::launch_adamw(*o, d_layer_ptrs, a, stream));
}

ga_status ga_layernorm_create(int64_t dim, ga_dtype x_dtype, ga_dtype p_dtype, int32_t backward,
                              ga_layernorm** out) {
    if (!out) return invalid("out is NULL");
    *out = nullptr;
    if (dim < 1) return invalid("dim < 1");
    if (!known(x_dtype) || (p_dtype != GA_FP32 && p_dtype != x_dtype))
        return invalid("p_dtype must be GA_FP32 or x_dtype");
    if (dim > GA_MAX_DIM) return ga::api_fail(GA_ERR_UNSUPPORTED, "dim exceeds GA_MAX_DIM");
    ga::LayerNorm* n = new (std::nothrow) ga::LayerNorm();
    if (!n) return ga::api_fail(GA_ERR_DEVICE, "out of host memory");
    n->dim = dim;
    n->ldp = (dim + 3) / 4 * 4;
    n->x_dtype = (int32_t)x_dtype;
    n->p_dtype = (int32_t)p_dtype;
    n->d_parts = nullptr;
    n->d_done = nullptr;
    hipError_t e = hipGetDevice(&n->device);
    if (e == hipSuccess && backward) {
        const size_t parts_b = sizeof(float) * (size_t)ga::kLnParts * 2 * (size_t)n->ldp;
        const uint32_t zeros[ga::kLnParts] = {};
        e = hipMalloc((void**)&n->d_parts, parts_b + sizeof zeros);
        n->d_done = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(n->d_parts) + parts_b);
        if (e == hipSuccess) e = hipMemcpy(n->d_done, zeros, sizeof zeros, hipMemcpyHostToDevice);
    }
    if (e != hipSuccess) {
        const ga_status bad = ga::api_fail(GA_ERR_DEVICE, hipGetErrorString(e));
        (void)hipGetLastError();
        ga_layernorm_destroy(reinterpret_cast<ga_layernorm*>(n));
        return bad;
    }
    *out = reinterpret_cast<ga_layernorm*>(n);
    return ga::api_ok();
}

void ga_layernorm_destroy(ga_layernorm* ln) {
    if (!ln) return;
    ga::LayerNorm* n = reinterpret_cast<ga::LayerNorm*>(ln);
    if (n->d_parts) (void)hipFree(n->d_parts);
    delete n;
}

ga_status ga_layernorm_forward(const ga_layernorm* ln, int64_t rows, const ga_rows* x, const ga_rows* residual,
                               const void* d_gamma, const void* d_beta, float eps, const ga_rows* y,
                               const ga_rows* sum, float* d_mean, float* d_rstd, hipStream_t stream) {
    if (!ln || !x || !y) return invalid("NULL argument");
    if (rows < 0) return invalid("rows < 0");
    if (!(eps > 0.f && eps < INFINITY)) return invalid("eps must be positive and finite");
    if (rows == 0) return ga::api_ok();
    if (!x->data || !y->data) return invalid("NULL argument");
    const ga::LayerNorm* n = as_ln(ln);
    const int64_t xs = size_of((ga_dtype)n->x_dtype), ps = size_of((ga_dtype)n->p_dtype);
    ga::LnFwd a;
    const char *py, *psum;
    ga_status st = check_rows(x, rows, n->dim, xs, &a.x, &a.ldx);
    if (st == GA_OK) st = check_rows(residual, rows, n->dim, xs, &a.res, &a.ldr);
    if (st == GA_OK) st = check_rows(y, rows, n->dim, xs, &py, &a.ldy);
    if (st == GA_OK) st = check_rows(sum, rows, n->dim, xs, &psum, &a.lds);
    if (st != GA_OK) return st;
    if (psum && !a.res) return invalid("a sum output needs a residual");
    if (psum && psum == py) return invalid("y and sum must be different tensors");
    if (!aligned(d_gamma, (uintptr_t)ps) || !aligned(d_beta, (uintptr_t)ps) || !aligned(d_mean, 4) ||
        !aligned(d_rstd, 4))
        return misaligned("a vector is not aligned to its element");
    st = on_device(n->device);
    if (st != GA_OK) return st;
    a.y = const_cast<char*>(py);
    a.sum = const_cast<char*>(psum);
    a.gamma = d_gamma;
    a.beta = d_beta;
    a.mean = d_mean;
    a.rstd = d_rstd;
    a.eps = eps;
    a.rows = rows;
    return launched(ga::launch_ln_fwd(*n, a, stream));
}

ga_status ga_layernorm_backward(const ga_layernorm* ln, int64_t rows, const ga_rows* dy, const ga_rows* x,
                                const void* d_gamma, const float* d_mean, const float* d_rstd, const ga_rows* dsum,
                                const ga_rows* dx, int32_t groups, void* d_dgamma, void* d_dbeta, ga_dtype dp_dtype,
                                hipStream_t stream) {
    if (!ln || !dy || !x || !dx) return invalid("NULL argument");
    if (rows < 0) return invalid("rows < 0");
    if (groups < 1) return invalid("groups < 1");
    if (groups > GA_MAX_GROUPS) return ga::api_fail(GA_ERR_UNSUPPORTED, "groups exceed GA_MAX_GROUPS");
    if (rows % groups != 0) return invalid("groups does not divide rows");
    if (!d_dgamma != !d_dbeta) return invalid("d_dgamma and d_dbeta are given together or not at all");
    if (d_dgamma && !known(dp_dtype)) return invalid("unknown type of the weight gradients");
    const ga::LayerNorm* n = as_ln(ln);
    if (!n->d_parts) return invalid("the handle was made without a backward pass");
    if (rows > 0 && (!dy->data || !x->data || !dx->data || !d_mean || !d_rstd)) return invalid("NULL argument");
    if (rows == 0 && !d_dgamma) return ga::api_ok();
    const int64_t xs = size_of((ga_dtype)n->x_dtype), ps = size_of((ga_dtype)n->p_dtype);
    ga::LnBwd a;
    memset(&a, 0, sizeof a);
    const char* pdx = nullptr;
    ga_status st = GA_OK;
    if (rows > 0) {
        st = check_rows(dy, rows, n->dim, xs, &a.dy, &a.ldy);
        if (st == GA_OK) st = check_rows(x, rows, n->dim, xs, &a.x, &a.ldx);
        if (st == GA_OK) st = check_rows(dsum, rows, n->dim, xs, &a.dsum, &a.lds);
        if (st == GA_OK) st = check_rows(dx, rows, n->dim, xs, &pdx, &a.ldd);
        if (st != GA_OK) return st;
    }
    const uintptr_t ds = d_dgamma ? (uintptr_t)size_of(dp_dtype) : 1;
    if (!aligned(d_gamma, (uintptr_t)ps) || !aligned(d_mean, 4) || !aligned(d_rstd, 4) || !aligned(d_dgamma, ds) ||
        !aligned(d_dbeta, ds))
        return misaligned("a vector is not aligned to its element");
    st = on_device(n->device);
    if (st != GA_OK) return st;
    a.dx = const_cast<char*>(pdx);
    a.gamma = d_gamma;
    a.mean = d_mean;
    a.rstd = d_rstd;
    a.rows = rows;
    a.group_rows = rows / groups;
    a.groups = groups;
    a.dgamma = d_dgamma;
    a.dbeta = d_dbeta;
    a.dp_dtype = (int32_t)dp_dtype;
    return launched(ga::launch_ln_bwd(*n, a, stream));
}

}  // extern "C"
