// C ABI of the layer operators: handles, argument validation and launches.  The
// operations are specified in include/gradagg.h.
#include "layers.h"

#include <math.h>
#include <string.h>

#include <new>

#include "plan.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

ga_status invalid(const char* msg) { return ga::api_fail(GA_ERR_INVALID, msg); }
ga_status misaligned(const char* msg) { return ga::api_fail(GA_ERR_ALIGN, msg); }
ga_status unsupported(const char* msg) { return ga::api_fail(GA_ERR_UNSUPPORTED, msg); }

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
int64_t size_of(int32_t t) { return t == GA_FP32 ? 4 : 2; }

constexpr int64_t kMost = ((int64_t)1 << 31) - 1;
// Strides in elements beyond this could not be those of memory; sums of products of two sizes stay within 63 bits.
constexpr int64_t kMostStride = (int64_t)1 << 44;

const ga::GroupNorm* as_gn(const ga_groupnorm* n) { return reinterpret_cast<const ga::GroupNorm*>(n); }
const ga::Router* as_router(const ga_router* r) { return reinterpret_cast<const ga::Router*>(r); }

// Images of C channels of `size` bytes, as the kernels take them.
ga_status check_images(const ga_images* m, int64_t N, int64_t S, int64_t C, int64_t size, ga::Images* out) {
    if (!m || !m->data) return invalid("NULL argument");
    const int64_t ld = S > 1 ? m->ld : C;
    const int64_t sample = N > 1 ? m->sample : C;
    if (ld < C || sample < C || ld > kMostStride || sample > kMostStride) return invalid("a stride is shorter than the channels, or too large");
    // S and N are below 2^31, strides at most 2^44: in binary64 where the exact products could pass 63 bits
    if (N > 1 && S > 1 && (double)sample < (double)(S - 1) * (double)ld + (double)C &&
        (double)ld < (double)(N - 1) * (double)sample + (double)C)
        return invalid("the samples overlap");
    if (!aligned(m->data, (uintptr_t)size)) return misaligned("a tensor is not aligned to its element");
    out->data = static_cast<const char*>(m->data);
    out->ld = ld * size;
    out->sample = sample * size;
    return GA_OK;
}

// Rows of E logits.
ga_status check_logits(const ga_rows* r, int64_t rows, int64_t E, int64_t size, const char** data, int64_t* ld) {
    if (!r || !r->data) return invalid("NULL argument");
    if (rows > 1 && (r->ld < E || r->ld > kMostStride)) return invalid("a row stride is shorter than a row, or too large");
    if (!aligned(r->data, (uintptr_t)size)) return misaligned("a tensor is not aligned to its element");
    *data = static_cast<const char*>(r->data);
    *ld = (rows > 1 ? r->ld : E) * size;
    return GA_OK;
}

ga_status check_tokens(const ga::Router& r, int64_t tokens) {
    if (tokens < 0) return invalid("tokens < 0");
    if (tokens > kMost / r.k) return unsupported("tokens * k exceeds 2^31 - 1");
    if (tokens % r.W != 0) return invalid("workers does not divide tokens");
    return GA_OK;
}

}  // namespace

extern "C" {

int32_t ga_layers_version(void) { return GA_LAYERS_VERSION; }

ga_status ga_groupnorm_create(int32_t channels, int32_t groups, ga_dtype x_dtype, ga_dtype p_dtype,
                              ga_activation activation, int32_t backward, ga_groupnorm** out) {
    if (!out) return invalid("out is NULL");
    *out = nullptr;
    if (channels < 1) return invalid("channels < 1");
    if (groups < 1 || channels % groups != 0) return invalid("groups must divide the channels");
    if (!known(x_dtype) || (p_dtype != GA_FP32 && p_dtype != x_dtype))
        return invalid("p_dtype must be GA_FP32 or x_dtype");
    if (activation != GA_ACT_NONE && activation != GA_ACT_RELU && activation != GA_ACT_SILU)
        return invalid("unknown activation");
    if (channels > GA_MAX_CHANNELS) return unsupported("channels exceed GA_MAX_CHANNELS");
    ga::GroupNorm* n = new (std::nothrow) ga::GroupNorm();
    if (!n) return ga::api_fail(GA_ERR_DEVICE, "out of host memory");
    n->C = channels;
    n->G = groups;
    n->x_dtype = (int32_t)x_dtype;
    n->p_dtype = (int32_t)p_dtype;
    n->act = (int32_t)activation;
    n->backward = backward != 0;
    n->ldp = (channels + 3) / 4 * 4;
    const int64_t rows = ga::kGnRowBytes / (2 * (int64_t)sizeof(float) * n->ldp);
    n->rows = rows < ga::kGnRows ? (int32_t)rows : ga::kGnRows;
    n->d_rows = nullptr;
    n->d_records = nullptr;
    hipError_t e = hipGetDevice(&n->device);
    if (e == hipSuccess && backward)
        e = hipMalloc((void**)&n->d_rows, 2 * sizeof(float) * (size_t)n->rows * (size_t)n->ldp);
    if (e == hipSuccess) e = hipMalloc(&n->d_records, 16 * (size_t)ga::kGnRecords);
    if (e != hipSuccess) {
        const ga_status bad = ga::api_fail(GA_ERR_DEVICE, hipGetErrorString(e));
        (void)hipGetLastError();
        ga_groupnorm_destroy(reinterpret_cast<ga_groupnorm*>(n));
        return bad;
    }
    *out = reinterpret_cast<ga_groupnorm*>(n);
    return ga::api_ok();
}

void ga_groupnorm_destroy(ga_groupnorm* gn) {
    if (!gn) return;
    ga::GroupNorm* n = reinterpret_cast<ga::GroupNorm*>(gn);
    if (n->d_rows) (void)hipFree(n->d_rows);
    if (n->d_records) (void)hipFree(n->d_records);
    delete n;
}

ga_status ga_groupnorm_forward(const ga_groupnorm* gn, int64_t samples, int64_t positions, const ga_images* x,
                               const void* d_gamma, const void* d_beta, float eps, const ga_images* y, float* d_mean,
                               float* d_rstd, hipStream_t stream) {
    if (!gn || !x || !y) return invalid("NULL argument");
    if (samples < 0 || positions < 0) return invalid("a size is negative");
    if (!(eps > 0.f && eps < INFINITY)) return invalid("eps must be positive and finite");
    if (samples == 0 || positions == 0) return ga::api_ok();
    const ga::GroupNorm* n = as_gn(gn);
    if (positions > kMost || samples > kMost / n->G) return unsupported("samples * groups or positions exceed 2^31 - 1");
    const int64_t xs = size_of(n->x_dtype), ps = size_of(n->p_dtype);
    ga::GnArgs a;
    memset(&a, 0, sizeof a);
    ga_status st = check_images(x, samples, positions, n->C, xs, &a.x);
    if (st == GA_OK) st = check_images(y, samples, positions, n->C, xs, &a.y);
    if (st != GA_OK) return st;
    if (!aligned(d_gamma, (uintptr_t)ps) || !aligned(d_beta, (uintptr_t)ps) || !aligned(d_mean, 4) ||
        !aligned(d_rstd, 4))
        return misaligned("a vector is not aligned to its element");
    st = on_device(n->device);
    if (st != GA_OK) return st;
    a.N = samples;
    a.S = positions;
    a.gamma = d_gamma;
    a.beta = d_beta;
    a.eps = eps;
    a.mean = d_mean;
    a.rstd = d_rstd;
    return launched(ga::launch_gn_fwd(*n, a, stream));
}

ga_status ga_groupnorm_backward(const ga_groupnorm* gn, int64_t samples, int64_t positions, const ga_images* dy,
                                const ga_images* x, const void* d_gamma, const void* d_beta, const float* d_mean,
                                const float* d_rstd, const ga_images* dx, int32_t workers, void* d_dgamma,
                                void* d_dbeta, ga_dtype dp_dtype, hipStream_t stream) {
    if (!gn || !dy || !x || !dx) return invalid("NULL argument");
    if (samples < 0 || positions < 0) return invalid("a size is negative");
    if (workers < 1) return invalid("workers < 1");
    if (workers > GA_MAX_WORKERS) return unsupported("workers exceed GA_MAX_WORKERS");
    if (samples % workers != 0) return invalid("workers does not divide samples");
    if (!d_dgamma != !d_dbeta) return invalid("d_dgamma and d_dbeta are given together or not at all");
    if (d_dgamma && !known(dp_dtype)) return invalid("unknown type of the weight gradients");
    const ga::GroupNorm* n = as_gn(gn);
    if (!n->backward) return invalid("the handle was made without a backward pass");
    const bool none = samples == 0 || positions == 0;
    if (none && !d_dgamma) return ga::api_ok();
    if (positions > kMost || samples > kMost / n->G) return unsupported("samples * groups or positions exceed 2^31 - 1");
    const int64_t xs = size_of(n->x_dtype), ps = size_of(n->p_dtype);
    ga::GnArgs a;
    memset(&a, 0, sizeof a);
    if (!none) {
        if (!d_mean || !d_rstd) return invalid("NULL argument");
        ga_status st = check_images(dy, samples, positions, n->C, xs, &a.dy);
        if (st == GA_OK) st = check_images(x, samples, positions, n->C, xs, &a.x);
        if (st == GA_OK) st = check_images(dx, samples, positions, n->C, xs, &a.y);
        if (st != GA_OK) return st;
    }
    const uintptr_t ds = d_dgamma ? (uintptr_t)size_of(dp_dtype) : 1;
    if (!aligned(d_gamma, (uintptr_t)ps) || !aligned(d_beta, (uintptr_t)ps) || !aligned(d_mean, 4) ||
        !aligned(d_rstd, 4) || !aligned(d_dgamma, ds) || !aligned(d_dbeta, ds))
        return misaligned("a vector is not aligned to its element");
    const ga_status st = on_device(n->device);
    if (st != GA_OK) return st;
    a.N = none ? 0 : samples;
    a.S = positions;
    a.gamma = d_gamma;
    a.beta = d_beta;
    a.mean = const_cast<float*>(d_mean);
    a.rstd = const_cast<float*>(d_rstd);
    a.workers = workers;
    a.per_worker = a.N / workers;
    a.dgamma = d_dgamma;
    a.dbeta = d_dbeta;
    a.dp_dtype = (int32_t)dp_dtype;
    return launched(ga::launch_gn_bwd(*n, a, stream));
}

ga_status ga_router_create(int32_t experts, int32_t k, ga_dtype x_dtype, int32_t workers, int32_t normalize,
                           ga_balance balance, ga_router** out) {
    if (!out) return invalid("out is NULL");
    *out = nullptr;
    if (experts < 1) return invalid("experts < 1");
    if (k < 1 || k > experts) return invalid("k must be between 1 and the number of experts");
    if (workers < 1) return invalid("workers < 1");
    if (!known(x_dtype)) return invalid("unknown type of the logits");
    if (balance != GA_BALANCE_ALL && balance != GA_BALANCE_WORKER) return invalid("unknown balance");
    if (experts > GA_MAX_EXPERTS) return unsupported("experts exceed GA_MAX_EXPERTS");
    if (k > GA_MAX_TOPK) return unsupported("k exceeds GA_MAX_TOPK");
    if (workers > GA_MAX_WORKERS) return unsupported("workers exceed GA_MAX_WORKERS");
    ga::Router* r = new (std::nothrow) ga::Router();
    if (!r) return ga::api_fail(GA_ERR_DEVICE, "out of host memory");
    r->E = experts;
    r->k = k;
    r->W = workers;
    r->x_dtype = (int32_t)x_dtype;
    r->normalize = normalize != 0;
    r->scope = (int32_t)balance;
    r->d_squares = nullptr;
    hipError_t e = hipGetDevice(&r->device);
    r->rows = workers > ga::kRouterRows ? workers : ga::kRouterRows;
    const size_t rows = (size_t)r->rows, all = rows * (size_t)experts;
    char* d = nullptr;
    if (e == hipSuccess) e = hipMalloc((void**)&d, 8 * (rows + GA_MAX_EXPERTS) + 4 * (2 * all + rows) + 8);
    if (e == hipSuccess) {
        r->d_squares = reinterpret_cast<double*>(d);
        r->d_dots = r->d_squares + rows;
        r->d_probs = reinterpret_cast<float*>(r->d_dots + GA_MAX_EXPERTS);
        r->d_counts = reinterpret_cast<int32_t*>(r->d_probs + all);
        r->d_tokens = r->d_counts + all;
        r->d_done = reinterpret_cast<uint32_t*>(r->d_tokens + rows);
        const uint32_t zeros[2] = {};
        e = hipMemcpy(r->d_done, zeros, sizeof zeros, hipMemcpyHostToDevice);
    }
    if (e != hipSuccess) {
        const ga_status bad = ga::api_fail(GA_ERR_DEVICE, hipGetErrorString(e));
        (void)hipGetLastError();
        ga_router_destroy(reinterpret_cast<ga_router*>(r));
        return bad;
    }
    *out = reinterpret_cast<ga_router*>(r);
    return ga::api_ok();
}

void ga_router_destroy(ga_router* router) {
    if (!router) return;
    ga::Router* r = reinterpret_cast<ga::Router*>(router);
    if (r->d_squares) (void)hipFree(r->d_squares);
    delete r;
}

ga_status ga_router_forward(const ga_router* router, int64_t tokens, const ga_rows* logits, const uint8_t* d_mask,
                            int32_t select, const ga_routing* routing, const ga_load* load, hipStream_t stream) {
    if (!router || !logits || !routing) return invalid("NULL argument");
    const ga::Router* r = as_router(router);
    if (load && (!load->counts || !load->probs || !load->tokens || !load->loss || !load->slope))
        return invalid("a load needs all its buffers");
    ga_status st = check_tokens(*r, tokens);
    if (st != GA_OK) return st;
    if (tokens == 0 && !load) return ga::api_ok();
    ga::RouteArgs a;
    memset(&a, 0, sizeof a);
    if (tokens > 0) {
        if (!routing->experts) return invalid("NULL argument");
        st = check_logits(logits, tokens, r->E, size_of(r->x_dtype), &a.x, &a.ldx);
        if (st != GA_OK) return st;
    }
    if (!aligned(routing->experts, 4) || !aligned(routing->gates, 4) || !aligned(routing->lse, 4) ||
        (load && (!aligned(load->counts, 4) || !aligned(load->probs, 4) || !aligned(load->tokens, 4) ||
                  !aligned(load->loss, 4) || !aligned(load->slope, 4))))
        return misaligned("a buffer is not aligned to its element");
    st = on_device(r->device);
    if (st != GA_OK) return st;
    a.T = tokens;
    a.per_worker = tokens / r->W;
    a.mask = d_mask;
    a.select = select != 0;
    a.r = *routing;
    a.with_load = load != nullptr;
    if (load) a.load = *load;
    return launched(ga::launch_router_fwd(*r, a, stream));
}

ga_status ga_router_backward(const ga_router* router, int64_t tokens, const ga_rows* logits, const uint8_t* d_mask,
                             const ga_routing* routing, const float* d_slope, const float* d_dgates, float balance,
                             float z, const ga_rows* dlogits, hipStream_t stream) {
    if (!router || !logits || !routing || !dlogits) return invalid("NULL argument");
    const ga::Router* r = as_router(router);
    ga_status st = check_tokens(*r, tokens);
    if (st != GA_OK) return st;
    if (!(fabsf(balance) < INFINITY) || !(fabsf(z) < INFINITY)) return invalid("balance and z must be finite");
    if (!d_slope && (balance != 0.f || z != 0.f)) return invalid("the losses' gradients need the slope");
    if (tokens == 0) return ga::api_ok();
    if (!routing->lse || (d_dgates && (!routing->experts || (r->normalize && !routing->gates))))
        return invalid("NULL argument");
    ga::RouteArgs a;
    memset(&a, 0, sizeof a);
    const char* pdx = nullptr;
    st = check_logits(logits, tokens, r->E, size_of(r->x_dtype), &a.x, &a.ldx);
    if (st == GA_OK) st = check_logits(dlogits, tokens, r->E, size_of(r->x_dtype), &pdx, &a.ldd);
    if (st != GA_OK) return st;
    if (!aligned(routing->experts, 4) || !aligned(routing->gates, 4) || !aligned(routing->lse, 4) ||
        !aligned(d_slope, 4) || !aligned(d_dgates, 4))
        return misaligned("a buffer is not aligned to its element");
    st = on_device(r->device);
    if (st != GA_OK) return st;
    a.T = tokens;
    a.per_worker = tokens / r->W;
    a.mask = d_mask;
    a.r = *routing;
    a.dx = const_cast<char*>(pdx);
    a.slope = d_slope;
    a.dgates = d_dgates;
    a.balance = balance;
    a.z = z;
    return launched(ga::launch_router_bwd(*r, a, stream));
}

}  // extern "C"
