// Router of a mixture of experts with its counts and balance loss
// (ga_router_forward, ga_router_backward).
//
// A token's row of E logits is read once, by a team of lanes that keeps it in registers: its largest logit, the sum of
// exp(l - largest), and from them lse = largest + log(sum) and p = exp(l - largest) / sum.  The k largest are found by
// rank: logits as whole numbers of the same order, a bound that at least k of them reach, those above it written to the
// team's list in LDS with their index, and for each of the list the number of larger ones, which is its place (or, where
// equal logits make the list long, the largest left of it, k times).  Counts go to
// a histogram in LDS (whole numbers, in any order), probabilities are summed in each lane's registers over the tokens that
// it takes.  A workgroup leaves one partial row of both; a second kernel adds the rows in order, and ends the losses.
//
// Backward, with h_e = balance * slope_e (+ dgate at its expert) and p = exp(l - lse) formed again:
//   dl_e = p_e (h_e - sum(h p) + z slope_z lse), and with normalised gates + gate_j (dgate_j - sum(dgate gate)) at expert j.
//
// What bounds it: forward vector instructions, 66 to 75% of the SIMDs' time, and waits of the 16 wavefronts that the lists
// leave room for on a CU (131072 x 256 binary32, 8 of them: 34 instructions to a logit, 45 us at 3.2 TB/s, its bytes alone 23;
// 65536 x 64 bf16, 6 of them: 64 to a logit, 14 us for 12 MB); backward HBM and the exponentials (131072 x 256 bf16: 31 us,
// 4.7 TB/s).  Small calls: the launch and a chain of some 5 us.
#include <type_traits>

#include "arrival.h"
#include "layers.h"
#include "rowvec.h"

namespace ga {

namespace {

constexpr int kThreads = 256;
// Of a workgroup that leaves a partial load: 256 workgroups fill the chip, and few rows are to be added (131072 x 256
// binary32, with other steps: 63 us, with 1024 workgroups of 256 threads 82).
constexpr int kLoadThreads = 1024;
constexpr float kLog2e = 1.44269504f;

// ---- teams of L lanes (a power of 2, aligned), all of whose lanes get the result ----

template <int L, typename OP>
__device__ __forceinline__ uint32_t team_reduce(uint32_t x, OP op) {
    if constexpr (L >= 2) x = op(x, lane_move<0xb1>(x));      // xor 1
    if constexpr (L >= 4) x = op(x, lane_move<0x4e>(x));      // xor 2
    if constexpr (L >= 8) x = op(x, lane_move<0x141>(x));     // mirror within 8
    if constexpr (L >= 16) x = op(x, lane_move<0x140>(x));    // mirror within 16
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = op(r[0], r[1]);
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = op(r[0], r[1]);
    }
    return x;
}

template <int L>
__device__ __forceinline__ float team_sum(float x) {
    return __uint_as_float(team_reduce<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t x) {
    return team_reduce<L>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int L>
__device__ __forceinline__ int team_sum(int x) {
    return (int)team_reduce<L>((uint32_t)x, [](uint32_t a, uint32_t b) { return a + b; });
}

// Sum of the team's lanes up to this one: within a row of 16 lanes by shifts, over rows by broadcasts of the last lane.
template <int L>
__device__ __forceinline__ int team_scan(int x) {
    const int ln = threadIdx.x & (L - 1);
    const auto from = [&](uint32_t y, int back) { return ln >= back ? (int)y : 0; };
    if constexpr (L >= 2) x += from(lane_move<0x111>((uint32_t)x), 1);
    if constexpr (L >= 4) x += from(lane_move<0x112>((uint32_t)x), 2);
    if constexpr (L >= 8) x += from(lane_move<0x114>((uint32_t)x), 4);
    if constexpr (L >= 16) x += from(lane_move<0x118>((uint32_t)x), 8);
    if constexpr (L >= 32) {
        const int y = __shfl(x, (threadIdx.x & 63 & ~31) + 15, 64);
        if (ln & 16) x += y;
    }
    if constexpr (L >= 64) {
        const int y = __shfl(x, 31, 64);
        if (ln & 32) x += y;
    }
    return x;
}

// What one lane of a wavefront wrote to LDS, another may now read: the hardware keeps a wavefront's accesses in order,
// this keeps the compiler's.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A lane's V elements of a row of E: vectors of N elements, those of a team's lanes next to each other.
template <int X, int L, int V>
struct Lane {
    static constexpr int N = kVec<X>, J = V / N;
    int ln, E;

    __device__ __forceinline__ explicit Lane(int experts) : ln(threadIdx.x & (L - 1)), E(experts) {}
    __device__ __forceinline__ int column(int i) const { return (i / N * L + ln) * N + i % N; }

    __device__ __forceinline__ void load(Raw<X, N> (&r)[J], uint64_t row) const {
#pragma unroll
        for (int j = 0; j < J; ++j) load_ahead<X, N, false>(r[j], row, (j * L + ln) * N, E);
    }

    // The values; past the row's end, and everywhere of an absent row, -infinity.
    __device__ __forceinline__ void widen(Raw<X, N> (&r)[J], float (&f)[V], bool present) const {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float t[N];
            into_place(r[j], (j * L + ln) * N, E);
            r[j].widen(t);
#pragma unroll
            for (int e = 0; e < N; ++e) f[j * N + e] = t[e];
        }
        if (E < L * V || !present) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = present && column(i) < E ? f[i] : -INFINITY;
        }
    }
};

// A logit as a whole number of the same order; zeros of both signs alike; a NaN, as the least (never selected), 0.
// -infinity is kLeast.
constexpr uint32_t kLeast = 0x007fffffu;

__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return v == v ? key : 0u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((int32_t)key < 0 ? 0x80000000u : 0xffffffffu));
}

// Of the maxima of the team's L * GROUPS groups of keys (a lane's V are GROUPS of them), the k-th when equal ones count
// once, the first one given; 0 where there are fewer.
template <int L, int V, int GROUPS>
__device__ __forceinline__ uint32_t kth_of_groups(const uint32_t (&key)[V], uint32_t first, int k) {
    constexpr int EACH = V / GROUPS;
    uint32_t top[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        top[g] = key[g * EACH];
#pragma unroll
        for (int i = 1; i < EACH; ++i) top[g] = top[g] > key[g * EACH + i] ? top[g] : key[g * EACH + i];
    }
    uint32_t bound = first;
    for (int j = 1; j < k; ++j) {
        uint32_t best = 0u;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const uint32_t x = top[g] < bound ? top[g] : 0u;
            best = best > x ? best : x;
        }
        bound = team_max<L>(best);
    }
    return bound;
}

// Whether, instead of ranking so many candidates against each other, found^2 / L comparisons to a lane, the k largest are
// found one after the other, each in found / L steps and two exchanges: where many logits are equal (all, where a router's
// weights are still 0).  Ranked against not, us, with a load: 65536 x 256, 8 of them (16 lanes), 25 candidates 42, 43; 33:
// 56, 47; 256: 497, 99.  16384 x 1024, 32 of them (64 lanes), 100: 63, 97; 145: 111, 113; 1024: 1543, 245.  131072 x 64 bf16,
// 1 of them (8 lanes), 12: 24, 23; 64: 136, 29.
template <int L>
__device__ __forceinline__ bool too_many(int found, int k) {
    return found > L + 2 * k;
}

// A candidate is its key and, below, the complement of its index, so that among equal ones the lowest index is the largest;
// the upper bits of that give way to a place where it is known.
__device__ __forceinline__ uint32_t placed(uint32_t index, int place) { return (index & 1023u) | (uint32_t)place << 10; }
__device__ __forceinline__ int place_of(uint32_t index) { return (int)(index >> 10); }
__device__ __forceinline__ int index_of(uint32_t index) { return (int)(~index & 1023u); }
static_assert(GA_MAX_EXPERTS <= 1024, "an index of 10 bits");

// Where the partial loads of the workgroups lie: row = worker * parts + part.
struct LoadParts {
    float* probs;          // [rows][E]
    int32_t* counts;       // [rows][E]
    double* squares;       // [rows]
    int32_t* tokens;       // [rows]
    double* dots;          // a part of the balance loss for each chunk of experts
    uint32_t* done;        // [2], of the parts of the loss and of the partial loads (see arrival); 0 between calls
    int32_t parts;
};

struct LossArgs {
    ga_load load;
    int32_t E, k, W, scope;
};

// CHUNK: experts of a chunk.
template <int THREADS, int CHUNK>
struct EndScratch {
    double p[THREADS / CHUNK][CHUNK];
    int64_t c[THREADS / CHUNK][CHUNK];
    int64_t n[THREADS / CHUNK > THREADS / 64 ? THREADS / CHUNK : THREADS / 64];
    double z[THREADS / 64];
};

// 1 / tokens; 0 without tokens.
__device__ __forceinline__ double share_of(int64_t n) { return n > 0 ? 1.0 / (double)n : 0.0; }

// Ends the load of chunk `chunk` of the experts: the workers' counts and sums, and the slope; returns the chunk's part
// of the balance loss in thread 0.  CHUNK threads side by side take an expert each, THREADS / CHUNK of them share its
// partial rows.
template <int THREADS, int CHUNK>
__device__ __forceinline__ double end_chunk(const LossArgs& a, const LoadParts& q, EndScratch<THREADS, CHUNK>& s, int chunk) {
    constexpr int SLICES = THREADS / CHUNK, WAVE = 64 / CHUNK;
    static_assert(CHUNK <= 64, "a wavefront adds the chunk's parts of the loss");
    const int col = threadIdx.x & (CHUNK - 1), slice = threadIdx.x / CHUNK, e = chunk * CHUNK + col;
    int at_once = 1;                                      // workers taken together
    while (at_once * 2 <= SLICES && at_once < a.W) at_once *= 2;
    const int per = SLICES / at_once, wl = slice / per, ps = slice % per;
    const bool all = a.scope == GA_BALANCE_ALL;
    double P = 0.0, dot = 0.0;
    int64_t F = 0, all_n = 0;
    for (int w0 = 0; w0 < a.W; w0 += at_once) {
        const int w = w0 + wl;
        double p = 0.0;
        int64_t c = 0, n = 0;
        if (w < a.W && e < a.E) {
#pragma unroll 8
            for (int i = ps; i < q.parts; i += per) {
                const int64_t row = (int64_t)w * q.parts + i, at = row * a.E + e;
                p += (double)q.probs[at];
                c += q.counts[at];
                n += q.tokens[row];
            }
        }
        // the slices of a wavefront, then the others
#pragma unroll
        for (int o = 1; o < WAVE; o <<= 1) {
            if (o >= per) break;
            p += __shfl_xor(p, o * CHUNK, 64);
            c += __shfl_xor(c, o * CHUNK, 64);
            n += __shfl_xor(n, o * CHUNK, 64);
        }
        __syncthreads();
        s.p[slice][col] = p;
        s.c[slice][col] = c;
        if (col == 0) s.n[slice] = n;
        __syncthreads();
        if (ps != 0 || w >= a.W || e >= a.E) continue;
#pragma unroll 4
        for (int i = WAVE; i < per; i += WAVE) {
            p += s.p[slice + i][col];
            c += s.c[slice + i][col];
            n += s.n[slice + i];
        }
        a.load.probs[(int64_t)w * a.E + e] = (float)p;
        a.load.counts[(int64_t)w * a.E + e] = (int32_t)c;
        P += p;
        F += c;
        all_n += n;
        if (!all) {
            const double share = share_of(n), slope = (double)c * a.E / a.k * share * share / a.W;
            a.load.slope[(int64_t)w * (a.E + 1) + e] = (float)slope;
            dot += slope * p;
        }
    }
    __syncthreads();
    s.p[slice][col] = all ? P : dot;
    s.c[slice][col] = F;
    if (col == 0) s.n[slice] = all_n;
    __syncthreads();
    if (slice == 0) {
#pragma unroll 4
        for (int i = 1; i < at_once; ++i) {
            P += s.p[i * per][col];
            dot += s.p[i * per][col];
            F += s.c[i * per][col];
            all_n += s.n[i * per];
        }
        if (all) {
            const double share = share_of(all_n), slope = (double)F * a.E / a.k * share * share;
            if (e < a.E) a.load.slope[e] = (float)slope;
            dot = slope * P;
        }
    }
    return threadIdx.x < 64 ? wave_sum_f64(slice == 0 && e < a.E ? dot : 0.0) : 0.0;
}

// What is not of a chunk: the workers' tokens, the z loss, and the slope's last column.  A wavefront takes a worker.
template <int THREADS, int CHUNK>
__device__ __forceinline__ void end_rest(const LossArgs& a, const LoadParts& q, EndScratch<THREADS, CHUNK>& s) {
    const bool all = a.scope == GA_BALANCE_ALL;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    double Z = 0.0;
    int64_t all_n = 0;
    for (int w = wave; w < a.W; w += THREADS / 64) {
        double z = 0.0;
        int32_t n = 0;
        for (int i = lane; i < q.parts; i += 64) {
            z += q.squares[(int64_t)w * q.parts + i];
            n += q.tokens[(int64_t)w * q.parts + i];
        }
        z = wave_sum_f64(z);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
        all_n += n;
        const double share = share_of(n) / a.W;
        Z += all ? z : z * share;
        if (lane == 0) {
            a.load.tokens[w] = n;
            if (!all) a.load.slope[(int64_t)w * (a.E + 1) + a.E] = (float)(2.0 * share);
        }
    }
    __syncthreads();
    if (lane == 0) {
        s.z[wave] = Z;
        s.n[wave] = all_n;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < THREADS / 64; ++i) {
        Z += s.z[i];
        all_n += s.n[i];
    }
    a.load.loss[1] = (float)(all ? Z * share_of(all_n) : Z);
    if (all) a.load.slope[a.E] = (float)(2.0 * share_of(all_n));
}

// Whether this workgroup is the last of the launch to get here; what the others stored before is then visible.  Each
// wavefront waits for its own stores: the barrier does not, and the release, thread 0's, writes back what the cache holds
// then.
__device__ __forceinline__ bool last_of(uint32_t* done) {
    __shared__ uint32_t last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t mine = arrival(blockIdx.x, gridDim.x);
        last = __hip_atomic_fetch_add(done, mine, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT) + mine == 0u;
    }
    __syncthreads();
    if (!last) return false;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    return true;
}

constexpr int kEndThreads = 1024;

// A workgroup for each chunk, and one for the rest.  256 rows of 64 to 256 experts: 6 to 7 us, launch and exchange for the most
// part; the exchange by a release, which writes the cache back, took 2 us more.
template <int CHUNK>
__global__ __launch_bounds__(kEndThreads) void k_load_end(LossArgs a, LoadParts q) {
    __shared__ EndScratch<kEndThreads, CHUNK> s;
    if (blockIdx.x + 1 == gridDim.x) {
        end_rest(a, q, s);
        return;
    }
    const double dot = end_chunk(a, q, s, (int)blockIdx.x);
    if (gridDim.x == 2) {
        if (threadIdx.x == 0) a.load.loss[0] = (float)dot;
        return;
    }
    if (threadIdx.x >= 64) return;
    // The parts of the loss are all that passes between workgroups: they are stored past the caches, and have arrived
    // before the count that says so, with no cache written back.
    uint32_t last = 0;
    if (threadIdx.x == 0) {
        __hip_atomic_store(q.dots + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint32_t mine = arrival(blockIdx.x, gridDim.x - 1);
        last = __hip_atomic_fetch_add(q.done, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + mine == 0u ? 1u : 0u;
    }
    if (__builtin_amdgcn_readfirstlane(last) == 0u) return;
    asm volatile("" ::: "memory");
    double loss = threadIdx.x + 1 < gridDim.x
                      ? __hip_atomic_load(q.dots + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    loss = wave_sum_f64(loss);
    if (threadIdx.x == 0) a.load.loss[0] = (float)loss;
}

static_assert(GA_MAX_EXPERTS / 16 <= 64, "a wavefront adds the chunks");

// ---- forward -----------------------------------------------------------------

// LOAD 0: the routing alone; 1: partial loads too; 2: and the workgroup that ends last adds them (which takes registers).
template <int X, int L, int V, int LOAD, int THREADS>
__global__ __launch_bounds__(THREADS) void k_route(RouteArgs a, LossArgs la, LoadParts q, int32_t normalize) {
    constexpr int TEAMS = THREADS / L, N = kVec<X>, J = V / N, EMAX = L * V;
    // while tokens are routed: the candidates of each team; then the wavefronts' sums; then what ends the load
    constexpr size_t LISTS = sizeof(uint64_t) * TEAMS * EMAX, COLS = sizeof(float) * (THREADS / 64) * EMAX;
    constexpr int CHUNK = EMAX < 64 ? EMAX : 64;
    constexpr size_t ENDS = LOAD == 2 ? sizeof(EndScratch<THREADS, CHUNK>) : 0, MORE = LOAD ? (COLS > ENDS ? COLS : ENDS) : 0;
    __shared__ __align__(16) char pool[LISTS > MORE ? LISTS : MORE];
    __shared__ int32_t hist[LOAD ? EMAX : 1];
    __shared__ float slots[TEAMS][EMAX < GA_MAX_TOPK ? EMAX : GA_MAX_TOPK];
    const int E = la.E, k = la.k, team = threadIdx.x / L;
    const Lane<X, L, V> lane(E);
    const int ln = lane.ln;
    const int64_t w = blockIdx.x / (uint32_t)q.parts, part = blockIdx.x % (uint32_t)q.parts;
    const int64_t end = (w + 1) * a.per_worker, step = (int64_t)q.parts * TEAMS;
    int64_t t = w * a.per_worker + part * TEAMS + team;
    float acc[LOAD ? V : 1];
    double squares = 0.0;
    int tokens = 0;
    if constexpr (LOAD) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        for (int e = threadIdx.x; e < EMAX; e += THREADS) hist[e] = 0;
        __syncthreads();
    }
    // the next row is on its way, unless the registers are taken by 16 binary32 logits and sums to a lane
    constexpr bool AHEAD = !(LOAD == 1 && X == kF32 && V == 16);
    Raw<X, N> next[J];
    bool next_present = false;
    auto load = [&](int64_t t) {
        next_present = !a.mask || a.mask[t];
        lane.load(next, reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx));
    };
    if (AHEAD && t < end) load(t);
    for (; t < end; t += step) {
        float l[V], p[V];
        if (!AHEAD) load(t);
        lane.widen(next, l, next_present);
        if (AHEAD && t + step < end) load(t + step);
        uint32_t key[V], most = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = key_of(l[i]);
            most = most > key[i] ? most : key[i];
        }
        most = team_max<L>(most);
        // where all are -infinity or NaN, p is 0 or NaN
        const float top = most > kLeast ? value_of(most) : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = __builtin_amdgcn_exp2f((l[i] - top) * kLog2e);
            sum += p[i];
        }
        sum = team_sum<L>(sum);
        // the hardware's reciprocal and logarithm, each within 1 ulp
        const bool absent = sum == 0.f;
        const float inv = absent ? 0.f : __builtin_amdgcn_rcpf(sum);
        const float lse = absent ? 0.f : fmaf(__builtin_amdgcn_logf(sum), 0.693147181f, top);
        if constexpr (LOAD) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
            if (ln == 0 && !absent) {
                squares = fma((double)lse, (double)lse, squares);
                ++tokens;
            }
        }
        if (a.r.lse && ln == 0) a.r.lse[t] = lse;
        int32_t* experts = a.r.experts + t * k;
        float* gates = a.r.gates ? a.r.gates + t * k : nullptr;
        uint64_t* list = reinterpret_cast<uint64_t*>(pool) + team * EMAX;
        int found = k;
        if (a.select) {
            // A bound that at least k logits reach: the k-th of the maxima of groups of logits, found one after the
            // other.  Few groups are quick to go through, four times k of them or more leave few logits above the bound.
            uint32_t bound;
            if (4 * k <= L) bound = kth_of_groups<L, V, 1>(key, most, k);
            else if (V >= 4 && 4 * k <= 2 * L) bound = kth_of_groups<L, V, 2>(key, most, k);
            else if (V >= 8 && 4 * k <= 4 * L) bound = kth_of_groups<L, V, 4>(key, most, k);
            else bound = kth_of_groups<L, V, V>(key, most, k);
            bound = bound > kLeast ? bound : kLeast + 1u;
            int count = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) count += key[i] >= bound ? 1 : 0;
            found = team_sum<L>(count);
            int at = team_scan<L>(count) - count;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] >= bound) list[at++] = (uint64_t)key[i] << 32 | (uint32_t)~lane.column(i);
        }
        wave_fence();
        // given experts may all lie far below the largest logit: gates that sum to 1 refer to the largest of theirs
        float about = top;
        if (!a.select && normalize) {
            uint32_t best = 0u;
            for (int c = ln; c < k; c += L) {
                const int at = experts[c];
                if (at < 0 || at >= E || absent) continue;
                const uint32_t x = key_of(load_one<X>(reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx + at * kSize<X>)));
                best = best > x ? best : x;
            }
            best = team_max<L>(best);
            about = best > kLeast ? value_of(best) : 0.f;
        }
        float chosen = 0.f;
        const bool many = a.select && too_many<L>(found, k);
        if (many) {
            // one after the other: a lane's largest candidate, the team's, whose lane notes its place
            for (int j = 0; j < k; ++j) {
                uint64_t best = 0;
                int from = ln;
                for (int c = ln; c < found; c += L) {
                    const uint64_t x = list[c];
                    if ((int32_t)x < 0 && x > best) {
                        best = x;
                        from = c;
                    }
                }
                const uint32_t key = team_max<L>((uint32_t)(best >> 32));
                const uint32_t index = team_max<L>((uint32_t)(best >> 32) == key ? (uint32_t)best : 0u);
                if (best == ((uint64_t)key << 32 | index)) list[from] = (uint64_t)key << 32 | placed(index, j);
            }
        }
        for (int c = ln; c < found; c += L) {
            int rank = c, at = -1;
            float g = 0.f;
            if (a.select) {
                const uint64_t mine = list[c];
                if (many) {
                    rank = place_of((uint32_t)mine);
                } else {
                    rank = 0;
#pragma unroll 4
                    for (int j = 0; j < found; ++j) rank += list[j] > mine ? 1 : 0;
                }
                if (rank >= k) continue;
                at = index_of((uint32_t)mine);
                g = __builtin_amdgcn_exp2f((value_of((uint32_t)(mine >> 32)) - top) * kLog2e);
                experts[rank] = at;
            } else {
                at = experts[c];
                if (at < 0 || at >= E) at = -1;
                if (at >= 0 && !absent) {
                    const float x = load_one<X>(reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx + at * kSize<X>));
                    g = __builtin_amdgcn_exp2f((x - about) * kLog2e);
                }
            }
            slots[team][rank] = g;
            chosen += g;
            if (LOAD && at >= 0 && !absent) atomicAdd(&hist[at], 1);
        }
        if (a.select) {
            for (int j = found + ln; j < k; j += L) {
                slots[team][j] = 0.f;
                experts[j] = -1;
            }
        }
        wave_fence();
        if (gates) {
            float by = inv;
            if (normalize) {
                chosen = team_sum<L>(chosen);
                by = sum != sum ? sum : chosen == 0.f ? 0.f : __builtin_amdgcn_rcpf(chosen);
            }
            for (int j = ln; j < k; j += L) gates[j] = absent ? 0.f : slots[team][j] * by;
        }
        wave_fence();
    }
    if constexpr (LOAD) {
        // the wavefront's teams, then the wavefronts, in order
        float(*cols)[EMAX] = reinterpret_cast<float(*)[EMAX]>(pool);
        __shared__ double sq[(THREADS / 64)];
        __shared__ int32_t tok[(THREADS / 64)];
        const int wave = threadIdx.x >> 6;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int o = L; o < 64; o <<= 1) acc[i] += __shfl_xor(acc[i], o, 64);
            if ((threadIdx.x & 63) < L) cols[wave][lane.column(i)] = acc[i];
        }
        squares = wave_sum_f64(squares);
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) tokens += __shfl_xor(tokens, o, 64);
        if ((threadIdx.x & 63) == 0) {
            sq[wave] = squares;
            tok[wave] = tokens;
        }
        __syncthreads();
        const int64_t row = blockIdx.x;
        for (int e = threadIdx.x; e < E; e += THREADS) {
            float s = cols[0][e];
#pragma unroll
            for (int j = 1; j < (THREADS / 64); ++j) s += cols[j][e];
            q.probs[row * E + e] = s;
            q.counts[row * E + e] = hist[e];
        }
        if (threadIdx.x == 0) {
            double s = sq[0];
            int n = tok[0];
            for (int j = 1; j < (THREADS / 64); ++j) {
                s += sq[j];
                n += tok[j];
            }
            q.squares[row] = s;
            q.tokens[row] = n;
        }
    }
    if constexpr (LOAD == 2) {
        if (!last_of(q.done + 1)) return;
        auto& end_scratch = *reinterpret_cast<EndScratch<THREADS, CHUNK>*>(pool);
        end_rest(la, q, end_scratch);
        double loss = 0.0;
        for (int c = 0; c * CHUNK < E; ++c) loss += end_chunk(la, q, end_scratch, c);
        if (threadIdx.x == 0) la.load.loss[0] = (float)loss;
    }
}

// ---- backward ----------------------------------------------------------------

template <int X, int L, int V, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_route_bwd(RouteArgs a, LossArgs la, int32_t normalize, int32_t parts) {
    constexpr int TEAMS = kThreads / L, N = kVec<X>, J = V / N, EMAX = L * V;
    constexpr int SLOTS = (EMAX < GA_MAX_TOPK ? EMAX : GA_MAX_TOPK) > L ? (EMAX < GA_MAX_TOPK ? EMAX : GA_MAX_TOPK) / L : 1;
    __shared__ __align__(16) float extra[TEAMS][EMAX];
    const int E = la.E, k = la.k, team = threadIdx.x / L;
    const Lane<X, L, V> lane(E);
    const int ln = lane.ln;
    const int64_t w = blockIdx.x / (uint32_t)parts, part = blockIdx.x % (uint32_t)parts;
    const int64_t end = (w + 1) * a.per_worker, step = (int64_t)parts * TEAMS;
    int64_t t = w * a.per_worker + part * TEAMS + team;
    const float* slope = a.slope ? a.slope + (la.scope == GA_BALANCE_ALL ? 0 : w * (E + 1)) : nullptr;
    float push[V];
#pragma unroll
    for (int i = 0; i < V; ++i) push[i] = slope && lane.column(i) < E ? a.balance * slope[lane.column(i)] : 0.f;
    const float zfactor = slope ? a.z * slope[E] : 0.f;
    if (a.dgates) {
        for (int i = threadIdx.x; i < TEAMS * EMAX; i += kThreads) (&extra[0][0])[i] = 0.f;
        __syncthreads();
    }
    Raw<X, N> next[J];
    bool next_present = false;
    float next_lse = 0.f;
    auto load = [&](int64_t t) {
        next_present = !a.mask || a.mask[t];
        next_lse = a.r.lse[t];
        lane.load(next, reinterpret_cast<uint64_t>(a.x) + (uint64_t)(t * a.ldx));
    };
    if (t < end) load(t);
    for (; t < end; t += step) {
        float l[V], h[V], direct[V];
        bool present = next_present;
        const float lse = present ? next_lse : 0.f;
        lane.widen(next, l, present);
        // of the slots j = s * L + ln: the expert, and the gate's gradient
        int at[SLOTS];
        float g[SLOTS], inner = 0.f;
        if (a.dgates) {
            if (lse == 0.f) {       // perhaps of a token without an expert
                bool some = false;
#pragma unroll
                for (int i = 0; i < V; ++i) some |= l[i] != -INFINITY;
                present = team_max<L>(some ? 1u : 0u) != 0u;
            }
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int j = s * L + ln;
                at[s] = -1;
                g[s] = 0.f;
                if (j < k && present) {
                    at[s] = a.r.experts[t * k + j];
                    if (at[s] < 0 || at[s] >= E) at[s] = -1;
                    if (at[s] >= 0) g[s] = a.dgates[t * k + j];
                }
            }
            if (normalize) {
                float gate[SLOTS];
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    gate[s] = at[s] >= 0 ? a.r.gates[t * k + s * L + ln] : 0.f;
                    inner = fmaf(gate[s], g[s], inner);
                }
                inner = team_sum<L>(inner);
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) g[s] = gate[s] * (g[s] - inner);
            }
            // each slot leaves its number with its expert: where another's stands then, an expert was given twice
            bool twice = false;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (at[s] >= 0) extra[team][at[s]] = __int_as_float(s * L + ln);
            wave_fence();
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (at[s] >= 0) twice |= __float_as_int(extra[team][at[s]]) != s * L + ln;
            wave_fence();
            if (__ballot(twice) == 0ull) {
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (at[s] >= 0) extra[team][at[s]] = g[s];
            } else {
                // one slot after the other, so that they add up in their order
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (at[s] >= 0) extra[team][at[s]] = 0.f;
                wave_fence();
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const int many = k - s * L < L ? k - s * L : L;
                    for (int j = 0; j < many; ++j) {
                        if (ln == j && at[s] >= 0) extra[team][at[s]] += g[s];
                        wave_fence();
                    }
                }
            }
            wave_fence();
        }
        if (t + step < end) load(t + step);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float add = a.dgates ? extra[team][lane.column(i)] : 0.f;
            h[i] = normalize ? push[i] : push[i] + add;
            direct[i] = normalize ? add : 0.f;
            l[i] = __builtin_amdgcn_exp2f((l[i] - lse) * kLog2e);
            dot = fmaf(h[i], l[i], dot);
        }
        if (a.dgates) {
            wave_fence();
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (at[s] >= 0) extra[team][at[s]] = 0.f;
            wave_fence();
        }
        const float shift = fmaf(zfactor, lse, -team_sum<L>(dot));
        const uint64_t out = reinterpret_cast<uint64_t>(a.dx) + (uint64_t)(t * a.ldd);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float d[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int i = j * N + e;
                d[e] = present ? fmaf(l[i], h[i] + shift, direct[i]) : 0.f;
            }
            store_part<X, STREAM>(d, out, (j * L + ln) * N, E);
        }
    }
}

// ---- on the host -------------------------------------------------------------

// Calls f with the lanes of a team and the elements of a lane.  129 to 256 experts: 16 lanes forward, where a token's steps
// are what it costs (131072 x 256 binary32, 8 of them: 52 us, with 32 lanes of 8 elements 64), 32 lanes backward, whose
// registers then leave room for more wavefronts (bf16: 31 us, 41).
template <int X, bool BACKWARD, typename F>
hipError_t with_team(int E, F f) {
#define GA_TEAM(L, V) \
    if (E <= L * V) return f(std::integral_constant<int, L>{}, std::integral_constant<int, V>{})
    if constexpr (X == kF32) {
        GA_TEAM(1, 4);
        GA_TEAM(2, 4);
        GA_TEAM(4, 4);
        GA_TEAM(8, 4);
        GA_TEAM(16, 4);
    } else {
        GA_TEAM(1, 8);
        GA_TEAM(2, 8);
        GA_TEAM(4, 8);
        GA_TEAM(8, 8);
    }
    GA_TEAM(16, 8);
    if constexpr (BACKWARD) {
        GA_TEAM(32, 8);
        GA_TEAM(64, 8);
    } else {
        GA_TEAM(16, 16);
        GA_TEAM(32, 16);
    }
    GA_TEAM(64, 16);
#undef GA_TEAM
    return hipErrorInvalidValue;
}

int64_t parts_of(int64_t tokens, int teams, int64_t most) {
    int64_t p = (tokens + teams - 1) / teams;
    if (p > most) p = most;
    return p < 1 ? 1 : p;
}

// Few partial loads are added by the workgroup that ends last, in one launch.  Against two launches, us (calls one after the
// other in a graph): 64 tokens x 8 experts (1 row of partial loads) 7.3, 8.0; 2048 x 64 (64 rows) 10.9, 11.8; 512 x 128 (32) 10.7,
// 12.3; but 4096 x 64 (128) 12.9, 12.0; 65536 x 8 (256) 14.7, 10.6; 256 x 256 (16) 17.2, 14.5.
constexpr int64_t kOneRows = 64, kOneExperts = 128, kOneElements = 4096;

// Up to this many rows a workgroup of the load's end takes 64 experts, else 16: few workgroups exchange their parts of the
// loss sooner, many share long columns.  64 against 16, us, bf16: 256 x 256 (4 rows) 14.9, 15.6; 64 x 1024 (4) 14.1, 14.8;
// 1024 x 256 (16) 15.2, 15.9; 8192 x 64 (64) 13.0, 14.0; 4096 x 256 (64) 16.7, 16.3; 16384 x 64 (128) 15.8, 14.5; 8192 x 128
// (128) 17.0, 13.9; 65536 x 64 (256) 23.3, 18.7.
constexpr int64_t kWideEnd = 64;

template <int X>
hipError_t router_fwd(const Router& r, const RouteArgs& args, hipStream_t s) {
    RouteArgs a = args;
    const LossArgs la = {a.load, r.E, r.k, r.W, r.scope};
    LoadParts q = {r.d_probs, r.d_counts, r.d_squares, r.d_tokens, r.d_dots, r.d_done, 1};
    return with_team<X, false>(r.E, [&](auto lanes, auto each) {
        constexpr int L = decltype(lanes)::value, V = decltype(each)::value;
        if (!a.with_load) {
            a.per_worker = a.T;
            q.parts = (int32_t)parts_of(a.T, kThreads / L, 4096);
            hipLaunchKernelGGL((k_route<X, L, V, 0, kThreads>), dim3((unsigned)q.parts), dim3(kThreads), 0, s, a, la, q,
                               r.normalize);
            return hipGetLastError();
        }
        q.parts = (int32_t)parts_of(a.per_worker, kThreads / L, r.rows / r.W);
        if constexpr (L * V <= kOneExperts) {
            const int64_t few = (int64_t)r.W * q.parts;
            if (few <= kOneRows && few * r.E <= kOneElements) {
                hipLaunchKernelGGL((k_route<X, L, V, 2, kThreads>), dim3((unsigned)few), dim3(kThreads), 0, s, a, la, q,
                                   r.normalize);
                return hipGetLastError();
            }
        }
        q.parts = (int32_t)parts_of(a.per_worker, kLoadThreads / L, r.rows / r.W);
        const int64_t rows = (int64_t)r.W * q.parts;
        hipLaunchKernelGGL((k_route<X, L, V, 1, kLoadThreads>), dim3((unsigned)rows), dim3(kLoadThreads), 0, s, a, la, q,
                           r.normalize);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (rows <= kWideEnd)
            hipLaunchKernelGGL(k_load_end<64>, dim3((unsigned)((r.E + 63) / 64) + 1), dim3(kEndThreads), 0, s, la, q);
        else
            hipLaunchKernelGGL(k_load_end<16>, dim3((unsigned)((r.E + 15) / 16) + 1), dim3(kEndThreads), 0, s, la, q);
        return hipGetLastError();
    });
}

template <int X>
hipError_t router_bwd(const Router& r, const RouteArgs& args, hipStream_t s) {
    RouteArgs a = args;
    const LossArgs la = {a.load, r.E, r.k, r.W, r.scope};
    return with_team<X, true>(r.E, [&](auto lanes, auto each) {
        constexpr int L = decltype(lanes)::value, V = decltype(each)::value, TEAMS = kThreads / L;
        int64_t workers = r.W;
        if (r.scope == GA_BALANCE_ALL) {
            a.per_worker = a.T;
            workers = 1;
        }
        // as many workgroups as the chip holds at once
        const int64_t parts = parts_of(a.per_worker, TEAMS, (V <= 8 ? 1536 : 1024) / workers);
        // whole cache lines pass the caches by
        const int64_t row = (int64_t)r.E * kSize<X>;
        const bool stream = row % 128 == 0 && a.ldd % 128 == 0 && (reinterpret_cast<uintptr_t>(a.dx) & 127) == 0;
        if (stream)
            hipLaunchKernelGGL((k_route_bwd<X, L, V, true>), dim3((unsigned)(workers * parts)), dim3(kThreads), 0, s, a, la,
                               r.normalize, (int32_t)parts);
        else
            hipLaunchKernelGGL((k_route_bwd<X, L, V, false>), dim3((unsigned)(workers * parts)), dim3(kThreads), 0, s, a, la,
                               r.normalize, (int32_t)parts);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_router_fwd(const Router& r, const RouteArgs& a, hipStream_t s) {
    if (r.x_dtype == GA_FP32) return router_fwd<kF32>(r, a, s);
    return r.x_dtype == GA_FP16 ? router_fwd<kF16>(r, a, s) : router_fwd<kB16>(r, a, s);
}

hipError_t launch_router_bwd(const Router& r, const RouteArgs& a, hipStream_t s) {
    if (r.x_dtype == GA_FP32) return router_bwd<kF32>(r, a, s);
    return r.x_dtype == GA_FP16 ? router_bwd<kF16>(r, a, s) : router_bwd<kB16>(r, a, s);
}

}  // namespace ga
