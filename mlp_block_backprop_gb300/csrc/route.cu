// route.cu -- the router of routed experts ("Nemotron Kernels From Inference To
// Backpropagation" -- "Kernel 4: Routed ReLU2 MoE": select, execute, weight and combine;
// this is the selection and its weights): logits -> expert ids and weights, and the
// gradient of the logits.
//
//   s_e   = softmax(l)_e over the open experts (l_e > -inf), or 1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e                       (decides what is selected, nothing else)
//   kept groups: the top_groups largest sums of a group's two best keys
//   ids   = the top_k experts of the kept groups by key, ties to the lower index
//   w_j   = scale * s_j / (sum_i s_i + 1e-20), or scale * s_j without renormalising
//
//   dw -> ds_j = scale * dw_j, or scale / (S + 1e-20) * (dw_j - sum_i dw_i s_i / (S + 1e-20));
//   ds -> dl_e = ds_e s_e (1 - s_e), or s_e (ds_e - sum_j ds_j s_j)
// (renormalised: the last sum is scale sum_i dw_i s_i / (S + 1e-20) * 1e-20 / (S + 1e-20), next to nothing
// unless a bias selects scores that vanish).
//
// A warp takes a few tokens.  First, token by token (32 / L of them side by side), what is done
// for every expert: a token belongs to L = 1 .. 32 lanes, each of which holds eight
// neighbouring experts and sorts their keys once (values alone: a maximum and a minimum
// a step); a round then takes the maximum of the lanes' best, and the lowest lane that
// holds it moves up.  Then what is done for every winner, a lane a winner of all tokens together:
// which expert it was (looked up in the keys that the lanes left in shared memory), its
// weight, its distance to the next.
//
// Selection by exact order: without a bias and groups the logits themselves are the keys.
// Otherwise keys are float32 values with a known error; where two neighbours in the
// result (or the two groups on either side of the cut) are closer than that and are not
// the same logit with the same bias, the token is selected again in
// float64.  So ids do not depend on how exp rounds.
//
// Bound by instruction issue and its latencies (790 instructions a token), not by HBM: 65536 tokens of 256 experts
// (33 MB of bf16 logits, 5 us of HBM; sigmoid, 8 groups, top-8) take 60 us, the gradient 14.
#include <cuda_bf16.h>
#include <float.h>

#include "mlpblk_internal.h"

namespace mlpblk {

namespace {

constexpr int kRouteThreads = 128;
constexpr int kRouteCtas = 8;            // an SM: the calls of the float64 path would take registers from everything else
constexpr int kRouteV = 8;               // experts of a lane
constexpr float kRouteTiny = 1e-20f;
constexpr float kHalf = 0x1p-24f;        // a rounding

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t T;
    int E, k, groups, top_groups, per;   // per: experts of a group
    int sigmoid, renorm;
    float scale;
    uint32_t by_k, by_k1;                // 65536 / k and 65536 / (k + 1), rounded up
    int *ids;
    float *weights;
    // backward
    const int *ids_in;
    const float *dw;
    void *dl;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// i / d for i < 1024 and d <= 17, given 65536 / d rounded up.
__device__ __forceinline__ int over(int i, uint32_t by) { return static_cast<int>(static_cast<uint32_t>(i) * by >> 16); }

// A logit as the formulas take it: +inf counts as the largest finite value (equal shares of
// the softmax); NaN and -inf are closed (-inf).
__device__ __forceinline__ float logit_of(float l) { return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY; }

// Eight neighbouring logits of a lane; experts behind E are closed.
template <class T>
__device__ __forceinline__ void load_logits(const T *row, int e0, int E, bool vec, float (&v)[kRouteV]) {
    if (vec && e0 + kRouteV <= E) {
        if (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + e0)), b = __ldg(reinterpret_cast<const float4 *>(row + e0) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(row + e0));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) v[i] = logit_of(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) v[i] = e0 + i < E ? logit_of(to_float(row[e0 + i])) : -INFINITY;
    }
}

// Sum and maximum over the L lanes of a token.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    if constexpr (L == 32) {
        float r;
        asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    } else {
#pragma unroll
        for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
template <int L, class F>
__device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / (1 + exp(-x)), for keys.
__device__ __forceinline__ float quick_sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

__device__ __forceinline__ void order_pair(float &a, float &b) {
    const float x = fmaxf(a, b), y = fminf(a, b);
    a = x;
    b = y;
}

// Eight keys into descending order (Batcher's odd-even merge sort: 19 comparisons).
__device__ __forceinline__ void sort8(float (&v)[kRouteV]) {
    order_pair(v[0], v[1]); order_pair(v[2], v[3]); order_pair(v[4], v[5]); order_pair(v[6], v[7]);
    order_pair(v[0], v[2]); order_pair(v[1], v[3]); order_pair(v[4], v[6]); order_pair(v[5], v[7]);
    order_pair(v[1], v[2]); order_pair(v[5], v[6]);
    order_pair(v[0], v[4]); order_pair(v[1], v[5]); order_pair(v[2], v[6]); order_pair(v[3], v[7]);
    order_pair(v[2], v[4]); order_pair(v[3], v[5]);
    order_pair(v[1], v[2]); order_pair(v[3], v[4]); order_pair(v[5], v[6]);
}

// first, second: the two best of a group so far; joined with another two.
__device__ __forceinline__ void join_two(float &first, float &second, float a, float b) {
    second = fmaxf(fmaxf(second, b), fminf(first, a));
    first = fmaxf(first, a);
}
__device__ __forceinline__ void join_two(double &first, double &second, double a, double b) {
    const double low = first < a ? first : a;
    first = first < a ? a : first;
    second = second < b ? b : second;
    second = second < low ? low : second;
}
// A group's mark from its two best keys, half their sum (which may leave float32's range): -inf where it has no open expert.
template <class F>
__device__ __forceinline__ F mark_of(F first, F second) {
    return second > -INFINITY ? F(0.5) * first + F(0.5) * second : F(0.5) * first;
}

// Is group g among the best?  marks in shared memory, `stride` apart; ties to the lower group.
template <class F>
__device__ __forceinline__ bool group_kept(const F *marks, int stride, int groups, int top_groups, int g) {
    const F m = marks[g * stride];
    int before = 0;
    for (int h = 0; h < groups; ++h) {
        const F o = marks[h * stride];
        before += o > m || (o == m && h < g);
    }
    return before < top_groups;
}

// What a warp keeps in shared memory: the keys of its N tokens by expert, the lanes' sorted keys,
// the winners' values and lanes, and the winners; instead of the sorted keys, float64 keys and
// marks of tokens that are selected again.
template <int L, int N_>
struct alignas(16) RouteWarp {   // (keys move four at a time)
    static constexpr int N = N_, E = L * kRouteV, S = MLPBLK_ROUTE_MAX_TOP_K + 1;
    float keys[N][E];
    union {
        float queue[N * L / 32][32][kRouteV + 1];
        struct {
            int64_t key[L * kRouteV];
            double mark[64];
            int list[L * kRouteV];
        } exact;
    };
    float top[N][S], most[N], z[N], m[N];
    int lane[N][S], won[N][S];
};

// The score of a logit x, given the softmax's maximum and one over its sum.
__device__ __forceinline__ float score_of(bool sigmoid, float x, float m, float inv_z) {
    return sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - m) * inv_z;
}

// The float64 path is rare (one token in a thousand), but a token that takes it late ends the kernel late: an exp
// in float64 takes a warp the better part of a microsecond, whether for one lane or for all, so a
// whole warp selects one token, and only the experts that come into question are computed.  Its code is
// kept short: the first run on an SM fetches it.
__device__ __noinline__ double exact_exp(double x) { return exp(x); }

// A key from a logit; z: the softmax's sum, m its largest logit.
__device__ __noinline__ double exact_key(bool sigmoid, float l, float bias, float m, double z) {
    const double x = logit_of(l);
    const double e = exact_exp(sigmoid ? -x : x - m);
    return (sigmoid ? 1.0 : e) / (sigmoid ? 1.0 + e : z) + bias;
}

// An integer that orders as a double does (-0 as 0); INT64_MIN is below all.
__device__ __forceinline__ int64_t ordered(double x) {
    const int64_t b = __double_as_longlong(x + 0.0);
    return b < 0 ? b ^ INT64_MAX : b;
}

// Selects one token again, in float64, into won[]: among every open expert if its groups are in
// doubt (regroup), else among those of `keys`, the float32 keys, that are not below `least`.
// The whole warp takes one token.
template <class T, class W>
__device__ __noinline__ void route_exactly(const RouteArgs &a, const T *row, bool regroup, float least, const float *keys, W &w, int *won) {
    const unsigned all = 0xffffffffu;
    const int lane = threadIdx.x % 32;
    int64_t *key = w.exact.key;      // of the candidates, in the experts' order
    int *list = w.exact.list;
    const int chunks = (a.E + 31) / 32;
    int n = 0;
    float m = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
        const int e = 32 * i + lane;
        const float l = e < a.E ? logit_of(to_float(row[e])) : -INFINITY;
        const bool open = l > -INFINITY && !(a.bias && !(a.bias[e] > -INFINITY));
        const bool in = open && (regroup || (keys[e] > -INFINITY && keys[e] >= least));
        const unsigned votes = __ballot_sync(all, in);
        if (in) list[n + __popc(votes & ((1u << lane) - 1u))] = e;
        n += __popc(votes);
        m = fmaxf(m, l);
    }
    m = lanes_max<32>(m);
    if (!(m > -INFINITY)) m = 0.0f;
    double inv_z = 0.0;
    if (!a.sigmoid) {
        double z = 0.0;
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
            const int e = 32 * i + lane;
            if (e >= a.E) continue;
            const double x = exact_exp(static_cast<double>(logit_of(to_float(row[e]))) - m);
            z += x;
            key[e] = __double_as_longlong(x);    // by expert, until the candidates' keys take the place
        }
        inv_z = 1.0 / lanes_sum<32>(z);
    }
    __syncwarp();
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += 32) {
        const int c = c0 + lane, e = c < n ? list[c] : 0;
        const float bias = a.bias ? a.bias[e] : 0.0f;
        const double x = a.sigmoid ? exact_key(true, to_float(row[e]), bias, 0.0f, 0.0) : __longlong_as_double(key[e]) * inv_z + bias;
        __syncwarp();                            // (a candidate's place is not behind its expert's)
        if (c < n) key[c] = ordered(x);
        __syncwarp();
    }
    if (regroup) {
        // two best a group, in its run of the list; then the marks' order
        double *mark = w.exact.mark;
#pragma unroll 1
        for (int g = lane; g < a.groups; g += 32) {
            int64_t first = INT64_MIN, second = INT64_MIN;
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
                if (list[c] < g * a.per || list[c] >= (g + 1) * a.per) continue;
                const int64_t x = key[c];
                second = x > first ? first : (x > second ? x : second);
                first = x > first ? x : first;
            }
            const double p = __longlong_as_double(first < 0 ? first ^ INT64_MAX : first), q = __longlong_as_double(second < 0 ? second ^ INT64_MAX : second);
            mark[g] = first == INT64_MIN ? -INFINITY : (second == INT64_MIN ? p : p + q);
        }
        __syncwarp();
        uint64_t groups = 0;
#pragma unroll 1
        for (int g = lane; g < a.groups; g += 32)
            if (group_kept(mark, 1, a.groups, a.top_groups, g)) groups |= 1ull << g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) groups |= __shfl_xor_sync(all, groups, o);
#pragma unroll 1
        for (int c = lane; c < n; c += 32) {
            const int e = list[c];
            if (!(groups >> (e / a.per) & 1)) key[c] = INT64_MIN;
            else if (a.bias == nullptr) key[c] = ordered(logit_of(to_float(row[e])));   // by logit within the groups
        }
        __syncwarp();
    }
    // the list's order is the experts'
    if (n <= 32) {                               // a lane a candidate: each counts those before it
        const int64_t mine = lane < n ? key[lane] : INT64_MIN;
        int rank = 0;
#pragma unroll 1
        for (int c = 0; c < n; ++c) {
            const int64_t y = __shfl_sync(all, mine, c);
            rank += y > mine || (y == mine && c < lane);
        }
        const int live = __popc(__ballot_sync(all, mine > INT64_MIN));
        if (mine > INT64_MIN && rank < a.k) won[rank] = list[lane];
        if (lane >= live && lane < a.k) won[lane] = -1;
        __syncwarp();
        return;
    }
    // rounds of the best
#pragma unroll 1
    for (int r = 0; r < a.k; ++r) {
        int64_t top = INT64_MIN;
        int at = n;
#pragma unroll 1
        for (int c = lane; c < n; c += 32)
            if (key[c] > top) top = key[c], at = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_xor_sync(all, top, o);
            const int f = __shfl_xor_sync(all, at, o);
            if (y > top || (y == top && f < at)) top = y, at = f;
        }
        if (lane == 0) {
            won[r] = at < n ? list[at] : -1;
            if (at < n) key[at] = INT64_MIN;
        }
        __syncwarp();
    }
}

// What the roundings of the scores may move between two keys (or two marks, half the sum of two keys each), given the
// largest score: 2 x 3.4 u of it (route_kernel says whence), and of the softmax 20 u of the scores' difference for the
// common sum (12 additions, its terms' own errors and the quotient).
__device__ __forceinline__ float score_slack(bool sigmoid, float most) { return (sigmoid ? 8.0f : 28.0f) * kHalf * most; }

// How far a mark may be off by the roundings of its keys' sums with the bias, its own and that of a bound mark -+ off: 3 u of
// half the keys' magnitudes, which are more than the mark's where the keys have opposite signs.  Infinite ones are exact.
__device__ __forceinline__ float mark_off(float first, float second, float mark) {
    if (!(fabsf(mark) < INFINITY)) return 0.0f;
    return 2.5f * kHalf * fabsf(first) + (second > -INFINITY ? 2.5f * kHalf * fabsf(second) : 0.0f);
}

// Groups of whole lanes whose marks lie too near the cut: settles which of them stay, in float64, from the
// experts that may be their two best.  A token belongs to L lanes, a group to `span` of them; mark, off,
// second, kept: the group's; low, high: the least bound mark - off that is kept, the largest mark + off that is not; returns
// whether the lane's group stays.  The whole warp calls it; tokens that are not `close` keep what they have.
template <class T, int L>
__device__ __noinline__ bool settle_groups(const RouteArgs &a, const T *row, const float *key, float second, float mark, float off, bool kept,
                                           float low, float high, float slack, bool close, int span) {
    const unsigned all = 0xffffffffu;
    const int sub = threadIdx.x % L, e0 = sub * kRouteV, lane0 = threadIdx.x % 32 / L * L;
    const unsigned mine = L == 32 ? all : ((1u << (L % 32)) - 1u) << lane0;
    const bool doubt = close && mark > -INFINITY && (kept ? mark - off <= high + slack : mark + off >= low - slack);
    const float least = second - (slack + 4.0f * kHalf * fabsf(second));   // of the keys that may be second best
    uint32_t which = 0;
#pragma unroll 1
    for (int i = 0; i < kRouteV; ++i)
        if (doubt && key[i] > -INFINITY && key[i] >= least) which |= 1u << i;
    float m = -INFINITY;
    double z = 0.0;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int i = 0; i < kRouteV; ++i) m = fmaxf(m, e0 + i < a.E ? logit_of(to_float(row[e0 + i])) : -INFINITY);
        m = lanes_max<L>(m);
#pragma unroll 1
        for (int i = 0; i < kRouteV; ++i)
            z += e0 + i < a.E && m > -INFINITY ? exact_exp(static_cast<double>(logit_of(to_float(row[e0 + i]))) - m) : 0.0;
        z = lanes_sum<L>(z);
    }
    double first64 = -INFINITY, second64 = -INFINITY;
#pragma unroll 1
    while (__any_sync(all, which != 0)) {
        if (which != 0) {
            const int e = e0 + __ffs(which) - 1;
            join_two(first64, second64, exact_key(a.sigmoid, to_float(row[e]), a.bias ? a.bias[e] : 0.0f, m, z), static_cast<double>(-INFINITY));
            which &= which - 1;
        }
    }
#pragma unroll 1
    for (int o = 1; o < span; o <<= 1) {
        const double x = __shfl_xor_sync(all, first64, o), y = __shfl_xor_sync(all, second64, o);
        join_two(first64, second64, x, y);
    }
    double mark64 = doubt ? mark_of(first64, second64) : -INFINITY;
    bool stays = kept && !doubt;
    const int left = a.top_groups - __popc(__ballot_sync(all, stays && sub % span == 0) & mine);
#pragma unroll 1
    for (int r = 0; r < a.top_groups; ++r) {
        double top = mark64;
#pragma unroll 1
        for (int o = 1; o < L; o <<= 1) {
            const double y = __shfl_xor_sync(all, top, o);
            top = y > top ? y : top;
        }
        const int owner = __ffs(__ballot_sync(all, mark64 == top) & mine) - 1 - lane0;
        if (r < left && top > -INFINITY && (owner & -span) == (sub & -span)) {
            stays = true;
            mark64 = -INFINITY;
        }
    }
    return stays;
}

// KEYED: the logits alone do not decide (a bias, or groups of which some are dropped).
// N: tokens of a warp.
template <class T, int L, int N, bool KEYED>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas)
route_kernel(const RouteArgs a) {
    using W = RouteWarp<L, N>;
    constexpr int kSide = 32 / L, kSteps = N / kSide;   // tokens of a step
    __shared__ W shared[kRouteThreads / 32];
    griddep_enter();
    W &w = shared[threadIdx.x / 32];
    const int lane = threadIdx.x % 32, sub = lane % L, seat = lane / L;
    const unsigned all = 0xffffffffu;
    const int lane0 = seat * L;                   // the token's first lane
    const unsigned mine = L == 32 ? all : ((1u << (L % 32)) - 1u) << lane0;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + threadIdx.x / 32) * N;
    if (t0 >= a.T) return;
    const T *rows = static_cast<const T *>(a.logits);
    const int e0 = sub * kRouteV;
    const bool vec = (a.E * sizeof(T)) % 16 == 0;
    const bool grouped = KEYED && a.top_groups < a.groups;
    const bool by_logit = !KEYED || a.bias == nullptr;   // the scores' order is the logits'
    const int rounds = by_logit ? a.k : a.k + 1;    // the next one, to see whether the last is clear
    const uint32_t by_rounds = by_logit ? a.by_k : a.by_k1;
    // Groups: a lane's experts belong to one group where a group is a power of two of lanes;
    // then two shuffles a step find its two best keys, and rounds of the best mark keep groups.
    const int span = a.per / kRouteV;               // lanes of a group
    const bool whole = a.per % kRouteV == 0 && (span & (span - 1)) == 0;
    float bias[kRouteV];
    if (KEYED) {
#pragma unroll
        for (int i = 0; i < kRouteV; ++i)           // (NaN becomes -inf: a NaN among the keys would win no round)
            bias[i] = !by_logit && e0 + i < a.E ? fmaxf(__ldg(a.bias + e0 + i), -INFINITY) : 0.0f;
    }
    unsigned again = 0, regroup = 0;                // tokens of the warp to select again, and their groups too

#pragma unroll 1
    for (int step = 0; step < kSteps; ++step) {
        const int at = step * kSide, n = at + seat;
        const int64_t t = min(t0 + n, a.T - 1);     // (behind the last token: the last again, not stored)
        float l[kRouteV], key[kRouteV];
        load_logits(rows + t * a.E, e0, a.E, vec, l);
        float m = 0.0f, inv_z = 1.0f;               // softmax: the largest logit, one over the sum
        if (!a.sigmoid) {
            m = l[0];
#pragma unroll
            for (int i = 1; i < kRouteV; ++i) m = fmaxf(m, l[i]);
            m = lanes_max<L>(m);
            if (!(m > -INFINITY)) m = 0.0f;
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < kRouteV; ++i) {
                key[i] = expf(l[i] - m);
                z += key[i];
            }
            z = lanes_sum<L>(z);
            inv_z = z > 0.0f ? 1.0f / z : 0.0f;
        }
        // Keys, and how far they may be off (u = 2^-24).  Sigmoid: ex2.approx 4 u of e and its
        // argument |x| u, both times s (1 - s) (1/4 at most; |x| s (1 - s) 0.23 at most), 1 + e u, the
        // reciprocal 2 u: 3.3 u.  Softmax: exp 2 u, its argument |l - m| u times s / max s (1/e at
        // most), the product u: 3.4 u of the largest score, and a sum whose roundings
        // move all scores alike (score_slack).  The sum with the bias u of the key.
        const float most = a.sigmoid ? 1.0f : inv_z;
        if (KEYED) {
#pragma unroll
            for (int i = 0; i < kRouteV; ++i) {
                const float x = a.sigmoid ? quick_sigmoid(l[i]) : key[i] * inv_z;
                key[i] = l[i] > -INFINITY ? x + bias[i] : -INFINITY;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRouteV; ++i) key[i] = l[i];
        }
        bool close = false;
        if (grouped) {
            uint32_t kept = 0;                      // of the lane's eight, those in kept groups
            float low, high;                        // bounds of the least mark that is kept, of the best that is not
            const float slack = score_slack(a.sigmoid, most);
            if (whole) {
                float first = fmaxf(key[0], key[1]), second = fminf(key[0], key[1]);
#pragma unroll
                for (int i = 2; i < kRouteV; i += 2) join_two(first, second, fmaxf(key[i], key[i + 1]), fminf(key[i], key[i + 1]));
                for (int o = 1; o < span; o <<= 1) {
                    const float x = __shfl_xor_sync(all, first, o), y = __shfl_xor_sync(all, second, o);
                    join_two(first, second, x, y);
                }
                const float own = mark_of(first, second), off = mark_off(first, second, own);
                float mark = own;
                // (the best mark's lowest group: no lane before the group's first has it)
                const unsigned before = mine & ((1u << (lane0 + (sub & -span))) - 1u);
                for (int r = 0; r < a.top_groups; ++r) {
                    const float best = lanes_max<L>(mark);
                    const unsigned votes = __ballot_sync(all, mark == best);
                    if (mark == best && (votes & before) == 0) {
                        // (a group without an open expert may be kept too: it has nothing to select)
                        kept = 0xFFu;
                        mark = -INFINITY;
                    }
                }
                low = -lanes_max<L>(kept != 0 ? off - own : -INFINITY);
                high = lanes_max<L>(kept != 0 ? -INFINITY : own + off);
                const bool doubt = high > -INFINITY && low < INFINITY && low - high <= slack;
                if (__any_sync(all, doubt)) {
                    float copy[kRouteV];
#pragma unroll
                    for (int i = 0; i < kRouteV; ++i) copy[i] = key[i];
                    kept = settle_groups<T, L>(a, rows + t * a.E, copy, second, own, off, kept != 0, low, high, slack, doubt, span) ? 0xFFu : 0u;
                }
                if (by_logit) {
#pragma unroll
                    for (int i = 0; i < kRouteV; ++i) key[i] = l[i];
                }
                if (kept == 0) {
#pragma unroll
                    for (int i = 0; i < kRouteV; ++i) key[i] = -INFINITY;
                }
            } else {
                float *keys = w.keys[n], *marks = keys;   // a mark at its group's first expert's place
#pragma unroll
                for (int i = 0; i < kRouteV; ++i) keys[e0 + i] = key[i];
                __syncwarp();
                for (int g = sub; g < a.groups; g += L) {
                    float first = -INFINITY, second = -INFINITY;
                    for (int i = 0; i < a.per; ++i) join_two(first, second, keys[g * a.per + i], -INFINITY);
                    const float own = mark_of(first, second);
                    marks[g * a.per] = own;         // (no other lane reads this group)
                    if (a.per > 1) marks[g * a.per + 1] = mark_off(first, second, own);
                }
                __syncwarp();
                // each lane settles some groups; a vote tells all of them
                low = INFINITY, high = -INFINITY;
                uint64_t groups = 0;
                for (int g0 = 0; g0 < a.groups; g0 += L) {
                    const int g = g0 + sub;
                    const bool on = g < a.groups && group_kept(marks, a.per, a.groups, a.top_groups, g);
                    if (g < a.groups) {
                        const float x = marks[g * a.per], off = a.per > 1 ? marks[g * a.per + 1] : mark_off(2.0f * x, -INFINITY, x);
                        if (on) low = fminf(low, x - off);
                        else high = fmaxf(high, x + off);
                    }
                    groups |= static_cast<uint64_t>((__ballot_sync(all, on) & mine) >> lane0) << g0;
                }
                low = -lanes_max<L>(-low);
                high = lanes_max<L>(high);
                close = high > -INFINITY && low < INFINITY && low - high <= slack;
#pragma unroll
                for (int i = 0; i < kRouteV; ++i) {
                    if (by_logit) key[i] = l[i];
                    if (!(groups >> min((e0 + i) / a.per, 63) & 1)) key[i] = -INFINITY;
                }
                __syncwarp();
            }
        }
        *reinterpret_cast<float4 *>(w.keys[n] + e0) = make_float4(key[0], key[1], key[2], key[3]);
        *reinterpret_cast<float4 *>(w.keys[n] + e0 + 4) = make_float4(key[4], key[5], key[6], key[7]);
        sort8(key);
        // the lane's sorted keys, then none (nine a lane: the lanes' heads lie in 32 banks)
        float *queue = w.queue[step][lane];
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) queue[i] = key[i];
        queue[kRouteV] = -INFINITY;
        if (sub == 0) {
            w.most[n] = most;
            w.m[n] = m;
            w.z[n] = inv_z;
        }
        const unsigned votes = KEYED ? __ballot_sync(all, close) : 0u;
        if (votes != 0) {
#pragma unroll
            for (int i = 0; i < kSide; ++i) regroup |= (votes >> (i * L) & 1u) << (at + i);
        }
        __syncwarp();
    }
    // The steps' rounds side by side: each waits for its maximum, not for the others'.
    const float *queue[kSteps];
    float head[kSteps];                             // the best of the lane's keys that are left
    const unsigned before = mine & ((1u << lane) - 1u);
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
        queue[step] = w.queue[step][lane];
        head[step] = *queue[step];
    }
    for (int r = 0; r < rounds; ++r) {
        float best[kSteps];
#pragma unroll
        for (int step = 0; step < kSteps; ++step) best[step] = lanes_max<L>(head[step]);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            const unsigned votes = __ballot_sync(all, head[step] == best[step]);
            if (head[step] == best[step] && (votes & before) == 0) {   // the lowest lane that has it
                w.top[step * kSide + seat][r] = best[step];
                w.lane[step * kSide + seat][r] = sub;
                if (best[step] > -INFINITY) head[step] = *++queue[step];
            }
        }
    }
    __syncwarp();

    // which of its lane's eight a winner was: equal keys of a lane went in order
    for (int i = lane; i < N * rounds; i += 32) {
        const int n = over(i, by_rounds), r = i - n * rounds;
        const float top = w.top[n][r];
        const int owner = w.lane[n][r];
        int skip = 0;
        for (int q = r - 1; q >= 0 && w.top[n][q] == top; --q) skip += w.lane[n][q] == owner;
        const float4 k0 = *reinterpret_cast<const float4 *>(w.keys[n] + owner * kRouteV), k1 = *reinterpret_cast<const float4 *>(w.keys[n] + owner * kRouteV + 4);
        uint32_t equal = (k0.x == top) | (k0.y == top) << 1 | (k0.z == top) << 2 | (k0.w == top) << 3 | (k1.x == top) << 4 |
                         (k1.y == top) << 5 | (k1.z == top) << 6 | (k1.w == top) << 7;
        for (; skip > 0; --skip) equal &= equal - 1;
        w.won[n][r] = top > -INFINITY ? owner * kRouteV + __ffs(equal) - 1 : -1;
    }
    __syncwarp();
    if (KEYED) {
        if (!by_logit) {
            // Neighbours that float32 cannot tell apart: near, or the same numbers (equal then, in order of
            // their experts).  What float32 may be off: two keys and, of the softmax, what the common sum
            // does to the scores' difference (at the cut the other one stands for everything below it, so
            // for the largest score); u of each key for its sum with the bias.
            enum : int { kApart = 0, kNear = 1, kSame = 2 };
            auto reach = [&](int n, float x, float y) {
                return score_slack(a.sigmoid, w.most[n]) + 2.0f * kHalf * (fabsf(x) + fabsf(y));
            };
            bool any = false;
            for (int i = lane; i < N * a.k; i += 32) {
                const int n = over(i, a.by_k), r = i - n * a.k;
                const int e = w.won[n][r], f = w.won[n][r + 1];
                int state = kApart;
                if (f >= 0 && t0 + n < a.T) {
                    const float ke = w.top[n][r], kf = w.top[n][r + 1];
                    if (ke < INFINITY && ke - kf <= reach(n, ke, kf)) {
                        const T *row = rows + (t0 + n) * a.E;
                        state = logit_of(to_float(row[e])) != logit_of(to_float(row[f])) || __ldg(a.bias + e) != __ldg(a.bias + f) ? kNear : kSame;
                    }
                }
                w.lane[n][r] = state;               // (the winners' lanes have been used)
                any |= state == kNear || (state == kSame && r + 1 == a.k);
            }
            if (__any_sync(all, any)) {
                __syncwarp();
                unsigned cut = 0;                   // tokens whose cut goes through experts of the same numbers
                for (int i0 = 0; i0 < N * a.k; i0 += 32) {
                    const int i = min(i0 + lane, N * a.k - 1), n = over(i, a.by_k), r = i - n * a.k;
                    const bool end = r + 1 == a.k;
                    const int state = i == i0 + lane ? w.lane[n][r] : kApart;
                    if (state == kSame && end) cut |= 1u << n;
                    // a pair by itself is settled here, its second key by the next lane
                    const bool alone = a.sigmoid && !end && (r == 0 || w.lane[n][r - 1] == kApart) && w.lane[n][min(r + 1, a.k - 1)] == kApart;
                    const bool pair = state == kNear && alone;
                    if (state == kNear && !alone) again |= 1u << n;   // more than two, or what was not selected
                    const unsigned pairs = __ballot_sync(all, pair);
                    if (pairs == 0) continue;
                    const T *row = rows + (t0 + n) * a.E;
                    auto key_of = [&](int e) { return exact_key(true, to_float(row[e]), a.bias[e], 0.0f, 0.0); };
                    const int e = w.won[n][r];
                    double x = 0.0;
                    if (pair || (pairs << 1 >> lane & 1u)) x = key_of(e);
                    double y = __shfl_down_sync(all, x, 1);
                    if (!pair) continue;
                    const int f = w.won[n][r + 1];
                    if (lane == 31) y = key_of(f);
                    if (y > x || (y == x && f < e)) {
                        w.won[n][r] = f;
                        w.won[n][r + 1] = e;
                    }
                }
                // behind those, there may be others that are near
                for (cut = __reduce_or_sync(all, cut); cut != 0; cut &= cut - 1) {
                    const int n = __ffs(cut) - 1, e = w.won[n][a.k];
                    const T *row = rows + (t0 + n) * a.E;
                    const float ke = w.top[n][a.k], l = logit_of(to_float(row[e])), b = __ldg(a.bias + e);
                    for (int f = lane; f < a.E; f += 32) {
                        const float kf = w.keys[n][f];
                        if (fabsf(kf - ke) <= reach(n, ke, ke) && (logit_of(to_float(row[f])) != l || __ldg(a.bias + f) != b)) again |= 1u << n;
                    }
                }
            }
        }
        again = __reduce_or_sync(all, again) | regroup;
        if (again != 0) {
            __syncwarp();
            for (; again != 0; again &= again - 1) {
                const int n = __ffs(again) - 1;
                if (t0 + n >= a.T) break;
                float least = -INFINITY;
                if (!by_logit && w.won[n][a.k] >= 0) least = w.top[n][a.k] - kHalf * (32.0f * w.most[n] + 8.0f * fabsf(w.top[n][a.k]));
                route_exactly(a, rows + (t0 + n) * a.E, regroup >> n & 1, least, w.keys[n], w, w.won[n]);
            }
        }
        __syncwarp();
    }
    // weights, from the logits of the selected
    for (int i = lane; i < N * a.k; i += 32) {
        const int n = over(i, a.by_k), r = i - n * a.k;
        const int e = w.won[n][r];
        w.top[n][r] = e >= 0 && t0 + n < a.T ? score_of(a.sigmoid, logit_of(to_float(rows[(t0 + n) * a.E + e])), w.m[n], w.z[n]) : 0.0f;
    }
    __syncwarp();
    for (int i = lane; i < N * a.k; i += 32) {
        const int n = over(i, a.by_k), r = i - n * a.k;
        if (t0 + n >= a.T) break;
        float x = w.top[n][r];
        if (a.renorm) {
            float total = 0.0f;
            for (int q = 0; q < a.k; ++q) total += w.top[n][q];
            x = x / (total + kRouteTiny);
        }
        a.ids[t0 * a.k + i] = w.won[n][r];
        a.weights[t0 * a.k + i] = a.scale * x;
    }
}

template <class T>
__device__ __forceinline__ void store_logits(T *row, int e0, int E, bool vec, const float (&v)[kRouteV]) {
    if (vec && e0 + kRouteV <= E) {
        if (sizeof(T) == 4) {
            float4 *p = reinterpret_cast<float4 *>(row + e0);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w[i]) : "f"(v[2 * i]), "f"(v[2 * i + 1]));
            *reinterpret_cast<uint4 *>(row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kRouteV; ++i)
            if (e0 + i < E) row[e0 + i] = static_cast<T>(v[i]);
    }
}

// A token's gradient: first what concerns its winners, a lane a winner of all the warp's tokens
// together, then the rows, in which their terms meet what every expert gets.
template <int L, int N_>
struct alignas(16) RouteBackWarp {
    static constexpr int N = N_, S = L * kRouteV < MLPBLK_ROUTE_MAX_TOP_K ? L * kRouteV : MLPBLK_ROUTE_MAX_TOP_K;
    float row[32 * kRouteV];
    float m[N], z[N], total[N], dot[N];
    int id[N][S];
    float s[N][S], slope[N][S], w[N][S];
};

template <class T, int L, int N>
__global__ void __launch_bounds__(kRouteThreads)
route_bwd_kernel(const RouteArgs a) {
    using W = RouteBackWarp<L, N>;
    constexpr int kSide = 32 / L;
    __shared__ W shared[kRouteThreads / 32];
    griddep_enter();
    W &w = shared[threadIdx.x / 32];
    const int lane = threadIdx.x % 32, sub = lane % L, seat = lane / L;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + threadIdx.x / 32) * N;
    if (t0 >= a.T) return;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(N), a.T - t0));
    const T *rows = static_cast<const T *>(a.logits);
    const bool vec = (a.E * sizeof(T)) % 16 == 0;
    const int e0 = sub * kRouteV;
    const bool softmax = !a.sigmoid;
    if (softmax) {
#pragma unroll 1
        for (int at = 0; at < N; at += kSide) {
            float l[kRouteV];
            load_logits(rows + min(t0 + at + seat, a.T - 1) * a.E, e0, a.E, vec, l);
            float m = l[0];
#pragma unroll
            for (int i = 1; i < kRouteV; ++i) m = fmaxf(m, l[i]);
            m = lanes_max<L>(m);
            if (!(m > -INFINITY)) m = 0.0f;
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < kRouteV; ++i) z += expf(l[i] - m);
            z = lanes_sum<L>(z);
            if (sub == 0) {
                w.m[at + seat] = m;
                w.z[at + seat] = z > 0.0f ? 1.0f / z : 0.0f;
            }
        }
        __syncwarp();
    }
    // scores, and their derivative by their own logit
    for (int i = lane; i < tokens * a.k; i += 32) {
        const int n = over(i, a.by_k), r = i - n * a.k;
        int e = a.ids_in[t0 * a.k + i];
        const float x = e >= 0 && e < a.E ? logit_of(to_float(rows[(t0 + n) * a.E + e])) : -INFINITY;
        float s = 0.0f, slope = 0.0f;
        if (x > -INFINITY) {
            if (softmax) {
                s = expf(x - w.m[n]) * w.z[n];
                slope = s;
            } else {
                const float g = expf(-fabsf(x)), q = 1.0f / (1.0f + g);
                s = x >= 0.0f ? q : g * q;
                slope = g * q * q;               // s (1 - s), without a difference
            }
        } else {
            e = -1;
        }
        w.id[n][r] = e;
        w.s[n][r] = s;
        w.slope[n][r] = slope;
        w.w[n][r] = e >= 0 ? a.dw[t0 * a.k + i] : 0.0f;   // (what stands beside no expert may be NaN)
    }
    __syncwarp();
    // sum_i s_i and sum_i dw_i s_i
    for (int n = lane; n < tokens; n += 32) {
        float total = 0.0f, dot = 0.0f;
        for (int r = 0; r < a.k; ++r) {
            total += w.s[n][r];
            dot += w.w[n][r] * w.s[n][r];
        }
        total += kRouteTiny;
        w.total[n] = total;
        w.dot[n] = a.renorm ? dot / total : dot;
    }
    __syncwarp();
    // each winner's term (the first slot that names an expert takes the others' along, in order)
    for (int i = lane; i < tokens * a.k; i += 32) {
        const int n = over(i, a.by_k), r = i - n * a.k;
        const int e = w.id[n][r];
        const float dot = a.renorm ? w.dot[n] : 0.0f;
        float sum = 0.0f;
        bool first = e >= 0;
        for (int q = 0; q < a.k; ++q) {
            if (w.id[n][q] != e) continue;
            if (q < r) first = false;
            sum += w.w[n][q] - dot;
        }
        if (a.renorm) sum = sum / w.total[n];
        w.s[n][r] = first ? a.scale * sum * w.slope[n][r] : 0.0f;
    }
#pragma unroll 1
    for (int at = 0; at < N; at += kSide) {
        const int n = at + seat;
        if (__all_sync(0xffffffffu, n >= tokens)) break;
        float out[kRouteV];
        float4 *mine = reinterpret_cast<float4 *>(w.row + lane * kRouteV);
        mine[0] = mine[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncwarp();
        if (n < tokens) {
            for (int r = sub; r < a.k; r += L) {
                const float ds = w.s[n][r];
                const int e = w.id[n][r];
                if (ds != 0.0f) w.row[seat * L * kRouteV + e] = ds;   // (NaN and infinities too)
            }
        }
        __syncwarp();
        const float4 o0 = mine[0], o1 = mine[1];
        out[0] = o0.x; out[1] = o0.y; out[2] = o0.z; out[3] = o0.w;
        out[4] = o1.x; out[5] = o1.y; out[6] = o1.z; out[7] = o1.w;
        if (softmax && n < tokens) {
            // s (ds - sum_j ds_j s_j): the first part stands in `out`
            const float part = a.renorm ? kRouteTiny / w.total[n] : 1.0f, mean = a.scale * w.dot[n] * part;
            // (renormalised it is mostly far below the roundings of dw - dot, and left out: 65536 tokens of
            // 256 experts 34 us with it, 26 without; a NaN is not)
            if (mean != 0.0f && !(part < 0x1p-60f && fabsf(mean) < INFINITY)) {
                const float m = w.m[n], z = w.z[n];
                float l[kRouteV];
                load_logits(rows + (t0 + n) * a.E, e0, a.E, vec, l);
#pragma unroll
                for (int i = 0; i < kRouteV; ++i) out[i] -= expf(l[i] - m) * z * mean;
            }
        }
        if (n < tokens) store_logits(static_cast<T *>(a.dl) + (t0 + n) * a.E, e0, a.E, vec, out);
        __syncwarp();
    }
}

// Tokens a warp: as many as its lanes hold side by side, more where that still leaves the SMs full
// of warps (the winners' part then fills the lanes; with few tokens it costs parallelism: 8 tokens
// of 256 experts 3.6 us, and 8.3 with four a warp), and two steps of those where a step has one token or
// two (65536 of 256 experts 63 us, one step 74, four 66; of 128 19.8, 23.5 and 23.6; of 60 20.3, two steps 24.4;
// the gradient, at least four tokens a warp: 20000 tokens of 256 experts 6.1 us, two 6.6, eight 9.8; 65536 14.3, 17.6, 15.2).
template <class T, int L>
int run_route(const RouteArgs &a, bool backward, int sms, cudaStream_t s) {
    constexpr int kSide = 32 / L, kWarps = kRouteThreads / 32;
    constexpr int kMany = kSide <= 2 ? 2 * kSide : kSide, kManyBack = kSide < 4 ? 4 : kSide;
    const bool many = a.T >= static_cast<int64_t>(sms) * 64 * kSide;
    const int n = kWarps * (many ? (backward ? kManyBack : kMany) : kSide);   // tokens of a CTA
    const dim3 grid(static_cast<unsigned>((a.T + n - 1) / n)), block(kRouteThreads);
    if (backward) return many ? launch_pdl(route_bwd_kernel<T, L, kManyBack>, grid, block, 0, s, a) : launch_pdl(route_bwd_kernel<T, L, kSide>, grid, block, 0, s, a);
    if (a.bias || a.top_groups < a.groups)
        return many ? launch_pdl(route_kernel<T, L, kMany, true>, grid, block, 0, s, a) : launch_pdl(route_kernel<T, L, kSide, true>, grid, block, 0, s, a);
    return many ? launch_pdl(route_kernel<T, L, kMany, false>, grid, block, 0, s, a) : launch_pdl(route_kernel<T, L, kSide, false>, grid, block, 0, s, a);
}

template <class T>
int run_route_lanes(const RouteArgs &a, bool backward, int sms, cudaStream_t s) {
    if (a.E <= 8) return run_route<T, 1>(a, backward, sms, s);
    if (a.E <= 16) return run_route<T, 2>(a, backward, sms, s);
    if (a.E <= 32) return run_route<T, 4>(a, backward, sms, s);
    if (a.E <= 64) return run_route<T, 8>(a, backward, sms, s);
    if (a.E <= 128) return run_route<T, 16>(a, backward, sms, s);
    return run_route<T, 32>(a, backward, sms, s);
}

}  // namespace

static RouteArgs route_args(const mlpblk_route_desc &d) {
    RouteArgs a = {};
    a.T = d.tokens;
    a.E = d.experts;
    a.k = d.top_k;
    a.by_k = static_cast<uint32_t>((65536 + a.k - 1) / a.k);
    a.by_k1 = static_cast<uint32_t>((65536 + a.k) / (a.k + 1));
    a.groups = d.groups;
    a.top_groups = d.top_groups;
    a.per = d.experts / d.groups;
    a.sigmoid = d.score == MLPBLK_ROUTE_SIGMOID;
    a.renorm = d.renorm;
    a.scale = d.scale;
    return a;
}

int launch_route(const mlpblk_route_desc &d, const void *logits, const float *bias, int *ids, float *weights, int sms, cudaStream_t s) {
    RouteArgs a = route_args(d);
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    return d.dtype == MLPBLK_BF16 ? run_route_lanes<__nv_bfloat16>(a, false, sms, s) : run_route_lanes<float>(a, false, sms, s);
}

int launch_route_bwd(const mlpblk_route_desc &d, const void *logits, const int *ids, const float *dw, void *dl, int sms, cudaStream_t s) {
    RouteArgs a = route_args(d);
    a.logits = logits;
    a.ids_in = ids;
    a.dw = dw;
    a.dl = dl;
    return d.dtype == MLPBLK_BF16 ? run_route_lanes<__nv_bfloat16>(a, true, sms, s) : run_route_lanes<float>(a, true, sms, s);
}

}  // namespace mlpblk
