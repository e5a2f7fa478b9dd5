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
// A token belongs to L = 1 .. 32 lanes of a warp, each of which holds eight neighbouring
// experts.  A lane sorts its eight keys once; a round then compares the lanes' best only
// and the winner moves up.  A key carries its index in its low half, so that one maximum
// decides ties too.
//
// Selection by exact order: without a bias and groups the logits themselves are the keys.
// Otherwise keys are float32 values with a known error; where two neighbours in the
// result (or the two groups on either side of the cut) are closer than that and are not
// the same logit with the same bias, the token's keys are computed again in float64.  So
// ids do not depend on how exp rounds.
#include <cuda_bf16.h>
#include <float.h>

#include "mlpblk_internal.h"

namespace mlpblk {

namespace {

constexpr int kRouteThreads = 128;
constexpr int kRouteV = 8;               // experts of a lane
constexpr float kRouteTiny = 1e-20f;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int64_t T;
    int E, k, groups, top_groups, per;   // per: experts of a group
    int sigmoid, renorm;
    float scale;
    int *ids;
    float *weights;
    // backward
    const int *ids_in;
    const float *dw;
    void *dl;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

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
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int L, class F>
__device__ __forceinline__ F lanes_sum(F v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// An order-preserving integer of a float or double key; 0 is below every key.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);  // -0 counts as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A key with its expert: larger keys first, then lower experts; 0 is none.
struct Key32 {
    uint64_t v;
    static __device__ __forceinline__ Key32 none() { return {0}; }
    static __device__ __forceinline__ Key32 of(float key, int e) { return {static_cast<uint64_t>(ordered(key)) << 32 | static_cast<uint32_t>(0xFFFF - e)}; }
    __device__ __forceinline__ bool before(const Key32 &o) const { return v > o.v; }
    __device__ __forceinline__ bool any() const { return v != 0; }
    __device__ __forceinline__ int expert() const { return 0xFFFF - static_cast<int>(v & 0xFFFFu); }
    __device__ __forceinline__ Key32 shfl_xor(int o) const { return {__shfl_xor_sync(0xffffffffu, v, o)}; }
};
struct Key64 {
    double key;
    int e;     // -1: none
    static __device__ __forceinline__ Key64 none() { return {0.0, -1}; }
    static __device__ __forceinline__ Key64 of(double key, int e) { return {key, e}; }
    __device__ __forceinline__ bool before(const Key64 &o) const {
        return e >= 0 && (o.e < 0 || key > o.key || (key == o.key && e < o.e));
    }
    __device__ __forceinline__ bool any() const { return e >= 0; }
    __device__ __forceinline__ int expert() const { return e; }
    __device__ __forceinline__ Key64 shfl_xor(int o) const {
        return {__shfl_xor_sync(0xffffffffu, key, o), __shfl_xor_sync(0xffffffffu, e, o)};
    }
};

template <class K>
__device__ __forceinline__ void order_pair(K &a, K &b) {
    const bool swap = b.before(a);
    const K x = swap ? b : a, y = swap ? a : b;
    a = x;
    b = y;
}

// Eight keys into descending order (Batcher's odd-even merge sort: 19 comparisons).
template <class K>
__device__ __forceinline__ void sort8(K (&v)[kRouteV]) {
    order_pair(v[0], v[1]); order_pair(v[2], v[3]); order_pair(v[4], v[5]); order_pair(v[6], v[7]);
    order_pair(v[0], v[2]); order_pair(v[1], v[3]); order_pair(v[4], v[6]); order_pair(v[5], v[7]);
    order_pair(v[1], v[2]); order_pair(v[5], v[6]);
    order_pair(v[0], v[4]); order_pair(v[1], v[5]); order_pair(v[2], v[6]); order_pair(v[3], v[7]);
    order_pair(v[2], v[4]); order_pair(v[3], v[5]);
    order_pair(v[1], v[2]); order_pair(v[3], v[4]); order_pair(v[5], v[6]);
}

// The best head of the token's lanes.
template <int L, class K>
__device__ __forceinline__ K lanes_best(K h) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        const K x = h.shfl_xor(o);
        if (x.before(h)) h = x;
    }
    return h;
}
template <>
__device__ __forceinline__ Key32 lanes_best<32, Key32>(Key32 h) {
    const uint32_t hi = static_cast<uint32_t>(h.v >> 32);
    const uint32_t top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t low = __reduce_max_sync(0xffffffffu, hi == top ? static_cast<uint32_t>(h.v) : 0u);
    return {static_cast<uint64_t>(top) << 32 | low};
}

// A token's scratch in shared memory: keys and marks of its experts and groups, and the
// experts in the order in which they were selected (and the next one).
struct RouteScratch {
    int won[MLPBLK_ROUTE_MAX_TOP_K + 1];
};

// Which of the token's groups are kept, as a bit mask held by every lane, and whether the
// cut is too close to call: the marks on either side of it differ by no more than `slack`.
// F: float or double; keys are the lane's eight, `row` a shared array of E of them.
template <int L, class F>
__device__ __forceinline__ uint64_t keep_groups(const RouteArgs &a, int sub, const F (&key)[kRouteV], F *row, F slack, bool *close) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRouteV; ++i)
        if (sub * kRouteV + i < a.E) row[sub * kRouteV + i] = key[i];
    __syncwarp();
    // a lane takes groups sub, sub + L, ...: their marks replace the first keys of each
    for (int g = sub; g < a.groups; g += L) {
        F first = -INFINITY, second = -INFINITY;
        for (int i = 0; i < a.per; ++i) {
            const F x = row[g * a.per + i];
            second = x > first ? first : (x > second ? x : second);
            first = x > first ? x : first;
        }
        row[g * a.per] = second > -INFINITY ? first + second : first;
    }
    __syncwarp();
    uint64_t kept = 0;
    F last = INFINITY, next = -INFINITY;   // the least mark that is kept, the best that is not
    for (int g = 0; g < a.groups; ++g) {
        const F m = row[g * a.per];
        int before = 0;
        for (int h = 0; h < a.groups; ++h) {
            const F o = row[h * a.per];
            before += o > m || (o == m && h < g);
        }
        if (before < a.top_groups) {
            kept |= 1ull << g;
            last = m < last ? m : last;
        } else {
            next = m > next ? m : next;
        }
    }
    *close = next > -INFINITY && last - next <= slack;
    __syncwarp();
    return kept;
}

// Selects into won[0 .. k] (expert or -1); with `open` a lane's eight experts by their keys.
template <int L, class K>
__device__ __forceinline__ void select(const RouteArgs &a, int sub, K (&v)[kRouteV], int rounds, int *won) {
    sort8(v);
    for (int r = 0; r < rounds; ++r) {
        const K best = lanes_best<L>(v[0]);
        const bool mine = best.any() && best.expert() == v[0].expert() && v[0].any();
        if (sub == 0) won[r] = best.any() ? best.expert() : -1;
        if (mine) {
#pragma unroll
            for (int i = 0; i + 1 < kRouteV; ++i) v[i] = v[i + 1];
            v[kRouteV - 1] = K::none();
        }
    }
    __syncwarp();
}

template <class T, int L>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const RouteArgs a) {
    constexpr int kTokens = kRouteThreads / L;
    // a token's row in shared memory: keys in float32 or float64 (grouped selection only)
    extern __shared__ double route_rows[];
    __shared__ RouteScratch scratch[kTokens];
    griddep_enter();
    const int sub = threadIdx.x % L, local = threadIdx.x / L;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + local;
    const bool live = t < a.T;
    if (!live) t = a.T - 1;      // the warp's lanes stay together
    const T *row = static_cast<const T *>(a.logits) + t * a.E;
    const int e0 = sub * kRouteV;
    float l[kRouteV];
    load_logits(row, e0, a.E, (a.E * sizeof(T)) % 16 == 0, l);
    int *won = scratch[local].won;
    double *keys64 = route_rows + static_cast<int64_t>(local) * a.E;
    const bool grouped = a.top_groups < a.groups;

    float m = 0.0f, inv_z = 1.0f;  // softmax: the largest logit, one over the sum
    if (!a.sigmoid) {
        m = l[0];
#pragma unroll
        for (int i = 1; i < kRouteV; ++i) m = fmaxf(m, l[i]);
        m = lanes_max<L>(m);
        if (!(m > -INFINITY)) m = 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) z += expf(l[i] - m);
        z = lanes_sum<L>(z);
        inv_z = z > 0.0f ? 1.0f / z : 0.0f;
    }
    auto score = [&](float x) {
        return a.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - m) * inv_z;
    };

    float key[kRouteV];
    const bool by_logit = a.bias == nullptr;   // the scores' order is the logits'
    if (!by_logit || grouped) {
#pragma unroll
        for (int i = 0; i < kRouteV; ++i)
            key[i] = l[i] > -INFINITY ? score(l[i]) + (by_logit ? 0.0f : __ldg(a.bias + e0 + i)) : -INFINITY;
    }
    // How far a float32 score may be from the exact one: exp's two ulps, its argument's
    // and the quotient's and sum's roundings, together below 12 ulps (7e-7) of a score
    // (softmax: |l - m| s is at most 1/e); then the sum with the bias, half an ulp.
    bool again = false;
    uint64_t kept = ~0ull;
    if (grouped) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) top = fmaxf(top, fabsf(key[i]) < INFINITY ? fabsf(key[i]) : 0.0f);
        top = lanes_max<L>(top);
        kept = keep_groups<L, float>(a, sub, key, reinterpret_cast<float *>(keys64), 4.0f * (1e-6f + 1.2e-7f * top), &again);
    }
    Key32 v[kRouteV];
#pragma unroll
    for (int i = 0; i < kRouteV; ++i) {
        const int e = e0 + i;
        const bool open = l[i] > -INFINITY && (!grouped || (kept >> (e / a.per) & 1));
        v[i] = open ? Key32::of(by_logit ? l[i] : key[i], e) : Key32::none();
    }
    select<L>(a, sub, v, a.k + 1, won);
    if (!by_logit) {
        const float most = a.sigmoid ? 1.0f : inv_z;   // no score is larger
        // neighbours that float32 cannot tell apart, and that are not the same numbers
        for (int r = sub; r < a.k; r += L) {
            const int e = won[r], f = won[r + 1];
            if (f < 0) continue;
            const float le = logit_of(to_float(row[e])), lf = logit_of(to_float(row[f]));
            const float be = a.bias[e], bf = a.bias[f];
            if (le == lf && be == bf) continue;
            const float ke = score(le) + be, kf = score(lf) + bf;
            if (fabsf(ke - kf) <= 2e-6f * most + 2.4e-7f * (fabsf(ke) + fabsf(kf))) again = true;
        }
    }
    // (a vote of the token's lanes; the warp walks the branch together)
    const unsigned votes = __ballot_sync(0xffffffffu, again);
    if (votes != 0) {
        const unsigned mine = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (threadIdx.x % 32 / L * L);
        const bool redo = (votes & mine) != 0;
        double key64[kRouteV];
        double z = 0.0;
        if (!a.sigmoid) {
#pragma unroll 1
            for (int i = 0; i < kRouteV; ++i) z += exp(static_cast<double>(l[i]) - static_cast<double>(m));
            z = lanes_sum<L>(z);
        }
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) key64[i] = -INFINITY;
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) {
            if (!(l[i] > -INFINITY)) continue;
            const double x = l[i];
            key64[i] = (a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / z) + (by_logit ? 0.0 : static_cast<double>(a.bias[e0 + i]));
        }
        uint64_t kept64 = ~0ull;
        if (grouped) {
            bool close;
            kept64 = keep_groups<L, double>(a, sub, key64, keys64, 0.0, &close);
        }
        Key64 w[kRouteV];
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) {
            const int e = e0 + i;
            const bool open = l[i] > -INFINITY && (!grouped || (kept64 >> (e / a.per) & 1));
            // by logit the order within the kept groups is the logits'
            w[i] = open ? Key64::of(by_logit ? static_cast<double>(l[i]) : key64[i], e) : Key64::none();
        }
        int *won64 = redo ? won : nullptr;
        // every token of the warp takes part; the ones that were clear keep their own
        __shared__ int spare[kTokens][MLPBLK_ROUTE_MAX_TOP_K + 1];
        select<L>(a, sub, w, a.k, won64 ? won64 : spare[local]);
    }
    // weights, from the logits of the selected
    float total = 0.0f;
    if (a.renorm) {
        for (int r = sub; r < a.k; r += L) total += won[r] >= 0 ? score(logit_of(to_float(row[won[r]]))) : 0.0f;
        total = lanes_sum<L>(total) + kRouteTiny;
    }
    for (int r = sub; r < a.k; r += L) {
        const int e = won[r];
        float s = e >= 0 ? score(logit_of(to_float(row[e]))) : 0.0f;
        if (a.renorm) s = s / total;
        if (live) {
            a.ids[t * a.k + r] = e;
            a.weights[t * a.k + r] = a.scale * s;
        }
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

// A token's gradient row: ds of the selected experts meets the row in shared memory.
template <class T, int L>
__global__ void __launch_bounds__(kRouteThreads)
route_bwd_kernel(const RouteArgs a) {
    constexpr int kTokens = kRouteThreads / L;
    __shared__ float rows[kTokens][L * kRouteV];
    griddep_enter();
    const int sub = threadIdx.x % L, local = threadIdx.x / L;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + local;
    const bool live = t < a.T;
    if (!live) t = a.T - 1;
    const bool vec = (a.E * sizeof(T)) % 16 == 0;
    const T *row = static_cast<const T *>(a.logits) + t * a.E;
    const int e0 = sub * kRouteV;
    const bool softmax = !a.sigmoid;
    float l[kRouteV];
    float m = 0.0f, inv_z = 1.0f;
    if (softmax) {
        load_logits(row, e0, a.E, vec, l);
        m = l[0];
#pragma unroll
        for (int i = 1; i < kRouteV; ++i) m = fmaxf(m, l[i]);
        m = lanes_max<L>(m);
        if (!(m > -INFINITY)) m = 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) {
            l[i] = expf(l[i] - m);
            z += l[i];
        }
        z = lanes_sum<L>(z);
        inv_z = z > 0.0f ? 1.0f / z : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kRouteV; ++i) rows[local][e0 + i] = 0.0f;
    __syncwarp();
    // s, S and sum dw s over the selected
    __shared__ float ds_of[kTokens][MLPBLK_ROUTE_MAX_TOP_K];
    float total = 0.0f, dot = 0.0f;
    for (int r = sub; r < a.k; r += L) {
        const int e = a.ids_in[t * a.k + r];
        if (e < 0 || e >= a.E) continue;
        const float x = logit_of(to_float(row[e]));
        const float s = softmax ? expf(x - m) * inv_z : 1.0f / (1.0f + expf(-x));
        total += s;
        dot += a.dw[t * a.k + r] * s;
    }
    total = lanes_sum<L>(total) + kRouteTiny;
    dot = lanes_sum<L>(dot);
    if (a.renorm) dot = dot / total;
    for (int r = sub; r < a.k; r += L) {
        const int e = a.ids_in[t * a.k + r];
        const float x = e >= 0 && e < a.E ? logit_of(to_float(row[e])) : -INFINITY;
        const float w = a.dw[t * a.k + r];
        float ds = a.renorm ? a.scale * ((w - dot) / total) : a.scale * w;
        if (a.sigmoid) {
            const float g = expf(-fabsf(x)), q = 1.0f / (1.0f + g);   // s (1 - s), without a difference
            ds *= g * q * q;
        } else if (a.renorm) {
            ds *= expf(x - m) * inv_z;
        }
        ds_of[local][r] = x > -INFINITY ? ds : 0.0f;
    }
    __syncwarp();
    // each lane adds what falls on its own experts, in slot order
    for (int r = 0; r < a.k; ++r) {
        const int e = a.ids_in[t * a.k + r];
        if (e >= e0 && e < e0 + kRouteV && e < a.E) rows[local][e] += ds_of[local][r];
    }
    __syncwarp();
    float out[kRouteV];
#pragma unroll
    for (int i = 0; i < kRouteV; ++i) out[i] = rows[local][e0 + i];
    if (softmax && a.renorm) {
        const float d = a.scale * dot * (kRouteTiny / total);
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) out[i] -= l[i] * inv_z * d;
    } else if (softmax) {
#pragma unroll
        for (int i = 0; i < kRouteV; ++i) out[i] = l[i] * inv_z * (out[i] - a.scale * dot);
    }
    if (live) store_logits(static_cast<T *>(a.dl) + t * a.E, e0, a.E, vec, out);
}

template <class T, int L>
int run_route(const RouteArgs &a, bool backward, cudaStream_t s) {
    constexpr int kTokens = kRouteThreads / L;
    const dim3 grid(static_cast<unsigned>((a.T + kTokens - 1) / kTokens));
    if (backward) return launch_pdl(route_bwd_kernel<T, L>, grid, dim3(kRouteThreads), 0, s, a);
    const size_t smem = a.top_groups < a.groups ? sizeof(double) * kTokens * a.E : 0;
    return launch_pdl(route_kernel<T, L>, grid, dim3(kRouteThreads), smem, s, a);
}

template <class T>
int run_route_lanes(const RouteArgs &a, bool backward, cudaStream_t s) {
    if (a.E <= 8) return run_route<T, 1>(a, backward, s);
    if (a.E <= 16) return run_route<T, 2>(a, backward, s);
    if (a.E <= 32) return run_route<T, 4>(a, backward, s);
    if (a.E <= 64) return run_route<T, 8>(a, backward, s);
    if (a.E <= 128) return run_route<T, 16>(a, backward, s);
    return run_route<T, 32>(a, backward, s);
}

}  // namespace

static RouteArgs route_args(const mlpblk_route_desc &d) {
    RouteArgs a = {};
    a.T = d.tokens;
    a.E = d.experts;
    a.k = d.top_k;
    a.groups = d.groups;
    a.top_groups = d.top_groups;
    a.per = d.experts / d.groups;
    a.sigmoid = d.score == MLPBLK_ROUTE_SIGMOID;
    a.renorm = d.renorm;
    a.scale = d.scale;
    return a;
}

int launch_route(const mlpblk_route_desc &d, const void *logits, const float *bias, int *ids, float *weights, cudaStream_t s) {
    RouteArgs a = route_args(d);
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    return d.dtype == MLPBLK_BF16 ? run_route_lanes<__nv_bfloat16>(a, false, s) : run_route_lanes<float>(a, false, s);
}

int launch_route_bwd(const mlpblk_route_desc &d, const void *logits, const int *ids, const float *dw, void *dl, cudaStream_t s) {
    RouteArgs a = route_args(d);
    a.logits = logits;
    a.ids_in = ids;
    a.dw = dw;
    a.dl = dl;
    return d.dtype == MLPBLK_BF16 ? run_route_lanes<__nv_bfloat16>(a, true, s) : run_route_lanes<float>(a, true, s);
}

}  // namespace mlpblk
