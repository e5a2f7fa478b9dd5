// norm.cu -- the pre-norm shell's residual sum and RMSNorm as operators of their own
// ("Nemotron Kernels From Inference To Backpropagation" -- "Setup: The Shared Transformer
// Shell", "Where Quantization Fits"; "Reverse-mode automatic differentiation" section 5,
// the LayerNorm rule without the mean terms):
//
//   s = x + residual                       rounded to the tensors' type: it is what is kept
//   r = 1 / sqrt(mean(s^2) + eps),  n = s r gamma
//   scale = max |n| / 448 over the row (or each 128 values), rounded to float32
//   codes = E4M3(n / scale), nearest even
//
//   g = dn gamma,  xh = s r:   dx = d_sum + r (g - xh mean(g xh)),   dgamma = sum_t dn xh
//
// One pass: a row stays in registers between its sums and its outputs, and the next row is
// already on its way.  max |s gamma| needs no r, so both reductions of a row are one.  Forward bound by HBM
// where there is a residual branch (16384 x 4096 bf16 74 us, 6.4 TB/s of 7 bytes an element) and by instruction
// issue without one (61 us), backward by HBM (84 us, 6.4 TB/s of 8 bytes).
//
// Order of the gradient's products: r alone may be 2^-60 or, with a small eps, 2^60 and more, and its square or cube
// leaves float32's range; s r and the products with it do not.
//
// Codes are those of the real number n / scale, rounded once: values half way between two codes
// are common (one in 1700 here: ratios of two short products), and which way they go is decided
// by the 25th bit of the scale.  So s gamma is exact (bf16), the sum of squares, r and r / scale are carried as sums
// of two floats (relative error below 2^-40), and where a float32 quotient's error may reach a
// border of two codes the product is taken to 48 bits and rounded to odd before it is rounded
// to E4M3.
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "mlpblk_internal.h"

namespace mlpblk {

namespace {

struct NormArgs {
    const void *x, *residual, *gamma;
    void *sum, *n;
    uint8_t *codes;
    float *scales, *rstd;
    int64_t T;
    int width, block;
    int warps;             // of a row
    float eps;
    // backward
    const void *dn, *d_sum;
    const float *rstd_in;
    void *dx;
    float *part;
    int pitch;             // floats of a partial row
    bool ask;              // rows are asked into L2 ahead of their loads
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// How a lane holds its part of a warp's unit of a row: E values, which in the vector forms
// lie next to each other and in the scalar form (rows of any length) 32 apart.  Raw: as they
// are loaded.
template <class T_, bool VEC_>
struct Lay {
    using T = T_;
    static constexpr bool VEC = VEC_;
    static constexpr bool kPacked = VEC && sizeof(T) == 2;
    static constexpr int E = kPacked ? 8 : 4;
    static constexpr int kUnit = 32 * E;                 // values of a unit
    static constexpr int kBlockLanes = 128 / E;          // lanes that share a block of 128
    struct Raw {
        uint32_t w[4];                                   // bf16 pairs, or a float (scalar bf16: its bits on top) each
    };
    // The column of a lane's value i in a unit whose first value is at `at` (first_col).
    static __device__ __forceinline__ int first_col(int unit, int lane) { return unit * kUnit + (VEC ? lane * E : lane); }
    static __device__ __forceinline__ int col(int at, int i) { return at + (VEC ? i : 32 * i); }
    // The lane's part of a unit; 0 behind the row's end.  inside: it is known to have none there (the
    // zeros' selects would be a move for each register and row).
    static __device__ __forceinline__ Raw load(const T *row, int at, int width, bool inside = false) {
        Raw r;
        if constexpr (VEC) {
            const uint4 a = inside || at < width ? *reinterpret_cast<const uint4 *>(row + at) : make_uint4(0, 0, 0, 0);
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(at, i);
                if constexpr (sizeof(T) == 2) r.w[i] = c < width ? static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[c]) << 16 : 0u;
                else r.w[i] = c < width ? __float_as_uint(row[c]) : 0u;
            }
        }
        return r;
    }
    static __device__ __forceinline__ void store(T *row, int at, int width, const Raw &r) {
        if constexpr (VEC) {
            if (at < width) *reinterpret_cast<uint4 *>(row + at) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(at, i);
                if (c >= width) continue;
                if constexpr (sizeof(T) == 2) reinterpret_cast<uint16_t *>(row)[c] = static_cast<uint16_t>(r.w[i] >> 16);
                else row[c] = __uint_as_float(r.w[i]);
            }
        }
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&v)[E]) {
        if constexpr (kPacked) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(r.w[i] << 16);
                v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
        }
    }
    // Rounded to the type.
    static __device__ __forceinline__ Raw pack(const float (&v)[E]) {
        Raw r;
        if constexpr (kPacked) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = pack2(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = sizeof(T) == 2 ? pack2(0.0f, v[i]) & 0xFFFF0000u : __float_as_uint(v[i]);
        }
        return r;
    }
    // a + b, rounded to the type.
    static __device__ __forceinline__ Raw add(const Raw &a, const Raw &b) {
        Raw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kPacked) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r.w[i]) : "r"(a.w[i]), "r"(b.w[i]));
            else if constexpr (sizeof(T) == 2) r.w[i] = pack2(0.0f, __uint_as_float(a.w[i]) + __uint_as_float(b.w[i])) & 0xFFFF0000u;
            else r.w[i] = __float_as_uint(__uint_as_float(a.w[i]) + __uint_as_float(b.w[i]));
        }
        return r;
    }
    // The largest magnitude of n units.
    template <int N>
    static __device__ __forceinline__ float largest(const Raw (&r)[N]) {
        if constexpr (kPacked) {
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(r[u].w[i]));
            return fmaxf(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xFFFF0000u)));
        } else {
            float m = 0.0f;
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(__uint_as_float(r[u].w[i])));
            return m;
        }
    }
    static __device__ __forceinline__ void store_codes(uint8_t *row, int at, int width, const uint32_t (&w)[E / 4]) {
        if constexpr (VEC) {
            if (at >= width) return;
            if constexpr (E == 8) *reinterpret_cast<uint2 *>(row + at) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(row + at) = w[0];
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(at, i);
                if (c < width) row[c] = static_cast<uint8_t>(w[0] >> (8 * i));
            }
        }
    }
};

// hi + lo += v, without losing v's low bits (Knuth's two-sum).
__device__ __forceinline__ void two_add(float &hi, float &lo, float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b));
    hi = s;
}

// The larger one; NaN if one of them is (fmaxf drops it).  Units with such a gamma marked ahead of the loop over the
// rows, instead: 8192 x 8192 by blocks 93 us, with this 87.
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A product as it orders: the float32 product and, in float32 tensors, its rounding error
// (bf16 products are exact).  A NaN stays: it is gamma's, and then the scale's.
struct Peak {
    float hi, lo;
    __device__ __forceinline__ void take(float h, float l) {
        lo = h > hi || (h == hi && l > lo) ? l : lo;
        hi = larger(hi, h);
    }
};

// The sum of hi + lo over the warp's lanes (hi >= 0, lo small beside it), as two floats: in
// fixed point below the largest lane's exponent, 25 bits and 24 more, which integers add
// exactly (three reductions of the warp instead of five steps of two-sums).
__device__ __forceinline__ void warp_sum(float &hi, float &lo) {
    const float h = __fadd_rn(hi, lo), l = __fsub_rn(lo, __fsub_rn(h, hi));   // l within half an ulp of h
    float most;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(most) : "f"(h));
    // 2^(24 - exponent) brings every lane below 2^25
    const uint32_t field = 278u - static_cast<uint32_t>(min(max(static_cast<int>(__float_as_uint(most) >> 23), 30), 254));
    const float up = __uint_as_float(field << 23), down = __uint_as_float((254u - field) << 23);
    const float x = h * up, whole = truncf(x);
    const int high = static_cast<int>(whole), low = __float2int_rn(((x - whole) + l * up) * 0x1p24f);   // below 2^25
    const int sum_high = __reduce_add_sync(0xffffffffu, high), sum_low = __reduce_add_sync(0xffffffffu, low);
    const float top = static_cast<float>(sum_high);    // of 30 bits: what it rounds off goes below
    const float rest = static_cast<float>(sum_high - static_cast<int>(top)) + static_cast<float>(sum_low) * 0x1p-24f;
    hi = most < INFINITY ? top * down : NAN;
    lo = rest * down;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ Peak warp_peak(Peak p, bool exact) {
    const float h = warp_max(p.hi);
    return {h, exact ? 0.0f : warp_max(p.hi == h ? p.lo : -INFINITY)};
}

// 1 / sqrt(mean + eps) from the row's sum of squares, as a sum of two floats: the
// approximate root once refined (the residual 1 - m y^2 taken exactly).
__device__ __forceinline__ void refined_root(float hi, float lo, float width, float inv_width, float eps, float &mh, float &rh, float &rl) {
    mh = __fmul_rn(hi, inv_width);
    float ml = (__fmaf_rn(-mh, width, hi) + lo) * inv_width;
    two_add(mh, ml, eps);
    const float y = rsqrtf(mh);
    const float y2 = __fmul_rn(y, y), y2l = __fmaf_rn(y, y, -y2);
    const float e = __fmaf_rn(-mh, y2, 1.0f) - mh * y2l - ml * y2;
    const float c = y * (0.5f * e + 0.375f * e * e);
    rh = __fadd_rn(y, c);
    rl = c - __fsub_rn(rh, y);
}
// The same of a mean below 2^-80, times 2^60: 1 / mean leaves float32's range, and lo is not small beside hi.
__device__ __noinline__ float2 tiny_root(float hi, float lo, float width, float inv_width, float eps) {
    float mh, rh, rl;
    const float h = __fadd_rn(hi, lo);
    refined_root(h * 0x1p60f, __fsub_rn(lo, __fsub_rn(h, hi)) * 0x1p60f, width, inv_width, eps * 0x1p60f, mh, rh, rl);
    return mh == 0.0f ? make_float2(INFINITY, 0.0f) : make_float2(rh * 0x1p30f, rl * 0x1p30f);   // (eps = 0 and a row of zeros)
}
__device__ __forceinline__ void inverse_root(float hi, float lo, float width, float inv_width, float eps, float &rh, float &rl) {
    float mh;
    refined_root(hi, lo, width, inv_width, eps, mh, rh, rl);
    if (mh < 0x1p-80f) {
        const float2 r = tiny_root(hi, lo, width, inv_width, eps);
        rh = r.x, rl = r.y;
    }
    if (!(hi < INFINITY)) rh = NAN, rl = 0.0f;         // an infinity or a NaN in the row
}

// The scale of a block whose largest |s gamma| is p, and r / scale as two floats.  up: where p is so
// small that r / scale would overflow, the quotient is 2^-64 of it and up is 2^64; else 1.
__device__ __forceinline__ float scale_of(const Peak &p, float rh, float rl, float &ch, float &cl, float &up) {
    const float t = __fmul_rn(rh, p.hi);
    const float tl = __fmaf_rn(rh, p.hi, -t) + rl * p.hi + rh * p.lo;
    constexpr float k = 1.0f / 448.0f;
    const float q = __fmul_rn(t, k);
    float scale = __fadd_rn(q, (__fmaf_rn(-q, 448.0f, t) + tl) * k);
    up = 1.0f;
    if (p.hi > 0x1p-60f && scale > 0x1p-100f && scale < 0x1p100f) {
        float y;
        asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(scale));
        ch = __fmul_rn(rh, y);
        cl = (__fmaf_rn(-ch, scale, rh) + rl) * y;
        return scale;
    }
    if (!(p.hi < INFINITY)) scale = NAN;
    if (scale == 0.0f) scale = 1.0f;                   // a block of zeros
    const bool small = p.hi < 0x1p-60f;
    up = small ? 0x1p64f : 1.0f;
    const float down = small ? 0x1p-64f : 1.0f, a = rh * down;
    ch = __fdiv_rn(a, scale);
    cl = __fdiv_rn(__fmaf_rn(-ch, scale, a) + rl * down, scale);
    if (!(p.hi > 0.0f)) ch = cl = 0.0f, up = 1.0f;     // zeros, or behind the row's end: codes of 0 (r may be infinite there)
    if (scale != scale) ch = cl = NAN;
    return scale;
}

// |p| (ch + cl) rounded to odd, with p's sign: the nearest float and what is left, then the
// neighbour towards the rest whose last bit is set, so that a rounding to fewer bits sees on
// which side of a border the value lies.
__device__ __forceinline__ float scaled_odd(float p, float pl, float ch, float cl) {
    const float a = fabsf(p);
    const float v = __fmul_rn(a, ch);
    float e = __fmaf_rn(a, ch, -v);
    e = __fmaf_rn(a, cl, e);
    e = __fmaf_rn(p < 0.0f ? -pl : pl, ch, e);
    const float w = __fadd_rn(v, e);
    e = __fsub_rn(e, __fsub_rn(w, v));
    uint32_t u = __float_as_uint(w) - (e < 0.0f ? 1u : 0u);
    u |= e != 0.0f ? 1u : 0u;
    return __uint_as_float(u | (__float_as_uint(p) & 0x80000000u));
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | e4m3x2(c, d) << 16; }

constexpr int kNormMaxWarps = 16;      // of a row

// The lowest log2(N) bits of i in the opposite order.
template <int N>
__device__ __forceinline__ int reversed(int i) {
    int r = 0;
#pragma unroll
    for (int b = 1; b < N; b <<= 1) r = r << 1 | (i & b ? 1 : 0);
    return r;
}

// Threads of row slot `slot` meet (its warps alone).
__device__ __forceinline__ void row_barrier(int slot, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(32 * warps) : "memory");
}

// n of a row in which s gamma leaves float32's range, from s once more: s r gamma need not leave it.
// (A call: inside the loop over the rows its registers cost the codes 3%.)
template <class L>
__device__ __noinline__ void norm_again(const NormArgs &a, const typename L::T *row, int64_t at, int w, float rh) {
    using T = typename L::T;
    constexpr int E = L::E;
    for (int c = L::first_col(w, threadIdx.x & 31); c < a.width; c += a.warps * L::kUnit) {
        float n[E], g[E];
        L::unpack(L::load(row + at, c, a.width), n);
        L::unpack(L::load(static_cast<const T *>(a.gamma), c, a.width), g);
#pragma unroll
        for (int i = 0; i < E; ++i) n[i] = (n[i] * rh) * g[i];
        L::store(static_cast<T *>(a.n) + at, c, a.width, L::pack(n));
    }
}

// RES: a residual branch is added.
template <class L, int N, bool RES>
__global__ void __launch_bounds__(32 * kNormMaxWarps)
add_rmsnorm_kernel(const NormArgs a) {
    using T = typename L::T;
    using Raw = typename L::Raw;
    constexpr int E = L::E;
    constexpr bool kExact = sizeof(T) == 2;   // products of two values are exact in float32
    constexpr bool kAhead = N <= 4;           // the next row is loaded while this one is worked on
    __shared__ float4 meet[2][kNormMaxWarps];
    griddep_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int W = a.warps, slot = warp / W, w = warp % W;
    const int slots = static_cast<int>(blockDim.x >> 5) / W;
    const float width = static_cast<float>(a.width), inv_width = 1.0f / width;
    Raw g[N], x[N], res[RES ? N : 1];
    int c[N];                                 // the lane's first column of each unit
#pragma unroll
    for (int u = 0; u < N; ++u) c[u] = L::first_col(w + u * W, lane);
#pragma unroll
    for (int u = 0; u < N; ++u) g[u] = L::load(static_cast<const T *>(a.gamma), c[u], a.width);
    auto fetch_row = [&](int64_t t, auto inside) {
        const int64_t at = t * a.width;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            x[u] = L::load(static_cast<const T *>(a.x) + at, c[u], a.width, decltype(inside)::value);
            if (RES) res[u] = L::load(static_cast<const T *>(a.residual) + at, c[u], a.width, decltype(inside)::value);
        }
    };
    // (two copies of the loads, not of the loop)
    const bool whole = L::VEC && W * N * L::kUnit == a.width;
    auto fetch = [&](int64_t t) {
        if (whole) fetch_row(t, std::true_type{});
        else fetch_row(t, std::false_type{});
    };
    int phase = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * slots;
    int64_t t = static_cast<int64_t>(blockIdx.x) * slots + slot;
    if (kAhead && t < a.T) fetch(t);
    for (; t < a.T; t += step) {
        const int64_t at = t * a.width;
        if (!kAhead) fetch(t);
        if (RES) {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                x[u] = L::add(x[u], res[u]);
                L::store(static_cast<T *>(a.sum) + at, c[u], a.width, x[u]);
            }
        }
        // The squares of a lane are added on top of a power of two that no sum of them reaches: each
        // addition then drops the same bits, and what it dropped is found exactly.
        constexpr uint32_t kRoom = (N * E <= 4 ? 3u : N * E <= 8 ? 4u : N * E <= 16 ? 5u : N * E <= 32 ? 6u : 7u) << 23;
        const float most = L::largest(x);
        const float base = __uint_as_float(min((__float_as_uint(most * most) & 0x7F800000u) + kRoom, 0x7F800000u));
        float hi = base, lo = 0.0f;
        float v[N][E];                          // s gamma (bf16), or s
        Peak peak[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float gv[E];
            L::unpack(x[u], v[u]);
            L::unpack(g[u], gv);
            peak[u] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float s = v[u][i];
                const float sum = __fmaf_rn(s, s, hi);
                lo += __fmaf_rn(s, s, -__fsub_rn(sum, hi));
                hi = sum;
                const float p = __fmul_rn(s, gv[i]);
                if (kExact) {
                    peak[u].hi = larger(peak[u].hi, fabsf(p));
                    v[u][i] = p;
                } else {
                    const float pl = __fmaf_rn(s, gv[i], -p);
                    peak[u].take(fabsf(p), p < 0.0f ? -pl : pl);
                }
            }
        }
        hi = __fsub_rn(hi, base);
        if (kAhead && t + step < a.T) fetch(t + step);
        Peak top = peak[0];
#pragma unroll
        for (int u = 1; u < N; ++u) {
            if (kExact) top.hi = larger(top.hi, peak[u].hi);
            else top.take(peak[u].hi, peak[u].lo);
        }
        warp_sum(hi, lo);
        top = warp_peak(top, kExact);
        if (W > 1) {
            // the buffer alternates, so one barrier a row is enough
            float4 *m = meet[phase] + slot * W;
            phase ^= 1;
            if (lane == 0) m[w] = make_float4(hi, lo, top.hi, top.lo);
            row_barrier(slot, W);
            const float4 q = lane < W ? m[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            hi = q.x, lo = q.y;
            warp_sum(hi, lo);
            top = warp_peak({q.z, q.w}, kExact);
        }
        float rh, rl;
        inverse_root(hi, lo, width, inv_width, a.eps, rh, rl);
        if (a.rstd && w == 0 && lane == 0) a.rstd[t] = rh;
        if (a.n) {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                float n[E], gv[E];
                L::unpack(g[u], gv);
#pragma unroll
                for (int i = 0; i < E; ++i) n[i] = (kExact ? v[u][i] : v[u][i] * gv[i]) * rh;
                L::store(static_cast<T *>(a.n) + at, c[u], a.width, L::pack(n));
            }
            if (!(top.hi < INFINITY)) norm_again<L>(a, static_cast<const T *>(RES ? a.sum : a.x), at, w, rh);
        }
        if (a.codes) {
            float ch, cl, up;                 // by blocks: of the block whose scale the lane has found
            constexpr int kGroup = L::kBlockLanes;
            if (!a.block) {
                const float scale = scale_of(top, rh, rl, ch, cl, up);
                if (w == 0 && lane == 0) a.scales[t] = scale;
            } else {
                // Each exchange halves the units that a lane goes on with, so that the lanes of a block end with
                // one unit's maximum each, and find its scale (8192 x 8192: 94 us with every lane finding all).
                Peak mine[N];
#pragma unroll
                for (int u = 0; u < N; ++u) mine[u] = peak[u];
#pragma unroll
                for (int o = 1, half = N / 2; o < kGroup; o <<= 1, half /= 2) {
                    const bool upper = lane & o;
#pragma unroll
                    for (int u = 0; u < (half > 0 ? half : 1); ++u) {
                        const Peak give = half > 0 && !upper ? mine[u + half] : mine[u];
                        if (half > 0 && upper) mine[u] = mine[u + half];
                        const float h = __shfl_xor_sync(0xffffffffu, give.hi, o);
                        if (kExact) mine[u].hi = larger(mine[u].hi, h);
                        else mine[u].take(h, __shfl_xor_sync(0xffffffffu, give.lo, o));
                    }
                }
                const float scale = scale_of(mine[0], rh, rl, ch, cl, up);
                const int b = (w + reversed<N>(lane) * W) * (L::kUnit / 128) + lane / kGroup;
                if (lane % kGroup < N && b * 128 < a.width) a.scales[t * ((a.width + 127) / 128) + b] = scale;
            }
            const bool far = __any_sync(0xffffffffu, up != 1.0f);
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int unit = w + u * W;
                if (unit * L::kUnit >= a.width) continue;
                float cu = ch, cul = cl, uu = up;
                if (a.block) {
                    const int from = (lane & -kGroup) | reversed<N>(u);
                    cu = __shfl_sync(0xffffffffu, ch, from);
                    cul = __shfl_sync(0xffffffffu, cl, from);
                    if (far) uu = __shfl_sync(0xffffffffu, up, from);
                }
                float gv[E];
                if (!kExact) L::unpack(g[u], gv);
                // the codes at both ends of what a float32 quotient may be off: where they are the same, so is
                // the exact one's (four values share a look)
                constexpr float kOff = kExact ? 0x1p-22f : 0x1p-21f;
                const float c_low = __fmul_rn(cu, 1.0f - kOff), c_high = __fmul_rn(cu, 1.0f + kOff);
                uint32_t codes[E / 4];
#pragma unroll
                for (int j = 0; j < E / 4; ++j) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = kExact ? v[u][4 * j + i] : __fmul_rn(v[u][4 * j + i], gv[4 * j + i]);
                    const uint32_t low = e4m3x4(p[0] * c_low, p[1] * c_low, p[2] * c_low, p[3] * c_low);
                    codes[j] = e4m3x4(p[0] * c_high, p[1] * c_high, p[2] * c_high, p[3] * c_high);
                    if (codes[j] != low || far) {
                        float q[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            q[i] = scaled_odd(p[i] * uu, kExact ? 0.0f : __fmaf_rn(v[u][4 * j + i], gv[4 * j + i], -p[i]) * uu, cu, cul);
                        codes[j] = e4m3x4(q[0], q[1], q[2], q[3]);
                    }
                }
                L::store_codes(a.codes + at, c[u], a.width, codes);
            }
        }
    }
}

// A CTA keeps its rows' share of dgamma in registers and leaves one partial row.
template <class L, int N>
__global__ void __launch_bounds__(32 * kNormMaxWarps)
add_rmsnorm_bwd_kernel(const NormArgs a) {
    using T = typename L::T;
    using Raw = typename L::Raw;
    constexpr int E = L::E;
    constexpr bool kAhead = N <= 2;           // as in the forward
    constexpr bool kKeep = N <= 4;            // a row stays in registers; else it is read again
    __shared__ float meet[2][kNormMaxWarps];
    extern __shared__ float shares[];         // [slots - 1][W * N * kUnit]: the other slots' dgamma
    griddep_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int W = a.warps, slot = warp / W, w = warp % W;
    const int slots = static_cast<int>(blockDim.x >> 5) / W;
    const float inv_width = 1.0f / static_cast<float>(a.width);
    Raw g[N], sr[N], dr[N], yr[N];
    int c[N];                                 // the lane's first column of each unit
#pragma unroll
    for (int u = 0; u < N; ++u) c[u] = L::first_col(w + u * W, lane);
    float acc[N][E], r_next = 0.0f;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        g[u] = L::load(static_cast<const T *>(a.gamma), c[u], a.width);
        yr[u] = Raw{};
#pragma unroll
        for (int i = 0; i < E; ++i) acc[u][i] = 0.0f;
    }
    auto fetch_unit = [&](int64_t t, int u) {
        const int64_t at = t * a.width;
        sr[u] = L::load(static_cast<const T *>(a.x) + at, c[u], a.width);
        dr[u] = L::load(static_cast<const T *>(a.dn) + at, c[u], a.width);
        if (a.d_sum) yr[u] = L::load(static_cast<const T *>(a.d_sum) + at, c[u], a.width);
    };
    auto fetch = [&](int64_t t) {
        r_next = a.rstd_in[t];
        if constexpr (kKeep) {
#pragma unroll
            for (int u = 0; u < N; ++u) fetch_unit(t, u);
        }
    };
    int phase = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * slots;
    int64_t t = static_cast<int64_t>(blockIdx.x) * slots + slot;
    if (kAhead && t < a.T) fetch(t);
    for (; t < a.T; t += step) {
        const int64_t at = t * a.width;
        if (!kAhead) fetch(t);
        const float r = r_next;
        Raw s0[N], d0[N], y0[N];
        float dot = 0.0f;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (!kKeep) fetch_unit(t, u);
            s0[u] = sr[u], d0[u] = dr[u], y0[u] = yr[u];
            float s[E], d[E], gv[E];
            L::unpack(s0[u], s);
            L::unpack(d0[u], d);
            L::unpack(g[u], gv);
#pragma unroll
            for (int i = 0; i < E; ++i) dot += d[i] * gv[i] * (s[i] * r);   // (g xh: rstd's powers alone leave float32's range)
        }
        if (kAhead && t + step < a.T) fetch(t + step);
        // The row after next is asked into L2, by a lane each of its first three warps or, of fewer, by the first warp's
        // first three lanes: what a warp has in flight
        // in its registers is one row (16384 x 4096 bf16 92 -> 86 us, 8192 x 768, which L2 holds, 15.2 -> 16.2;
        // with the warp's pointer kept over the loop the registers spill and nothing is won).
        const int array = W > 2 ? w + 3 * lane : lane + 3 * w;
        if (L::VEC && a.ask && array < 3 && t + 2 * step < a.T) {
            const void *src = array == 0 ? a.x : array == 1 ? a.dn : a.d_sum;
            if (src)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const T *>(src) + (t + 2 * step) * a.width),
                             "r"(a.width * static_cast<int>(sizeof(T)))
                             : "memory");
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (W > 1) {
            float *m = meet[phase] + slot * W;
            phase ^= 1;
            if (lane == 0) m[w] = dot;
            row_barrier(slot, W);
            dot = m[lane % W];
            for (int o = 1; o < W; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float mean = dot * inv_width;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float s[E], d[E], y[E], gv[E], v[E];
            if (!kKeep) {
                fetch_unit(t, u);
                s0[u] = sr[u], d0[u] = dr[u], y0[u] = yr[u];
            }
            L::unpack(s0[u], s);
            L::unpack(d0[u], d);
            L::unpack(y0[u], y);
            L::unpack(g[u], gv);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float xh = s[i] * r;
                v[i] = r * (d[i] * gv[i] - xh * mean) + y[i];
                acc[u][i] += d[i] * xh;
            }
            L::store(static_cast<T *>(a.dx) + at, c[u], a.width, L::pack(v));
        }
    }
    // the CTA's partial row: slot 0's warps add the other slots' shares in order
    const int stride = W * N * L::kUnit;
    if (slot > 0) {
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) shares[(slot - 1) * stride + L::col(c[u], i)] = acc[u][i];
    }
    if (slots > 1) __syncthreads();
    if (slot > 0) return;
    float *out = a.part + static_cast<int64_t>(blockIdx.x) * a.pitch;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int j = L::col(c[u], i);
            float v = acc[u][i];
            for (int k = 1; k < slots; ++k) v += shares[(k - 1) * stride + j];
            if (j < a.width) out[j] = v;
        }
}

// dgamma += (or =) the partial rows: 32 columns a CTA, 32 slices of rows in order, then a
// fixed pairwise tree.
__global__ void __launch_bounds__(1024)
norm_dgamma_kernel(const float *__restrict__ part, int parts, int pitch, int width, float *__restrict__ dgamma, int overwrite) {
    __shared__ float red[32][33];
    griddep_enter();
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = static_cast<int>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 4
        for (int p = slice; p < parts; p += 32) s += part[static_cast<int64_t>(p) * pitch + c];
    }
    red[slice][lane] = s;
    __syncthreads();
    for (int h = 16; h >= 1; h >>= 1) {
        if (slice < h) red[slice][lane] += red[slice + h][lane];
        __syncthreads();
    }
    if (slice == 0 && c < width) dgamma[c] = overwrite ? red[0][lane] : dgamma[c] + red[0][lane];
}

// Warps of a row and units of a warp.  Many rows: four units a warp forward, two backward (three arrays, and dgamma's
// sums), so that with the next row on its way a warp has 64 KB an SM in flight and a row meets in few
// warps.  Few rows (no more than the SMs): as many warps as there are units, backward also for few values
// (2000 x 777 9.3 us with one unit a warp, 10.6 with two; 4097 x 1001 float32, whose rows take twice the
// instructions a value, 11.8 and 13.2; 4096 x 2048 20.7 and 19.7).
struct NormShape {
    int warps, units;
};
NormShape norm_shape(int width, int unit, bool vec, int64_t T, int sms, bool backward) {
    const int U = (width + unit - 1) / unit;
    const bool few = T <= sms || (backward && T * width <= (vec ? 2 : 8) << 20);
    const int each = few ? 1 : backward ? 2 : 4;
    NormShape s = {1, 0};
    while (s.warps < kNormMaxWarps && s.warps * each < U) s.warps *= 2;
    s.units = 1;
    while (s.units * s.warps < U) s.units *= 2;
    return s;
}

template <class L, int N>
int run_norm(NormArgs a, bool backward, int sms, cudaStream_t s, int *parts) {
    // Many rows: CTAs as large as they go (fewer partial rows of dgamma, and the rows of a CTA lie together:
    // 16384 x 4096 forward 66 us with 512 threads, 72 with 128, backward 77 and 80).  Few: 128 (300 x 1000
    // forward 2.9 us, with 512 3.4; backward 512 there too: 300 x 4096 8.0 us, 8.1 with 128).
    const int least = backward || a.T >= static_cast<int64_t>(sms) * 16 ? 32 * kNormMaxWarps : 128;
    const int threads = 32 * a.warps > least ? 32 * a.warps : least;
    const int slots = threads / (32 * a.warps);
    const size_t smem = backward ? static_cast<size_t>(slots - 1) * a.warps * N * L::kUnit * 4 : 0;
    void (*const kernel)(NormArgs) = backward ? add_rmsnorm_bwd_kernel<L, N> : (a.residual ? add_rmsnorm_kernel<L, N, true> : add_rmsnorm_kernel<L, N, false>);
    static int occ[3][2][5][64] = {};   // resident CTAs an SM, by kernel, size, log2(warps) and device
    int dev = 0, lg = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    while ((1 << lg) < a.warps) ++lg;
    int &o = occ[backward ? 2 : (a.residual ? 1 : 0)][threads == 32 * kNormMaxWarps][lg][dev];
    if (o == 0) {
        int n = 0;
        const int rc = cuda_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem));
        if (rc != MLPBLK_OK) return rc;
        o = n < 1 ? 1 : n;
    }
    int64_t grid = (a.T + slots - 1) / slots;
    const int64_t most = static_cast<int64_t>(sms) * o;
    if (grid > most) grid = most;
    if (backward) {
        if (grid > kNormMaxParts) grid = kNormMaxParts;
        *parts = static_cast<int>(grid);
    }
    return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, s, a);
}

template <class L>
int run_norm_lay(NormArgs a, bool backward, int sms, cudaStream_t s, int *parts) {
    const NormShape sh = norm_shape(a.width, L::kUnit, L::VEC, a.T, sms, backward);
    a.warps = sh.warps;
    switch (sh.units) {
        case 1: return run_norm<L, 1>(a, backward, sms, s, parts);
        case 2: return run_norm<L, 2>(a, backward, sms, s, parts);
        case 4: return run_norm<L, 4>(a, backward, sms, s, parts);
        default: break;
    }
    if constexpr (L::E == 4) return run_norm<L, 8>(a, backward, sms, s, parts);   // (16 warps of 4 units of 256 are kNormMaxWidth)
    return MLPBLK_EINVAL;
}

int run_norm_type(const NormArgs &a, int dtype, bool backward, int sms, cudaStream_t s, int *parts) {
    if (dtype == MLPBLK_BF16)
        return a.width % 8 == 0 ? run_norm_lay<Lay<__nv_bfloat16, true>>(a, backward, sms, s, parts)
                                : run_norm_lay<Lay<__nv_bfloat16, false>>(a, backward, sms, s, parts);
    return a.width % 4 == 0 ? run_norm_lay<Lay<float, true>>(a, backward, sms, s, parts)
                            : run_norm_lay<Lay<float, false>>(a, backward, sms, s, parts);
}

}  // namespace

int launch_add_rmsnorm(const mlpblk_norm_desc &d, const void *x, const void *residual, const void *gamma, void *sum, void *n,
                       uint8_t *codes, float *scales, float *rstd, int sms, cudaStream_t s) {
    NormArgs a = {};
    a.x = x;
    a.residual = residual;
    a.gamma = gamma;
    a.sum = sum;
    a.n = n;
    a.codes = codes;
    a.scales = scales;
    a.rstd = rstd;
    a.T = d.tokens;
    a.width = static_cast<int>(d.width);
    a.block = d.block;
    a.eps = d.eps;
    return run_norm_type(a, d.dtype, false, sms, s, nullptr);
}

int launch_add_rmsnorm_bwd(const mlpblk_norm_desc &d, const void *dn, const void *d_sum, const void *sum, const float *rstd,
                           const void *gamma, void *dx, float *part, int *parts, int sms, cudaStream_t s) {
    NormArgs a = {};
    a.x = sum;
    a.gamma = gamma;
    a.dn = dn;
    a.d_sum = d_sum;
    a.rstd_in = rstd;
    a.dx = dx;
    a.part = part;
    a.pitch = static_cast<int>(norm_part_pitch(d.width));
    a.T = d.tokens;
    a.width = static_cast<int>(d.width);
    a.ask = d.tokens * d.width * (d.dtype == MLPBLK_BF16 ? 2 : 4) >= 24 << 20;   // two or three such arrays: more than half of L2
    return run_norm_type(a, d.dtype, true, sms, s, parts);
}

int launch_norm_dgamma(const float *part, int parts, int64_t width, float *dgamma, int overwrite, cudaStream_t s) {
    return launch_pdl(norm_dgamma_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(1024), 0, s, part, parts,
                      static_cast<int>(norm_part_pitch(width)), static_cast<int>(width), dgamma, overwrite);
}

}  // namespace mlpblk
