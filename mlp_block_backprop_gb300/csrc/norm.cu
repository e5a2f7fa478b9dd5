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
// One pass: a row stays in registers between its sums and its outputs.  max |s gamma| needs
// no r, so both reductions of a row are one.  Bound by HBM (7 bytes an element forward
// with a residual branch in bf16, 8 backward).
//
// Codes are those of the real number n / scale: s gamma is exact (bf16), r and r / scale are
// carried as sums of two floats (relative error about 2^-45), the product is rounded to odd
// and only then to E4M3, so that no value is rounded twice.  Values half way between two
// codes are common (a ratio of two short products), and a float32 quotient would send them
// either way.
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
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// How a lane holds its part of a warp's unit of a row: E values, which in the vector forms
// lie next to each other and in the scalar form (rows of any length) 32 apart.
template <class T_, bool VEC_>
struct Lay {
    using T = T_;
    static constexpr bool VEC = VEC_;
    static constexpr int E = VEC && sizeof(T) == 2 ? 8 : 4;
    static constexpr int kUnit = 32 * E;                 // values of a unit
    static constexpr int kBlockLanes = 128 / E;          // lanes that share a block of 128
    static __device__ __forceinline__ int col(int unit, int lane, int i) {
        return VEC ? unit * kUnit + lane * E + i : unit * kUnit + lane + 32 * i;
    }
    // E values from column col(unit, lane, 0) on; 0 behind the row's end
    static __device__ __forceinline__ void load(const T *row, int unit, int lane, int width, float (&v)[E]) {
        if constexpr (VEC) {
            const int c = unit * kUnit + lane * E;
            if (c >= width) {
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = 0.0f;
            } else if constexpr (sizeof(T) == 2) {
                const uint4 a = *reinterpret_cast<const uint4 *>(row + c);
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
            } else {
                const float4 a = *reinterpret_cast<const float4 *>(row + c);
                v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(unit, lane, i);
                v[i] = c < width ? static_cast<float>(row[c]) : 0.0f;
            }
        }
    }
    static __device__ __forceinline__ void store(T *row, int unit, int lane, int width, const float (&v)[E]) {
        if constexpr (VEC) {
            const int c = unit * kUnit + lane * E;
            if (c >= width) return;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint4 *>(row + c) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
            else
                *reinterpret_cast<float4 *>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(unit, lane, i);
                if (c < width) row[c] = static_cast<T>(v[i]);
            }
        }
    }
    static __device__ __forceinline__ void store_codes(uint8_t *row, int unit, int lane, int width, const uint32_t (&w)[E / 4]) {
        if constexpr (VEC) {
            const int c = unit * kUnit + lane * E;
            if (c >= width) return;
            if constexpr (E == 8) *reinterpret_cast<uint2 *>(row + c) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(row + c) = w[0];
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = col(unit, lane, i);
                if (c < width) row[c] = static_cast<uint8_t>(w[0] >> (8 * i));
            }
        }
    }
};

// Rounded as the type keeps it.
template <class T>
__device__ __forceinline__ float rounded(float v) { return v; }
template <>
__device__ __forceinline__ float rounded<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// hi + lo += v, without losing v's low bits (Knuth's two-sum).
__device__ __forceinline__ void two_add(float &hi, float &lo, float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b));
    hi = s;
}

// A product as it orders: the float32 product and, in float32 tensors, its rounding error
// (bf16 products are exact).
struct Peak {
    float hi, lo;
    __device__ __forceinline__ void take(float h, float l) {
        const bool more = h > hi || (h == hi && l > lo);
        hi = more ? h : hi;
        lo = more ? l : lo;
    }
};

// 1 / sqrt(mean + eps) from the row's sum of squares, as a sum of two floats: the
// approximate root once refined (the residual 1 - m y^2 taken exactly).
__device__ __forceinline__ void inverse_root(float hi, float lo, float width, float eps, float &rh, float &rl) {
    const float q = __fdiv_rn(hi, width);
    const float q1 = __fdiv_rn(__fmaf_rn(-q, width, hi) + lo, width);
    float mh = q, ml = q1;
    two_add(mh, ml, eps);
    const float y = rsqrtf(mh);
    const float y2 = __fmul_rn(y, y), y2l = __fmaf_rn(y, y, -y2);
    const float e = __fmaf_rn(-mh, y2, 1.0f) - mh * y2l - ml * y2;
    const float c = y * (0.5f * e + 0.375f * e * e);
    rh = __fadd_rn(y, c);
    rl = c - __fsub_rn(rh, y);
    if (mh == 0.0f) rh = y, rl = 0.0f;                 // eps = 0 and a row of zeros: infinite
    if (!(hi < INFINITY)) rh = NAN, rl = 0.0f;         // an infinity or a NaN in the row
}

// The scale of a block whose largest |s gamma| is p, and r / scale (times 1 / up) as two floats.
// up is 2^64 where p is so small that r / scale would overflow, else 1.
__device__ __forceinline__ float scale_of(const Peak &p, float rh, float rl, float &ch, float &cl, float &up) {
    const float t = __fmul_rn(rh, p.hi);
    const float tl = __fmaf_rn(rh, p.hi, -t) + rl * p.hi + rh * p.lo;
    const float q = __fdiv_rn(t, 448.0f);
    float scale = __fadd_rn(q, __fdiv_rn(__fmaf_rn(-q, 448.0f, t) + tl, 448.0f));
    if (!(p.hi < INFINITY)) scale = NAN;
    if (scale == 0.0f) scale = 1.0f;                   // a block of zeros
    up = p.hi < 0x1p-60f ? 0x1p64f : 1.0f;
    const float down = p.hi < 0x1p-60f ? 0x1p-64f : 1.0f;
    const float a = rh * down;
    ch = __fdiv_rn(a, scale);
    cl = __fdiv_rn(__fmaf_rn(-ch, scale, a) + rl * down, scale);
    if (!(p.hi > 0.0f)) ch = cl = 0.0f;                // (r may be infinite there)
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

constexpr int kNormThreads = 128;      // of a CTA, at least
constexpr int kNormMaxWarps = 16;      // of a row

// Threads of row slot `slot` meet (its warps alone).
__device__ __forceinline__ void row_barrier(int slot, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(32 * warps) : "memory");
}

template <class L, int N>
__global__ void __launch_bounds__(32 * kNormMaxWarps)
add_rmsnorm_kernel(const NormArgs a) {
    using T = typename L::T;
    constexpr int E = L::E;
    constexpr bool kExact = sizeof(T) == 2;   // products of two values are exact in float32
    __shared__ float4 meet[2][kNormMaxWarps];
    griddep_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int W = a.warps, slot = warp / W, w = warp % W;
    const int slots = static_cast<int>(blockDim.x >> 5) / W;
    const float width = static_cast<float>(a.width);
    float g[N][E];
#pragma unroll
    for (int u = 0; u < N; ++u) L::load(static_cast<const T *>(a.gamma), w + u * W, lane, a.width, g[u]);
    int phase = 0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * slots + slot; t < a.T; t += static_cast<int64_t>(gridDim.x) * slots) {
        const int64_t at = t * a.width;
        float s[N][E];
#pragma unroll
        for (int u = 0; u < N; ++u) L::load(static_cast<const T *>(a.x) + at, w + u * W, lane, a.width, s[u]);
        if (a.residual) {
            float r[N][E];
#pragma unroll
            for (int u = 0; u < N; ++u) L::load(static_cast<const T *>(a.residual) + at, w + u * W, lane, a.width, r[u]);
#pragma unroll
            for (int u = 0; u < N; ++u) {
#pragma unroll
                for (int i = 0; i < E; ++i) s[u][i] = rounded<T>(s[u][i] + r[u][i]);
                L::store(static_cast<T *>(a.sum) + at, w + u * W, lane, a.width, s[u]);
            }
        }
        float hi = 0.0f, lo = 0.0f;
        Peak peak[N];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            peak[u] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float q = __fmul_rn(s[u][i], s[u][i]), p = __fmul_rn(s[u][i], g[u][i]);
                two_add(hi, lo, q);
                if (kExact) {
                    peak[u].hi = fmaxf(peak[u].hi, fabsf(p));
                } else {
                    lo += __fmaf_rn(s[u][i], s[u][i], -q);
                    const float pl = __fmaf_rn(s[u][i], g[u][i], -p);
                    peak[u].take(fabsf(p), p < 0.0f ? -pl : pl);
                }
            }
        }
        Peak top = peak[0];
#pragma unroll
        for (int u = 1; u < N; ++u) top.take(peak[u].hi, peak[u].lo);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
            two_add(hi, lo, h);
            lo += l;
            top.take(__shfl_xor_sync(0xffffffffu, top.hi, o), kExact ? 0.0f : __shfl_xor_sync(0xffffffffu, top.lo, o));
        }
        if (W > 1) {
            // the buffer alternates, so one barrier a row is enough
            float4 *m = meet[phase] + slot * W;
            phase ^= 1;
            if (lane == 0) m[w] = make_float4(hi, lo, top.hi, top.lo);
            row_barrier(slot, W);
            const float4 q = m[lane % W];
            hi = q.x, lo = q.y, top = {q.z, q.w};
            for (int o = 1; o < W; o <<= 1) {
                const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
                two_add(hi, lo, h);
                lo += l;
                top.take(__shfl_xor_sync(0xffffffffu, top.hi, o), kExact ? 0.0f : __shfl_xor_sync(0xffffffffu, top.lo, o));
            }
        }
        float rh, rl;
        inverse_root(hi, lo, width, a.eps, rh, rl);
        if (a.rstd && w == 0 && lane == 0) a.rstd[t] = rh;
        if (a.n) {
#pragma unroll
            for (int u = 0; u < N; ++u) {
                float v[E];
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = s[u][i] * g[u][i] * rh;
                L::store(static_cast<T *>(a.n) + at, w + u * W, lane, a.width, v);
            }
        }
        if (a.codes) {
            float ch, cl, up;
            if (!a.block) {
                const float scale = scale_of(top, rh, rl, ch, cl, up);
                if (w == 0 && lane == 0) a.scales[t] = scale;
            }
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int unit = w + u * W;
                if (unit * L::kUnit >= a.width) continue;
                if (a.block) {
#pragma unroll
                    for (int o = 1; o < L::kBlockLanes; o <<= 1)
                        peak[u].take(__shfl_xor_sync(0xffffffffu, peak[u].hi, o),
                                     kExact ? 0.0f : __shfl_xor_sync(0xffffffffu, peak[u].lo, o));
                    const float scale = scale_of(peak[u], rh, rl, ch, cl, up);
                    const int b = unit * (L::kUnit / 128) + lane / L::kBlockLanes;
                    if (lane % L::kBlockLanes == 0 && b * 128 < a.width) a.scales[t * ((a.width + 127) / 128) + b] = scale;
                }
                uint32_t codes[E / 4];
#pragma unroll
                for (int j = 0; j < E / 4; ++j) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = s[u][4 * j + i], y = g[u][4 * j + i];
                        const float p = __fmul_rn(x, y);
                        v[i] = scaled_odd(p * up, kExact ? 0.0f : __fmaf_rn(x, y, -p) * up, ch, cl);
                    }
                    codes[j] = e4m3x2(v[0], v[1]) | e4m3x2(v[2], v[3]) << 16;
                }
                L::store_codes(a.codes + at, unit, lane, a.width, codes);
            }
        }
    }
}

// A CTA keeps its rows' share of dgamma in registers and leaves one partial row.
template <class L, int N>
__global__ void __launch_bounds__(32 * kNormMaxWarps)
add_rmsnorm_bwd_kernel(const NormArgs a) {
    using T = typename L::T;
    constexpr int E = L::E;
    __shared__ float meet[2][kNormMaxWarps];
    extern __shared__ float shares[];         // [slots - 1][W * N * kUnit]: the other slots' dgamma
    griddep_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int W = a.warps, slot = warp / W, w = warp % W;
    const int slots = static_cast<int>(blockDim.x >> 5) / W;
    const float inv_width = 1.0f / static_cast<float>(a.width);
    float g[N][E], acc[N][E];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        L::load(static_cast<const T *>(a.gamma), w + u * W, lane, a.width, g[u]);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[u][i] = 0.0f;
    }
    int phase = 0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * slots + slot; t < a.T; t += static_cast<int64_t>(gridDim.x) * slots) {
        const int64_t at = t * a.width;
        const float r = a.rstd_in[t];
        float s[N][E], d[N][E], y[N][E];
#pragma unroll
        for (int u = 0; u < N; ++u) {
            L::load(static_cast<const T *>(a.x) + at, w + u * W, lane, a.width, s[u]);
            L::load(static_cast<const T *>(a.dn) + at, w + u * W, lane, a.width, d[u]);
            if (a.d_sum) L::load(static_cast<const T *>(a.d_sum) + at, w + u * W, lane, a.width, y[u]);
        }
        float dot = 0.0f;
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) dot += d[u][i] * g[u][i] * s[u][i];
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
        const float c = r * r * r * (dot * inv_width);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            float v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                v[i] = r * (d[u][i] * g[u][i]) - s[u][i] * c;
                if (a.d_sum) v[i] += y[u][i];
                acc[u][i] += d[u][i] * (s[u][i] * r);
            }
            L::store(static_cast<T *>(a.dx) + at, w + u * W, lane, a.width, v);
        }
    }
    // the CTA's partial row: slot 0's warps add the other slots' shares in order
    const int stride = W * N * L::kUnit;
    if (slot > 0) {
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < E; ++i) shares[(slot - 1) * stride + L::col(w + u * W, lane, i)] = acc[u][i];
    }
    if (slots > 1) __syncthreads();
    if (slot > 0) return;
    float *out = a.part + static_cast<int64_t>(blockIdx.x) * a.pitch;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = L::col(w + u * W, lane, i);
            float v = acc[u][i];
            for (int k = 1; k < slots; ++k) v += shares[(k - 1) * stride + c];
            if (c < a.width) out[c] = v;
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

// Warps of a row and units of a warp.  Many rows: four units a warp, so that a warp has
// four 16-byte loads of each array in flight and a row meets in few warps.  Few rows (no more
// than the SMs): as many warps as there are units.
struct NormShape {
    int warps, units;
};
NormShape norm_shape(int width, int unit, int64_t T, int sms) {
    const int U = (width + unit - 1) / unit;
    const int each = T <= sms ? 1 : 4;
    NormShape s = {1, 0};
    while (s.warps < kNormMaxWarps && s.warps * each < U) s.warps *= 2;
    s.units = 1;
    while (s.units * s.warps < U) s.units *= 2;
    return s;
}

template <class L, int N>
int run_norm(NormArgs a, bool backward, int sms, cudaStream_t s, int *parts) {
    const int threads = 32 * a.warps > kNormThreads ? 32 * a.warps : kNormThreads;
    const int slots = threads / (32 * a.warps);
    const size_t smem = backward ? static_cast<size_t>(slots - 1) * a.warps * N * L::kUnit * 4 : 0;
    static int occ[2][5][64] = {};   // resident CTAs an SM, by direction, log2(warps) and device
    int dev = 0, lg = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    while ((1 << lg) < a.warps) ++lg;
    int &o = occ[backward ? 1 : 0][lg][dev];
    if (o == 0) {
        int n = 0;
        const cudaError_t e = backward ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, add_rmsnorm_bwd_kernel<L, N>, threads, smem)
                                       : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, add_rmsnorm_kernel<L, N>, threads, smem);
        const int rc = cuda_status(e);
        if (rc != MLPBLK_OK) return rc;
        o = n < 1 ? 1 : n;
    }
    int64_t grid = (a.T + slots - 1) / slots;
    const int64_t most = static_cast<int64_t>(sms) * o;
    if (grid > most) grid = most;
    if (backward) {
        if (grid > kNormMaxParts) grid = kNormMaxParts;
        *parts = static_cast<int>(grid);
        return launch_pdl(add_rmsnorm_bwd_kernel<L, N>, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, s, a);
    }
    return launch_pdl(add_rmsnorm_kernel<L, N>, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, s, a);
}

template <class L>
int run_norm_lay(NormArgs a, bool backward, int sms, cudaStream_t s, int *parts) {
    const NormShape sh = norm_shape(a.width, L::kUnit, a.T, sms);
    a.warps = sh.warps;
    switch (sh.units) {
        case 1: return run_norm<L, 1>(a, backward, sms, s, parts);
        case 2: return run_norm<L, 2>(a, backward, sms, s, parts);
        case 4: return run_norm<L, 4>(a, backward, sms, s, parts);
        default: return run_norm<L, 8>(a, backward, sms, s, parts);
    }
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
    return run_norm_type(a, d.dtype, true, sms, s, parts);
}

int launch_norm_dgamma(const float *part, int parts, int64_t width, float *dgamma, int overwrite, cudaStream_t s) {
    return launch_pdl(norm_dgamma_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(1024), 0, s, part, parts,
                      static_cast<int>(norm_part_pitch(width)), static_cast<int>(width), dgamma, overwrite);
}

}  // namespace mlpblk
