// ortho.cu -- the passes over memory around the products of an orthogonalising update
// (csrc/gemm_ns.cu): the Frobenius norm, the scaled start, and Muon's momentum and weights.
//
//   momentum <- beta momentum + g,   u = g + beta momentum (Nesterov) or momentum
//   X0 = u / (|u| + eps)                      kept as sx X0 = hi + lo, two fp16 values
//   w <- w (1 - lr wd) - lr scale X
//
// Bound by HBM: 4 bytes an element of a float32 u read twice, 2 or 4 written.
#include <cuda_bf16.h>
#include <math.h>

#include "ortho.h"

namespace mlpblk {

namespace {

constexpr int kOrthoThreads = 256;

struct SourceArgs {
    OrthoSource u;
    int64_t n;          // elements of a matrix
    bool vec;           // matrices are whole 16-byte pieces
};

// Four neighbouring elements of u, at `at` counted through the batch (`count` of them exist).  first: the momentum is
// updated on the way; otherwise it has been.
template <bool FIRST>
__device__ __forceinline__ void source4(const OrthoSource &u, float gs, int64_t at, int count, bool vec, float (&v)[4]) {
    if (u.u) {
        if (u.dtype == MLPBLK_FP32) {
            const float *p = static_cast<const float *>(u.u) + at;
            if (vec && count == 4) {
                const float4 a = *reinterpret_cast<const float4 *>(p);
                v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = i < count ? p[i] : 0.0f;
            }
        } else {
            const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(u.u) + at;
            if (vec && count == 4) {
                const uint2 a = *reinterpret_cast<const uint2 *>(p);
                v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
                v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = i < count ? __bfloat162float(p[i]) : 0.0f;
            }
        }
        return;
    }
    float m[4], g[4];
    if (vec && count == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(u.momentum + at), b = *reinterpret_cast<const float4 *>(u.grad + at);
        m[0] = a.x; m[1] = a.y; m[2] = a.z; m[3] = a.w;
        g[0] = b.x; g[1] = b.y; g[2] = b.z; g[3] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = i < count ? u.momentum[at + i] : 0.0f;
            g[i] = i < count ? u.grad[at + i] : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        g[i] *= gs;
        if (FIRST) m[i] = __fmaf_rn(u.beta, m[i], g[i]);
        v[i] = u.nesterov ? __fmaf_rn(u.beta, m[i], g[i]) : m[i];
    }
    if (FIRST) {
        if (vec && count == 4) {
            *reinterpret_cast<float4 *>(u.momentum + at) = make_float4(m[0], m[1], m[2], m[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < count) u.momentum[at + i] = m[i];
        }
    }
}

// Squares of any size (Blue's three accumulators): a group of four whose largest value is
// beyond 2^60 or below 2^-40 is scaled by a power of two before it is squared.
struct Squares {
    float big, mid, small;   // times 2^-160, 1, 2^160
};
__device__ __forceinline__ void add_squares(Squares &q, const float (&v)[4]) {
    const float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    if (m >= 0x1p-40f && m <= 0x1p60f) {
        q.mid += (v[0] * v[0] + v[1] * v[1]) + (v[2] * v[2] + v[3] * v[3]);
    } else {
        const float f = m < 1.0f ? 0x1p80f : 0x1p-80f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s += (v[i] * f) * (v[i] * f);   // NaN and infinities stay what they are
        if (m < 1.0f) q.small += s;
        else q.big += s;
    }
}

__global__ void __launch_bounds__(kOrthoThreads)
ortho_norm_kernel(const SourceArgs a, double *__restrict__ partial) {
    __shared__ double red[kOrthoThreads / 32];
    griddep_enter();
    const int64_t base = static_cast<int64_t>(blockIdx.y) * a.n;
    const float gs = a.u.grad_scale ? *a.u.grad_scale : 1.0f;
    const int64_t groups = (a.n + 3) / 4;
    Squares q = {0.0f, 0.0f, 0.0f};
    const int64_t step = static_cast<int64_t>(gridDim.x) * kOrthoThreads;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kOrthoThreads + threadIdx.x;
    for (; i + 3 * step < groups; i += 4 * step) {   // four loads in flight
        float v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            source4<true>(a.u, gs, base + (i + k * step) * 4, static_cast<int>(min(static_cast<int64_t>(4), a.n - (i + k * step) * 4)), a.vec, v[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) add_squares(q, v[k]);
    }
    for (; i < groups; i += step) {
        float v[4];
        source4<true>(a.u, gs, base + i * 4, static_cast<int>(min(static_cast<int64_t>(4), a.n - i * 4)), a.vec, v);
        add_squares(q, v);
    }
    double s = static_cast<double>(q.big) * 0x1p160 + static_cast<double>(q.mid) + static_cast<double>(q.small) * 0x1p-160;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kOrthoThreads / 32; ++w) s += red[w];
        partial[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
    }
}

struct ScaleArgs {
    SourceArgs s;
    int64_t rows, cols, pitch;
    const double *partial;
    int parts;
    float eps, sx;
    __half *x, *x_lo;
};

__global__ void __launch_bounds__(kOrthoThreads)
ortho_scale_kernel(const ScaleArgs a) {
    __shared__ float factor[2];
    griddep_enter();
    const int b = static_cast<int>(blockIdx.y);
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int p = threadIdx.x; p < a.parts; p += 32) s += a.partial[static_cast<int64_t>(b) * a.parts + p];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            // a power of two first, so that neither factor leaves float32's range
            const double d = sqrt(s) + static_cast<double>(a.eps);
            int e = 0;
            if (d > 0.0 && d < INFINITY) frexp(d, &e);
            e = min(max(e, -120), 120);
            factor[0] = ldexpf(1.0f, -e);
            factor[1] = static_cast<float>(static_cast<double>(a.sx) / ldexp(d, -e));
        }
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1];
    const float gs = a.s.u.grad_scale ? *a.s.u.grad_scale : 1.0f;
    const int64_t per = (a.cols + 3) / 4, groups = a.rows * per;
    const int64_t base = static_cast<int64_t>(b) * a.s.n, out = static_cast<int64_t>(b) * a.rows * a.pitch;
    const bool vec = a.cols % 4 == 0;   // (a.s.vec says it of whole matrices)
    const int64_t step = static_cast<int64_t>(gridDim.x) * kOrthoThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kOrthoThreads + threadIdx.x; i < groups; i += step) {
        const int64_t r = i / per, c = (i - r * per) * 4;
        float v[4];
        source4<false>(a.s.u, gs, base + r * a.cols + c, static_cast<int>(min(static_cast<int64_t>(4), a.cols - c)), vec, v);
        __half hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float w = (v[k] * f0) * f1;
            hi[k] = __float2half_rn(w);
            lo[k] = __float2half_rn(w - __half2float(hi[k]));
        }
        // (the pitch is a multiple of 64: the last group's zeros stay in the row)
        *reinterpret_cast<uint2 *>(a.x + out + r * a.pitch + c) = *reinterpret_cast<const uint2 *>(hi);
        if (a.x_lo) *reinterpret_cast<uint2 *>(a.x_lo + out + r * a.pitch + c) = *reinterpret_cast<const uint2 *>(lo);
    }
}

__global__ void __launch_bounds__(kOrthoThreads)
muon_apply_kernel(const __half *__restrict__ x, int64_t rows, int64_t cols, int64_t pitch, float keep, float rate,
                  float *__restrict__ master, void *__restrict__ weight, int dtype) {
    griddep_enter();
    const int64_t per = (cols + 3) / 4, groups = rows * per;
    const int64_t base = static_cast<int64_t>(blockIdx.y) * rows * cols, in = static_cast<int64_t>(blockIdx.y) * rows * pitch;
    const bool vec = cols % 4 == 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kOrthoThreads + threadIdx.x; i < groups;
         i += static_cast<int64_t>(gridDim.x) * kOrthoThreads) {
        const int64_t r = i / per, c = (i - r * per) * 4, at = base + r * cols + c;
        const uint2 h = *reinterpret_cast<const uint2 *>(x + in + r * pitch + c);
        const float2 h0 = __half22float2(*reinterpret_cast<const __half2 *>(&h.x)), h1 = __half22float2(*reinterpret_cast<const __half2 *>(&h.y));
        const float o[4] = {h0.x, h0.y, h1.x, h1.y};
        float w[4];
        if (vec) {
            const float4 m = *reinterpret_cast<const float4 *>(master + at);
            w[0] = m.x; w[1] = m.y; w[2] = m.z; w[3] = m.w;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = w[k] * keep - rate * o[k];
            *reinterpret_cast<float4 *>(master + at) = make_float4(w[0], w[1], w[2], w[3]);
            if (weight && dtype == MLPBLK_BF16) {
                __nv_bfloat162 q[2] = {__floats2bfloat162_rn(w[0], w[1]), __floats2bfloat162_rn(w[2], w[3])};
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(weight) + at) = *reinterpret_cast<const uint2 *>(q);
            } else if (weight) {
                *reinterpret_cast<float4 *>(static_cast<float *>(weight) + at) = make_float4(w[0], w[1], w[2], w[3]);
            }
        } else {
            for (int k = 0; k < 4 && c + k < cols; ++k) {
                const float v = master[at + k] * keep - rate * o[k];
                master[at + k] = v;
                if (weight && dtype == MLPBLK_BF16) static_cast<__nv_bfloat16 *>(weight)[at + k] = __float2bfloat16_rn(v);
                else if (weight) static_cast<float *>(weight)[at + k] = v;
            }
        }
    }
}

// CTAs a matrix: enough for every SM, eight groups of four a thread where there is that much.
unsigned ctas_of(int64_t groups, int batch, int sms, int64_t most) {
    int64_t n = (groups + kOrthoThreads * 4 - 1) / (kOrthoThreads * 4);
    const int64_t cap = most / batch > 0 ? most / batch : 1, wave = static_cast<int64_t>(sms) * 6 / batch + 1;
    if (n > cap) n = cap;
    if (n > wave) n = wave;
    return static_cast<unsigned>(n < 1 ? 1 : n);
}

}  // namespace

int launch_ortho_norm(const OrthoSource &u, int64_t n, int batch, double *partial, int *parts, int sms, cudaStream_t s) {
    SourceArgs a = {u, n, n % 4 == 0};
    const unsigned ctas = ctas_of((n + 3) / 4, batch, sms, kOrthoNormParts);
    *parts = static_cast<int>(ctas);
    return launch_pdl(ortho_norm_kernel, dim3(ctas, static_cast<unsigned>(batch)), dim3(kOrthoThreads), 0, s, a, partial);
}

int launch_ortho_scale(const OrthoSource &u, int64_t rows, int64_t cols, int batch, const double *partial, int parts, float eps,
                       float sx, __half *x, __half *x_lo, int sms, cudaStream_t s) {
    ScaleArgs a = {};
    a.s = {u, rows * cols, false};
    a.rows = rows;
    a.cols = cols;
    a.pitch = ortho_pitch(cols);
    a.partial = partial;
    a.parts = parts;
    a.eps = eps;
    a.sx = sx;
    a.x = x;
    a.x_lo = x_lo;
    const unsigned ctas = ctas_of(rows * ((cols + 3) / 4), batch, sms, INT32_MAX);
    return launch_pdl(ortho_scale_kernel, dim3(ctas, static_cast<unsigned>(batch)), dim3(kOrthoThreads), 0, s, a);
}

int launch_muon_apply(const __half *x, int64_t rows, int64_t cols, int batch, float keep, float rate, float *master,
                      void *weight, int dtype, int sms, cudaStream_t s) {
    const unsigned ctas = ctas_of(rows * ((cols + 3) / 4), batch, sms, INT32_MAX);
    return launch_pdl(muon_apply_kernel, dim3(ctas, static_cast<unsigned>(batch)), dim3(kOrthoThreads), 0, s, x, rows, cols,
                      ortho_pitch(cols), keep, rate, master, weight, dtype);
}

}  // namespace mlpblk
