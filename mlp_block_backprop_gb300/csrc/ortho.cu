// ortho.cu -- the passes over memory around the products of an orthogonalising update
// (csrc/gemm_ns.cu): the Frobenius norm, the scaled start, and Muon's momentum and weights.
//
//   momentum <- beta momentum + g,   u = g + beta momentum (Nesterov) or momentum
//   X0 = u / (|u| + eps)                      kept as sx X0 = hi + lo, two fp16 values
//   w <- w (1 - lr wd) - lr scale X
//
// Bound by HBM: 4 bytes an element of a float32 u read twice, 2 or 4 written (16384 x 4096: 52 us for the
// norm, 82 for X0, 6.5 TB/s).
#include <cuda_bf16.h>
#include <math.h>

#include "ortho.h"

namespace mlpblk {

namespace {

constexpr int kOrthoThreads = 256;

enum SourceKind : int { kSourceF32 = 0, kSourceBf16 = 1, kSourceMomentum = 2 };

struct SourceArgs {
    OrthoSource u;
    int64_t n;          // elements of a matrix
};

constexpr int kPiece = 8;   // neighbouring elements that a thread takes at once

// Up to eight neighbouring elements of u, at `at` counted through the batch; `count` of them exist, the
// others are 0.  VEC: all eight, at a 16-byte boundary.  FIRST: the momentum is updated on the way; otherwise it
// has been.
template <int KIND, bool FIRST, bool VEC>
__device__ __forceinline__ void source(const OrthoSource &u, float gs, int64_t at, int count, float (&v)[kPiece]) {
    if constexpr (KIND == kSourceF32) {
        const float *p = static_cast<const float *>(u.u) + at;
        if (VEC) {
            const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v[i] = i < count ? p[i] : 0.0f;
        }
    } else if constexpr (KIND == kSourceBf16) {
        const uint16_t *p = static_cast<const uint16_t *>(u.u) + at;
        if (VEC) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v[i] = i < count ? __uint_as_float(static_cast<uint32_t>(p[i]) << 16) : 0.0f;
        }
    } else {
        float m[kPiece], g[kPiece];
        if (VEC) {
#pragma unroll
            for (int i = 0; i < kPiece; i += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(u.momentum + at + i), b = *reinterpret_cast<const float4 *>(u.grad + at + i);
                m[i] = a.x; m[i + 1] = a.y; m[i + 2] = a.z; m[i + 3] = a.w;
                g[i] = b.x; g[i + 1] = b.y; g[i + 2] = b.z; g[i + 3] = b.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                m[i] = i < count ? u.momentum[at + i] : 0.0f;
                g[i] = i < count ? u.grad[at + i] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            g[i] *= gs;
            if (FIRST) m[i] = __fmaf_rn(u.beta, m[i], g[i]);
            v[i] = u.nesterov ? __fmaf_rn(u.beta, m[i], g[i]) : m[i];
        }
        if (FIRST) {
            if (VEC) {
                *reinterpret_cast<float4 *>(u.momentum + at) = make_float4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<float4 *>(u.momentum + at + 4) = make_float4(m[4], m[5], m[6], m[7]);
            } else {
#pragma unroll
                for (int i = 0; i < kPiece; ++i)
                    if (i < count) u.momentum[at + i] = m[i];
            }
        }
    }
}

// Squares of any size (Blue's three accumulators): a piece whose largest value is beyond 2^40 or below
// 2^-40 is scaled by a power of two before it is squared.  A thread adds up to 2^23 pieces of eight: below 2^106 in
// `mid`, 2^122 in `big`.
struct Squares {
    float big, mid, small;   // times 2^-160, 1, 2^160
};
__device__ __forceinline__ void add_squares(Squares &q, const float (&v)[kPiece]) {
    float m = fabsf(v[0]), s = 0.0f;
#pragma unroll
    for (int i = 1; i < kPiece; ++i) m = fmaxf(m, fabsf(v[i]));
    if (m >= 0x1p-40f && m <= 0x1p40f) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) s = __fmaf_rn(v[i], v[i], s);
        q.mid += s;
    } else {
        const float f = m < 1.0f ? 0x1p80f : 0x1p-80f;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) s += (v[i] * f) * (v[i] * f);   // NaN and infinities stay what they are
        if (m < 1.0f) q.small += s;
        else q.big += s;
    }
}

// Bound by HBM: eight pieces in flight a thread (16384 x 4096 float32: 52 us, 5.2 TB/s).
template <int KIND, bool VEC>
__global__ void __launch_bounds__(kOrthoThreads)
ortho_norm_kernel(const SourceArgs a, double *__restrict__ partial) {
    __shared__ double red[kOrthoThreads / 32];
    griddep_enter();
    const int64_t base = static_cast<int64_t>(blockIdx.y) * a.n;
    const float gs = a.u.grad_scale ? *a.u.grad_scale : 1.0f;
    Squares q = {0.0f, 0.0f, 0.0f};
    const int64_t step = static_cast<int64_t>(gridDim.x) * kOrthoThreads * kPiece;
    int64_t i = (static_cast<int64_t>(blockIdx.x) * kOrthoThreads + threadIdx.x) * kPiece;
    constexpr int kDeep = 8;
    for (; i + (kDeep - 1) * step + kPiece <= a.n; i += kDeep * step) {
        float v[kDeep][kPiece];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) source<KIND, true, VEC>(a.u, gs, base + i + k * step, kPiece, v[k]);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) add_squares(q, v[k]);
    }
    for (; i < a.n; i += step) {
        float v[kPiece];
        const int count = static_cast<int>(min(static_cast<int64_t>(kPiece), a.n - i));
        source<KIND, true, VEC>(a.u, gs, base + i, count, v);   // (VEC: matrices are whole pieces)
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
    int rows, cols;
    int64_t pitch;
    const double *partial;
    int parts;
    float eps, sx;
    __half *x, *x_lo;
};

template <int KIND, bool VEC>
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
            factor[1] = d == 0.0 ? 0.0f : static_cast<float>(static_cast<double>(a.sx) / ldexp(d, -e));   // (eps = 0 and a matrix of zeros)
        }
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1];
    const float gs = a.s.u.grad_scale ? *a.s.u.grad_scale : 1.0f;
    // a thread walks the pieces of the rows by steps of the grid
    const int per = (a.cols + kPiece - 1) / kPiece;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kOrthoThreads, first = static_cast<int64_t>(blockIdx.x) * kOrthoThreads + threadIdx.x;
    const int step_r = static_cast<int>(step / per), step_c = static_cast<int>(step - static_cast<int64_t>(step_r) * per);
    int64_t r = first / per;
    int c = static_cast<int>(first - r * per);
    const int64_t base = static_cast<int64_t>(b) * a.s.n, out = static_cast<int64_t>(b) * a.rows * a.pitch;
    while (r < a.rows) {
        float v[kPiece];
        source<KIND, false, VEC>(a.s.u, gs, base + r * a.cols + c * kPiece, min(kPiece, a.cols - c * kPiece), v);
        __half2 hi[kPiece / 2], lo[kPiece / 2];
#pragma unroll
        for (int k = 0; k < kPiece / 2; ++k) {
            const float x = (v[2 * k] * f0) * f1, y = (v[2 * k + 1] * f0) * f1;
            hi[k] = __floats2half2_rn(x, y);
            const float2 h = __half22float2(hi[k]);
            lo[k] = __floats2half2_rn(x - h.x, y - h.y);
        }
        // (the pitch is a multiple of 64: the last piece's zeros stay in the row)
        const int64_t at = out + r * a.pitch + c * kPiece;
        *reinterpret_cast<uint4 *>(a.x + at) = *reinterpret_cast<const uint4 *>(hi);
        if (a.x_lo) *reinterpret_cast<uint4 *>(a.x_lo + at) = *reinterpret_cast<const uint4 *>(lo);
        r += step_r;
        c += step_c;
        if (c >= per) {
            c -= per;
            ++r;
        }
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

// CTAs a matrix of `pieces` pieces: four pieces a thread where there are that many, `resident` CTAs an SM (one
// wave of them).
unsigned ctas_of(int64_t pieces, int batch, int sms, int resident, int64_t most) {
    int64_t n = (pieces + kOrthoThreads * 4 - 1) / (kOrthoThreads * 4);
    const int64_t cap = most / batch > 0 ? most / batch : 1, wave = static_cast<int64_t>(sms) * resident / batch;
    if (n > cap) n = cap;
    if (n > wave) n = wave;
    return static_cast<unsigned>(n < 1 ? 1 : n);
}

int kind_of(const OrthoSource &u) { return !u.u ? kSourceMomentum : (u.dtype == MLPBLK_FP32 ? kSourceF32 : kSourceBf16); }

}  // namespace

int launch_ortho_norm(const OrthoSource &u, int64_t n, int batch, double *partial, int *parts, int sms, cudaStream_t s) {
    const SourceArgs a = {u, n};
    const unsigned ctas = ctas_of((n + kPiece - 1) / kPiece, batch, sms, 3, kOrthoNormParts);
    *parts = static_cast<int>(ctas);
    const bool vec = n % kPiece == 0;
    void (*const kernels[3][2])(SourceArgs, double *) = {{ortho_norm_kernel<kSourceF32, false>, ortho_norm_kernel<kSourceF32, true>},
                                                         {ortho_norm_kernel<kSourceBf16, false>, ortho_norm_kernel<kSourceBf16, true>},
                                                         {ortho_norm_kernel<kSourceMomentum, false>, ortho_norm_kernel<kSourceMomentum, true>}};
    return launch_pdl(kernels[kind_of(u)][vec], dim3(ctas, static_cast<unsigned>(batch)), dim3(kOrthoThreads), 0, s, a, partial);
}

int launch_ortho_scale(const OrthoSource &u, int64_t rows, int64_t cols, int batch, const double *partial, int parts, float eps,
                       float sx, __half *x, __half *x_lo, int sms, cudaStream_t s) {
    ScaleArgs a = {};
    a.s = {u, rows * cols};
    a.rows = static_cast<int>(rows);
    a.cols = static_cast<int>(cols);
    a.pitch = ortho_pitch(cols);
    a.partial = partial;
    a.parts = parts;
    a.eps = eps;
    a.sx = sx;
    a.x = x;
    a.x_lo = x_lo;
    const unsigned ctas = ctas_of(rows * ((cols + kPiece - 1) / kPiece), batch, sms, 8, INT32_MAX);
    const bool vec = cols % kPiece == 0;
    void (*const kernels[3][2])(ScaleArgs) = {{ortho_scale_kernel<kSourceF32, false>, ortho_scale_kernel<kSourceF32, true>},
                                              {ortho_scale_kernel<kSourceBf16, false>, ortho_scale_kernel<kSourceBf16, true>},
                                              {ortho_scale_kernel<kSourceMomentum, false>, ortho_scale_kernel<kSourceMomentum, true>}};
    return launch_pdl(kernels[kind_of(u)][vec], dim3(ctas, static_cast<unsigned>(batch)), dim3(kOrthoThreads), 0, s, a);
}

int launch_muon_apply(const __half *x, int64_t rows, int64_t cols, int batch, float keep, float rate, float *master,
                      void *weight, int dtype, int sms, cudaStream_t s) {
    const unsigned ctas = ctas_of(rows * ((cols + kPiece - 1) / kPiece), batch, sms, 8, INT32_MAX);
    return launch_pdl(muon_apply_kernel, dim3(ctas, static_cast<unsigned>(batch)), dim3(kOrthoThreads), 0, s, x, rows, cols,
                      ortho_pitch(cols), keep, rate, master, weight, dtype);
}

}  // namespace mlpblk
