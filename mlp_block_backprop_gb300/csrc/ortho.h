// ortho.h -- what the orthogonalising update's translation units share: its matrices in the
// workspace and the products of a Newton-Schulz step.
#pragma once

#include <cuda_fp16.h>

#include "mlpblk_internal.h"

namespace mlpblk {

constexpr int kOrthoNormParts = 2048;   // partial sums of squares, over the whole batch, at most

// Elements of a row of a workspace matrix: whole 128-byte lines of fp16.
inline int64_t ortho_pitch(int64_t cols) { return (cols + 63) / 64 * 64; }

// Products of one step on a batch of matrices.  X is [rows, cols] (pitch elements a row);
// G, P and the other y are square on the short side and symmetric.
//   kNsGram    out = alpha X X^T (rows <= cols) or alpha X^T X
//   kNsSquare  out = b Y + c Y Y, diag_out = what rounding took from out's diagonal
//   kNsApply   out = (a + diag) Y + P Y
//   kNsJoin    out = (a + diag) Y + P Y + b P with Y's own remainders diag2: the polynomial of two
//              steps, (a I + P) (b I + Y) less a b I; its diagonal goes to diag_out whole, and is zero in out
//   kNsUpdate  out = (a + diag) X + P X or X P;  o: alpha times it in bf16 instead
// diag: the remainders of P's diagonal (after kNsJoin, the diagonal).
enum NsOp : int { kNsGram = 0, kNsSquare = 1, kNsUpdate = 2, kNsApply = 3, kNsJoin = 4 };

struct NsProduct {
    int op;
    bool tall;                 // rows > cols
    int64_t rows, cols;        // of X
    int batch;
    const __half *x, *x_lo;    // kNsGram, kNsUpdate: X; x_lo NULL: none
    const __half *y;           // kNsSquare, kNsApply, kNsJoin: Y
    const __half *p;           // kNsApply, kNsJoin, kNsUpdate: P
    const float *diag, *diag2; // [batch][ortho_pitch(short side)]
    float *diag_out;
    __half *out, *out_lo;      // out_lo NULL: none
    void *o;                   // kNsUpdate: bf16 [batch][rows][cols] in place of out
    float alpha, a, b, c;
};

int launch_ns_product(const NsProduct &p, int sms, cudaStream_t s);

// All steps of small matrices in one launch, from x[0]; the last X in x[steps & 1], or o.
struct NsFusedProblem {
    int64_t rows, cols;
    int batch, steps;
    __half *x[2], *lo, *g, *p;
    float *diag;
    void *o;
    float sx;
    const float (*coefficients)[3];
};
bool ns_fused_fits(int64_t rows, int64_t cols, int batch, int sms);
int launch_ns_fused(const NsFusedProblem &p, cudaStream_t s);
int take_device_error_gemm_ns();

// Where a step's input comes from: a matrix, or momentum and gradient.
struct OrthoSource {
    const void *u;             // bf16 or float32; NULL: momentum
    int dtype;
    float *momentum;
    const float *grad, *grad_scale;
    float beta;
    int nesterov;
};

// Partial sums of squares (momentum <- beta momentum + grad first); *parts of them a matrix.
int launch_ortho_norm(const OrthoSource &u, int64_t n, int batch, double *partial, int *parts, int sms, cudaStream_t s);
// x (+ x_lo) = sx * u / (|u| + eps).
int launch_ortho_scale(const OrthoSource &u, int64_t rows, int64_t cols, int batch, const double *partial, int parts, float eps,
                       float sx, __half *x, __half *x_lo, int sms, cudaStream_t s);
// master = master * keep - rate * x; weight = its rounded copy.
int launch_muon_apply(const __half *x, int64_t rows, int64_t cols, int batch, float keep, float rate, float *master,
                      void *weight, int dtype, int sms, cudaStream_t s);

}  // namespace mlpblk
