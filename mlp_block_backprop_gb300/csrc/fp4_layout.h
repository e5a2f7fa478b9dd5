// fp4_layout.h -- the layout of an MXFP4 matrix (include/mlpblk.h) and the launchers
// of its kernels.
#pragma once

#include "mlpblk_internal.h"

namespace mlpblk {

constexpr int kFp4TileBytes = 512;  // scales of 128 rows x 4 blocks (128 columns)

// Bytes of a row of codes: whole blocks of 32 values.
__host__ __device__ inline int64_t fp4_row_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }

// Scale tiles along a row: an even count, so that a pipeline stage of 256 columns is
// one copy of two tiles.
__host__ __device__ inline int64_t fp4_col_tiles(int64_t cols) { return (cols + 255) / 256 * 2; }

// Bytes of the scales of one matrix.
__host__ __device__ inline int64_t fp4_scales_bytes(int64_t rows, int64_t cols) {
    return (rows + 127) / 128 * fp4_col_tiles(cols) * kFp4TileBytes;
}

// Host: MXFP4 quantisation and reading back (fp4.cu).
int launch_fp4_quantize(int dtype, const void *x, const int *row_map, int map_div, int source_rows, int64_t rows,
                        int64_t cols, int batch, bool transposed, bool relu2, uint8_t *codes, uint8_t *scales, cudaStream_t s);
int launch_fp4_dequantize(int dtype, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                          int batch, void *y, cudaStream_t s);

// What a product walks over (gemm_f4.cu): one pair of matrices, the rows of sorted
// segments with an expert's B each, or K ranges of sorted segments with a C each.
enum Fp4Mode : int { kFp4Dense = 0, kFp4GroupRows = 1, kFp4GroupK = 2 };

struct Fp4Product {
    int mode;              // Fp4Mode
    int64_t m, n, k;
    int experts;           // grouped modes
    int64_t max_rows;      // kFp4GroupRows: rows of one expert, at most
    const uint8_t *a, *sa, *b, *sb;
    const int *count, *seg;
    void *c;
    int out_dtype, accumulate;
};

// The kernel that a product takes (a rule on sizes and types alone).
struct Fp4Choice {
    bool pair;     // f4_pair, else f4_small
    bool tma;      // rows of C are whole 16-byte pieces: f4_pair stores them by TMA
    int split;     // f4_small: CTAs that share a tile's K
    int workers;   // CTAs, CTA pairs or clusters that walk the tiles
};
Fp4Choice choose_fp4_matmul(const Fp4Product &p, int num_sms);

int launch_fp4_matmul(const Fp4Product &p, int num_sms, cudaStream_t s);
int take_device_error_gemm_f4();

}  // namespace mlpblk
