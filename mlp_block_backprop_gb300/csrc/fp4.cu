// fp4.cu -- MXFP4 quantisation and reading back ("Where Quantization Fits": a storage
// and arithmetic policy for particular tensor edges; the format is the OCP
// Microscaling Formats specification's MXFP4: blocks of 32 E2M1 codes with one E8M0
// scale).
//
//   scale byte = max(exponent field of max|v| - 2, 0)      (2^(byte - 127))
//   code       = E2M1(v * 2^(127 - byte)), to nearest even, saturated at 6
//
// The scaling is by a power of two, so a code is rounded once and is the same
// whatever precision computes it.  Both directions are bound by HBM: x is read once,
// 17 bytes a block of 32 written.
#include "fp4_layout.h"

namespace mlpblk {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// 8 floats -> 8 E2M1 codes (first value in the lowest four bits), nearest-even,
// saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n"
        "  .reg .b8 a, b, c, d;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "  mov.b32 %0, {a, b, c, d};\n"
        "}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The scale byte of a block whose largest |v| has the bits `m` (NaN and infinities
// order above every finite value).
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
    const uint32_t e = m >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(127 - byte): what a block's values are multiplied by (0 for a NaN block: its
// codes are zero).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

template <bool RELU2>
__device__ __forceinline__ float act(float v) {
    if (!RELU2) return v;
    const float r = v < 0.0f ? 0.0f : v;  // keeps a NaN
    return r * r;
}

template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// The 8 values x[0..8) of a row from column c on (0 at and behind cols).  VEC: the
// row is 16-byte aligned and cols a multiple of a 16-byte access.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T *row, int64_t c, int64_t cols, float (&v)[8]) {
    if (VEC && sizeof(T) == 2) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (c < cols) u = __ldg(reinterpret_cast<const uint4 *>(row + c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else if (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c + 4 * h < cols) u = __ldg(reinterpret_cast<const float4 *>(row + c + 4 * h));
            v[4 * h] = u.x;
            v[4 * h + 1] = u.y;
            v[4 * h + 2] = u.z;
            v[4 * h + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float<T>(__ldg(row + c + i)) : 0.0f;
    }
}

// Q's row r of x under a row map (Fp4Args): the source row, or -1 for a row of zeros.
__device__ __forceinline__ int64_t source_row(const int *row_map, int map_div, int64_t r) {
    if (!row_map) return r;
    const int m = row_map[r];
    return m < 0 ? -1 : (map_div > 0 ? m / map_div : r);
}

// Blocks along the source's rows.  An item is the rows r, r + 32, r + 64, r + 96 of a
// 128-row scale tile over 256 columns: a lane holds 8 consecutive values of each, a
// block is four lanes, and the four rows' scales of 4 blocks are 16 consecutive
// bytes of a tile (one store), with the rows' neighbours filling the rest of a
// sector.  The four rows' loads are in flight together.
template <class T, bool VEC, bool RELU2>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const T *__restrict__ x, const int *__restrict__ row_map, int map_div, int64_t rows, int64_t cols,
                     int64_t row_tiles, int64_t chunks, int64_t items, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales) {
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const int64_t ld = fp4_row_bytes(cols);
    for (int64_t it = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5); it < items;
         it += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t chunk = it % chunks;
        const int64_t q = it / chunks;
        const int64_t tile = q / 32;  // of the whole batch
        const int64_t mat = tile / row_tiles;
        const int64_t r0 = (tile - mat * row_tiles) * 128 + q % 32;
        const int64_t c = chunk * 256 + lane * 8;
        float v[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + 32 * j;
            const int64_t src = r < rows ? source_row(row_map, map_div, r) : -1;
            if (src >= 0) {
                load8<T, VEC>(x + (mat * rows + src) * cols, c, cols, v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            }
        }
        uint32_t word[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] = act<RELU2>(v[j][i]);
                m = max(m, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
            }
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t sb = scale_byte(m);
            const float inv = scale_inverse(sb);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = sb == 255u ? 0.0f : v[j][i] * inv;
            const int64_t r = r0 + 32 * j;
            if (r < rows && c < 2 * ld)
                *reinterpret_cast<uint32_t *>(codes + (mat * rows + r) * ld + c / 2) = e2m1x8(v[j]);
            // the four blocks' bytes of this half warp
            uint32_t w = sb << (8 * ((lane >> 2) & 3));
            w |= __shfl_xor_sync(0xffffffffu, w, 4);
            w |= __shfl_xor_sync(0xffffffffu, w, 8);
            word[j] = w;
        }
        if ((lane & 15) == 0) {
            uint8_t *st = scales + ((tile * chunks + chunk) * 2 + (lane >> 4)) * 512 + (q % 32) * 16;
            *reinterpret_cast<uint4 *>(st) = make_uint4(word[0], word[1], word[2], word[3]);
        }
    }
}

// Two neighbouring values of a source row, columns c and c + 1 (0 at and behind
// `width`).  VEC: width is even, so a pair is one aligned access.
template <class T, bool VEC>
__device__ __forceinline__ float2 load2(const T *row, int64_t c, int64_t width) {
    float2 f = make_float2(0.0f, 0.0f);
    if (VEC) {
        if (c < width) {
            if (sizeof(T) == 2) {
                const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(row + c));
                f = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
            } else {
                f = __ldg(reinterpret_cast<const float2 *>(row + c));
            }
        }
    } else {
        if (c < width) f.x = to_float<T>(__ldg(row + c));
        if (c + 1 < width) f.y = to_float<T>(__ldg(row + c + 1));
    }
    return f;
}

// Blocks along the source's columns: Q = x^T, Q's rows are x's columns.  A CTA
// takes 64 columns and 256 rows of x; warp w holds rows 32w .. 32w + 31 of it, two
// columns a lane, so a block is one lane's 32 registers.  The codes cross shared
// memory to leave as 128 consecutive bytes a row of Q.
constexpr int kTCols = 64;              // x's columns of a CTA (Q's rows)
constexpr int kTPitch = 128 + 16;       // bytes of a Q row in shared memory

template <class T, bool VEC, bool RELU2>
__global__ void __launch_bounds__(kThreads)
quantize_cols_kernel(const T *__restrict__ x, const int *__restrict__ row_map, int map_div, int64_t rows, int64_t cols,
                     int64_t row_tiles, int64_t chunks, int64_t items, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales) {
    __shared__ __align__(16) uint8_t sc[kTCols][kTPitch];
    __shared__ __align__(8) uint8_t ss[kTCols][8];
    griddep_enter();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t ld = fp4_row_bytes(cols);
    const int64_t halves = row_tiles * 2;  // 64-row parts of the scale tiles of one matrix
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t half = it % halves;
        const int64_t q = it / halves;
        const int64_t chunk = q % chunks, mat = q / chunks;
        const int64_t r0 = half * kTCols;             // Q's first row
        const int64_t c0 = chunk * 256 + wid * 32;    // Q's first column of this warp: x's row
        const T *base = x + mat * rows * cols;
        const int64_t own = c0 + lane;
        const int64_t mine = own < cols ? source_row(row_map, map_div, own) : -1;
        float a[32], b[32];
        uint32_t ma = 0, mb = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int64_t src = __shfl_sync(0xffffffffu, mine, i);
            float2 f = make_float2(0.0f, 0.0f);
            if (src >= 0) f = load2<T, VEC>(base + src * rows, r0 + 2 * lane, rows);
            a[i] = f.x;
            b[i] = f.y;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            a[i] = act<RELU2>(a[i]);
            b[i] = act<RELU2>(b[i]);
            ma = max(ma, __float_as_uint(a[i]) & 0x7FFFFFFFu);
            mb = max(mb, __float_as_uint(b[i]) & 0x7FFFFFFFu);
        }
        const uint32_t sa = scale_byte(ma), sb = scale_byte(mb);
        const float ia = scale_inverse(sa), ib = scale_inverse(sb);
        uint32_t wa[4], wb[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float va[8], vb[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                va[i] = sa == 255u ? 0.0f : a[8 * g + i] * ia;
                vb[i] = sb == 255u ? 0.0f : b[8 * g + i] * ib;
            }
            wa[g] = e2m1x8(va);
            wb[g] = e2m1x8(vb);
        }
        *reinterpret_cast<uint4 *>(&sc[2 * lane][wid * 16]) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
        *reinterpret_cast<uint4 *>(&sc[2 * lane + 1][wid * 16]) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
        ss[2 * lane][wid] = static_cast<uint8_t>(sa);
        ss[2 * lane + 1][wid] = static_cast<uint8_t>(sb);
        __syncthreads();
        for (int p = threadIdx.x; p < kTCols * 8; p += kThreads) {
            const int r = p >> 3, blk = p & 7;
            const int64_t at = chunk * 128 + blk * 16;
            if (r0 + r < rows && at < ld)
                *reinterpret_cast<uint4 *>(codes + (mat * rows + r0 + r) * ld + at) =
                    *reinterpret_cast<const uint4 *>(&sc[r][blk * 16]);
        }
        if (threadIdx.x < kTCols * 2) {
            const int r = threadIdx.x >> 1, g = threadIdx.x & 1;  // row, 4-block group
            const int64_t tile = mat * row_tiles + half / 2;
            const int rt = static_cast<int>((half & 1) * 64) + r;  // row of the scale tile
            *reinterpret_cast<uint32_t *>(scales + ((tile * chunks + chunk) * 2 + g) * 512 + (rt % 32) * 16 + (rt / 32) * 4) =
                *reinterpret_cast<const uint32_t *>(&ss[r][g * 4]);
        }
        __syncthreads();
    }
}

// 8 codes -> 8 values (exact), times the block's scale.
__device__ __forceinline__ void decode8(uint32_t u, float scale, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("{\n"
            "  .reg .b8 a, b, c, d;\n"
            "  mov.b32 {a, b, c, d}, %1;\n"
            "  cvt.rn.f16x2.e2m1x2 %0, a;\n"
            "}\n"
            : "=r"(h)
            : "r"(u >> (8 * i)));
        float lo, hi;
        asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
            : "=f"(lo), "=f"(hi)
            : "r"(h));
        v[2 * i] = lo * scale;
        v[2 * i + 1] = hi * scale;
    }
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7FC00000u);
    return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// One thread per 8 values: 4 bytes of codes and their block's scale byte.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows, int64_t cols,
                  int64_t row_tiles, int64_t chunks, int64_t items, int64_t per_row, T *__restrict__ y) {
    griddep_enter();
    const int64_t ld = fp4_row_bytes(cols);
    for (int64_t it = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; it < items;
         it += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t row = it / per_row, c = (it - row * per_row) * 8;
        const int64_t mat = row / rows, r = row - mat * rows;
        const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(codes + row * ld + c / 2));
        const int64_t tile = (mat * row_tiles + r / 128) * chunks * 2 + c / 128;
        const uint32_t sb = __ldg(scales + tile * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + (c / 32) % 4);
        float v[8];
        decode8(u, scale_value(sb), v);
        T *out = y + row * cols + c;
        if (VEC && sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(out) =
                make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        } else if (VEC) {
            *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
            if (c + 4 < cols) *(reinterpret_cast<float4 *>(out) + 1) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < cols) {
                    if (sizeof(T) == 2) reinterpret_cast<uint16_t *>(out)[i] = static_cast<uint16_t>(pack2(v[i], 0.0f) & 0xFFFFu);
                    else reinterpret_cast<float *>(out)[i] = v[i];
                }
        }
    }
}

unsigned grid_for(int64_t blocks, int per_sm) {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    const int64_t cap = static_cast<int64_t>(n > 0 ? n : 1) * per_sm;
    return static_cast<unsigned>(blocks < 1 ? 1 : (blocks < cap ? blocks : cap));
}

template <class T, bool RELU2>
int quantize_typed(const void *x, const int *row_map, int map_div, int64_t rows, int64_t cols, int batch,
                   bool transposed, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int64_t row_tiles = (rows + 127) / 128, chunks = (cols + 255) / 256;
    const T *xt = static_cast<const T *>(x);
    if (transposed) {
        const int64_t items = row_tiles * 2 * chunks * batch;
        auto kern = rows % 2 == 0 ? quantize_cols_kernel<T, true, RELU2> : quantize_cols_kernel<T, false, RELU2>;
        return launch_pdl(kern, dim3(grid_for(items, 16)), dim3(kThreads), 0, s, xt, row_map, map_div, rows, cols,
                          row_tiles, chunks, items, codes, scales);
    }
    const int64_t items = row_tiles * 32 * chunks * batch;
    auto kern = cols * sizeof(T) % 16 == 0 ? quantize_rows_kernel<T, true, RELU2> : quantize_rows_kernel<T, false, RELU2>;
    return launch_pdl(kern, dim3(grid_for((items + kWarps - 1) / kWarps, 16)), dim3(kThreads), 0, s, xt, row_map,
                      map_div, rows, cols, row_tiles, chunks, items, codes, scales);
}

template <class T>
int dequantize_typed(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, int batch, void *y,
                     cudaStream_t s) {
    const int64_t row_tiles = (rows + 127) / 128, chunks = (cols + 255) / 256;
    const int64_t per_row = (cols + 7) / 8, items = per_row * rows * batch;
    auto kern = cols * sizeof(T) % 16 == 0 ? dequantize_kernel<T, true> : dequantize_kernel<T, false>;
    return launch_pdl(kern, dim3(grid_for((items + kThreads - 1) / kThreads, 16)), dim3(kThreads), 0, s, codes, scales,
                      rows, cols, row_tiles, chunks, items, per_row, static_cast<T *>(y));
}

}  // namespace

int launch_fp4_quantize(int dtype, const void *x, const int *row_map, int map_div, int64_t rows, int64_t cols,
                        int batch, bool transposed, bool relu2, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    if (dtype == MLPBLK_BF16) {
        if (relu2) return quantize_typed<uint16_t, true>(x, row_map, map_div, rows, cols, batch, transposed, codes, scales, s);
        return quantize_typed<uint16_t, false>(x, row_map, map_div, rows, cols, batch, transposed, codes, scales, s);
    }
    if (relu2) return quantize_typed<float, true>(x, row_map, map_div, rows, cols, batch, transposed, codes, scales, s);
    return quantize_typed<float, false>(x, row_map, map_div, rows, cols, batch, transposed, codes, scales, s);
}

int launch_fp4_dequantize(int dtype, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                          int batch, void *y, cudaStream_t s) {
    if (dtype == MLPBLK_BF16) return dequantize_typed<uint16_t>(codes, scales, rows, cols, batch, y, s);
    return dequantize_typed<float>(codes, scales, rows, cols, batch, y, s);
}

}  // namespace mlpblk
