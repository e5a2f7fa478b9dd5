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
#include <type_traits>

#include "fp4_layout.h"

namespace mlpblk {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// 8 floats -> 8 E2M1 codes (first value in the lowest four bits), nearest-even,
// saturating; RELU: negative values become 0.
template <bool RELU>
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
#define MLPBLK_E2M1(RELU_)                                                   \
    asm("{\n"                                                                \
        "  .reg .b8 a, b, c, d;\n"                                           \
        "  cvt.rn.satfinite" RELU_ ".e2m1x2.f32 a, %2, %1;\n"                \
        "  cvt.rn.satfinite" RELU_ ".e2m1x2.f32 b, %4, %3;\n"                \
        "  cvt.rn.satfinite" RELU_ ".e2m1x2.f32 c, %6, %5;\n"                \
        "  cvt.rn.satfinite" RELU_ ".e2m1x2.f32 d, %8, %7;\n"                \
        "  mov.b32 %0, {a, b, c, d};\n"                                      \
        "}\n"                                                                \
        : "=r"(r)                                                            \
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]))
    if (RELU) MLPBLK_E2M1(".relu");
    else MLPBLK_E2M1("");
#undef MLPBLK_E2M1
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

// ReLU^2 needs no clamp of its own: the block's maximum is the square of the largest
// v (0 at least), and v |v| has v^2's size and a sign that the conversion's .relu
// reads.  max(m, v), a NaN once there is one:
__device__ __forceinline__ float max_signed(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(v));
    return r;
}
__device__ __forceinline__ uint32_t max_signed_bf16x2(uint32_t m, uint32_t v) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(v));
    return r;
}

// max(|m|, |v|), a NaN once there is one (the bf16 form's signs are of no meaning: one
// instruction fewer than clearing them first, in kernels bound by the integer pipe).
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t v) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(v));
    return r;
}

// Both bf16 values of v times those of m.  Exact for powers of two in m, but for
// results below bf16's normal range, whose code is 0 either way.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t v, uint32_t m) {
    uint32_t r;
    asm("mul.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(m));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// The source row of Q's row (or, transposed, column) r under a row map, or -1 for zeros.
// A gathered row behind the source's own (a map of another batch) is taken as none, so no
// access leaves x.
__device__ __forceinline__ int source_row(const int *row_map, int map_div, int source_rows, int64_t r) {
    const int m = row_map[r];
    if (m < 0) return -1;
    if (map_div == 0) return static_cast<int>(r);
    const int q = m / map_div;
    return q < source_rows ? q : -1;
}

// The bits of a block's largest |value| (or largest value, squared) from its maxima:
// `m` packed bf16, or a float.
template <bool RELU2>
__device__ __forceinline__ uint32_t top_bits(uint32_t m) {
    if (!RELU2) {
        m &= 0x7FFF7FFFu;
        return max(m << 16, m & 0xFFFF0000u);
    }
    const float t = max_signed(bf16_lo(m), bf16_hi(m));
    return __float_as_uint(t * t);
}
template <bool RELU2>
__device__ __forceinline__ uint32_t top_bits(float m) {
    return __float_as_uint(RELU2 ? m * m : m);
}

// 8 consecutive values of a row, as loaded: 4 words of bf16 pairs or 8 floats.
template <bool BF16>
struct Oct;
template <>
struct Oct<true> {
    uint32_t w[4];
    // columns c .. c + 7, 16-byte aligned, all of them below cols or none
    __device__ __forceinline__ void load(const uint16_t *row, int64_t c, int64_t cols) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (c < cols) u = __ldg(reinterpret_cast<const uint4 *>(row + c));
        w[0] = u.x;
        w[1] = u.y;
        w[2] = u.z;
        w[3] = u.w;
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    // what is rounded: the values times inv, a power of two (in bf16, two at a time), or
    // their signed squares times inv
    template <bool RELU2>
    __device__ __forceinline__ void scaled(float inv, float (&v)[8]) const {
        if (RELU2) {
            floats(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * fabsf(v[i]) * inv;
            return;
        }
        const uint32_t m = __float_as_uint(inv) >> 16, m2 = m | (m << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = mul_bf16x2(w[i], m2);
            v[2 * i] = bf16_lo(u);
            v[2 * i + 1] = bf16_hi(u);
        }
    }
    using Max = uint32_t;
    static constexpr Max kNone = 0u;
    template <bool RELU2>
    __device__ __forceinline__ void top(Max &m) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = RELU2 ? max_signed_bf16x2(m, w[i]) : max_abs_bf16x2(m, w[i]);
    }
};
template <>
struct Oct<false> {
    float f[8];
    __device__ __forceinline__ void load(const float *row, int64_t c, int64_t cols) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c + 4 * h < cols) u = __ldg(reinterpret_cast<const float4 *>(row + c + 4 * h));
            f[4 * h] = u.x;
            f[4 * h + 1] = u.y;
            f[4 * h + 2] = u.z;
            f[4 * h + 3] = u.w;
        }
    }
    __device__ __forceinline__ void load_shared(const float *p) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 u = *reinterpret_cast<const float4 *>(p + 4 * h);
            f[4 * h] = u.x;
            f[4 * h + 1] = u.y;
            f[4 * h + 2] = u.z;
            f[4 * h + 3] = u.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i];
    }
    template <bool RELU2>
    __device__ __forceinline__ void scaled(float inv, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (RELU2 ? f[i] * fabsf(f[i]) : f[i]) * inv;
    }
    using Max = float;
    static constexpr Max kNone = 0.0f;
    template <bool RELU2>
    __device__ __forceinline__ void top(Max &m) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = RELU2 ? max_signed(m, f[i]) : max_abs(m, f[i]);
    }
};

// Four rows of zeros (`out`, each 32 rows behind the one before; those below `left`) and their
// 16 bytes of every scale tile: padding between sorted segments, which is whole tiles of
// a warp's rows where the experts' rows are few.
__device__ __forceinline__ void zero_rows(uint8_t *out, int64_t ld, int64_t left, uint8_t *tile_scales, int col_tiles) {
    const int lane = threadIdx.x & 31;
    for (int64_t u = static_cast<int64_t>(blockIdx.y) * 32 + lane; u < ld / 16; u += static_cast<int64_t>(gridDim.y) * 32)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (32 * j < left) *reinterpret_cast<uint4 *>(out + 32 * j * ld + u * 16) = make_uint4(0u, 0u, 0u, 0u);
    for (int g = blockIdx.y * 32 + lane; g < col_tiles; g += gridDim.y * 32)
        *reinterpret_cast<uint4 *>(tile_scales + static_cast<int64_t>(g) * 512) = make_uint4(0u, 0u, 0u, 0u);
}

// Blocks along the source's rows, float32.  A CTA takes 8 values of r % 32 of one 128-row scale
// tile, a warp the rows r, r + 32, r + 64, r + 96, 256 columns at a time: a lane holds
// 8 consecutive values of each row, a block is four lanes, and the four rows'
// scales of 4 blocks are 16 consecutive bytes of a tile (one store), with the next
// row's beside them.  The four rows' loads are in flight together.
template <bool VEC, bool RELU2, bool MAP>
__global__ void __launch_bounds__(kThreads, 3)
quantize_rows_kernel(const float *__restrict__ x, const int *__restrict__ row_map, int map_div, int source_rows, int64_t rows,
                     int64_t cols, int row_tiles, int chunks, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales) {
    __shared__ __align__(16) float turn[VEC ? 1 : kWarps][4][VEC ? 8 : 256];
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const int64_t ld = fp4_row_bytes(cols);
    const int tile = static_cast<int>(blockIdx.x >> 2);  // of the whole batch
    const int mat = tile / row_tiles;
    const int rr = static_cast<int>(blockIdx.x & 3) * 8 + (threadIdx.x >> 5);
    const int64_t r0 = static_cast<int64_t>(tile - mat * row_tiles) * 128 + rr;
    const float *src[4];
    bool live[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + 32 * j;
        int64_t at = r < rows ? r : -1;
        if (MAP && r < rows) at = source_row(row_map, map_div, source_rows, r);
        live[j] = at >= 0;
        src[j] = x + (mat * rows + (at < 0 ? 0 : at)) * cols;
    }
    uint8_t *out = codes + (mat * rows + r0) * ld;
    if (MAP && !(live[0] || live[1] || live[2] || live[3])) {
        zero_rows(out, ld, rows - r0, scales + static_cast<int64_t>(tile) * chunks * 1024 + rr * 16, chunks * 2);
        return;
    }
    for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
        const int64_t c = static_cast<int64_t>(chunk) * 256 + lane * 8;
        Oct<false> o[4];
        if (VEC) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (live[j]) o[j].load(src[j], c, cols);
                else o[j].zero();
            }
        } else {
            float *mine = &turn[VEC ? 0 : threadIdx.x >> 5][0][0];
            const int64_t c0 = static_cast<int64_t>(chunk) * 256 + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) mine[j * 256 + 32 * i + lane] = live[j] && c0 + 32 * i < cols ? __ldg(src[j] + c0 + 32 * i) : 0.0f;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j].load_shared(mine + j * 256 + lane * 8);
            __syncwarp();
        }
        uint32_t word[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool out_row = r0 + 32 * j < rows;
            if (!live[j]) {  // a row of zeros, or none
                if (out_row && c < 2 * ld) *reinterpret_cast<uint32_t *>(out + 32 * j * ld + c / 2) = 0u;
                word[j] = 0u;
                continue;
            }
            float v[8];
            Oct<false>::Max top = Oct<false>::kNone;
            o[j].top<RELU2>(top);
            uint32_t m = top_bits<RELU2>(top);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t sb = scale_byte(m);
            o[j].scaled<RELU2>(scale_inverse(sb), v);
            const uint32_t q = sb == 255u ? 0u : e2m1x8<RELU2>(v);
            if (c < 2 * ld) *reinterpret_cast<uint32_t *>(out + 32 * j * ld + c / 2) = q;
            // the four blocks' bytes of this half warp
            uint32_t w = sb << (8 * ((lane >> 2) & 3));
            w |= __shfl_xor_sync(0xffffffffu, w, 4);
            w |= __shfl_xor_sync(0xffffffffu, w, 8);
            word[j] = w;
        }
        if ((lane & 15) == 0) {
            uint8_t *st = scales + ((static_cast<int64_t>(tile) * chunks + chunk) * 2 + (lane >> 4)) * 512 + rr * 16;
            *reinterpret_cast<uint4 *>(st) = make_uint4(word[0], word[1], word[2], word[3]);
        }
    }
}

// 32 bf16 values at p, of which `left` lie before the row's end (0 behind it).  Rows that do
// not begin on 16-byte boundaries are read in aligned 16-byte accesses all the same and
// shifted into place by two words, one word, half a word; the access that the row's end cuts
// is read by elements, so nothing behind the row is read.
__device__ __forceinline__ void load_block(const uint16_t *__restrict__ p, int left, Oct<true> (&o)[4]) {
    const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / 2;
    const uint16_t *a = p - phase;
    left += phase;
    uint32_t w[20];
#pragma unroll
    for (int u = 0; u < 5; ++u) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (8 * u + 8 <= left && (u < 4 || phase != 0)) v = __ldg(reinterpret_cast<const uint4 *>(a + 8 * u));
        w[4 * u] = v.x;
        w[4 * u + 1] = v.y;
        w[4 * u + 2] = v.z;
        w[4 * u + 3] = v.w;
    }
    if (left < 40) {
        uint32_t t[4] = {0u, 0u, 0u, 0u};
        const int n = left > 0 ? left & 7 : 0, at = left >> 3;
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) t[i >> 1] |= static_cast<uint32_t>(__ldg(a + 8 * at + i)) << (16 * (i & 1));
#pragma unroll
        for (int u = 0; u < 5; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (u == at && n > 0) w[4 * u + i] = t[i];
    }
    if (phase & 4) {
#pragma unroll
        for (int i = 0; i < 18; ++i) w[i] = w[i + 2];
    }
    if (phase & 2) {
#pragma unroll
        for (int i = 0; i < 17; ++i) w[i] = w[i + 1];
    }
    const int sh = (phase & 1) * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i >> 2].w[i & 3] = __funnelshift_r(w[i], w[i + 1], sh);
}

// Blocks along the source's rows, bf16 rows in 16-byte accesses: a lane holds a whole
// block (its 16-byte loads 64 bytes from its neighbour's; the sectors' other halves
// come from L1), so a block's maximum needs no shuffle and its codes are one 16-byte
// store.  A warp takes one column tile (128 columns) of the rows r, r + 32, r + 64, r + 96
// of a scale tile for eight neighbouring r, two rows in flight (HALVES 2: two of the four
// rows alone); four lanes then transpose their 4 x 4 scale bytes, and the warp stores 128
// consecutive bytes of the tile.  Warps are numbered along a row's tiles first, so a
// CTA's cover neighbouring parts of a row and no lane idles but in a row's last 256
// columns.  8192 x 16384: 49.5 us (6.86 TB/s), with ReLU^2 too, where a lane with 8 values
// and shuffles takes 67; 192 MB in rows of 1056: 40 and 63, of 1031: 55 and 88.  (float32 gains nothing: four rows'
// loads of 8 values take 38 us for 192 MB, blocks of 128 bytes a lane 51.)
constexpr int kBlockWarps = 4;  // of a CTA (16384 x 16384: 98 us with eight, ReLU^2 100)

template <bool RELU2, bool MAP, bool ALIGNED, int HALVES>
__global__ void __launch_bounds__(32 * kBlockWarps, RELU2 ? 4 : 6)
quantize_blocks_kernel(const uint16_t *__restrict__ x, const int *__restrict__ row_map, int map_div, int source_rows, int64_t rows,
                       int64_t cols, int row_tiles, int col_tiles, uint32_t warps, uint8_t *__restrict__ codes,
                       uint8_t *__restrict__ scales) {
    constexpr int kParts = 4;  // Octs of a block
    constexpr int kRows = 2;   // rows in flight
    griddep_enter();
    const int lane = threadIdx.x & 31;
    uint32_t w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (w >= warps) return;
    const int own = HALVES == 2 ? static_cast<int>(w & 1u) : -1;  // the half of the four rows, -1: both
    w /= HALVES;
    const uint32_t eight = w / col_tiles;  // rows r .. r + 7, of the whole batch
    const int col_tile = static_cast<int>(w - eight * col_tiles);
    const int tile = static_cast<int>(eight >> 2);
    const int mat = tile / row_tiles;
    const int rr = static_cast<int>(eight & 3) * 8 + (lane >> 2);
    const int64_t ld = fp4_row_bytes(cols);
    const int64_t r0 = static_cast<int64_t>(tile - mat * row_tiles) * 128 + rr;
    const int64_t c = static_cast<int64_t>(col_tile) * 128 + (lane & 3) * 32;
    const uint16_t *base = x + mat * rows * cols;
    uint8_t *out = codes + (mat * rows + r0) * ld + c / 2;
    int64_t src[4];  // source rows, -1: zeros
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + 32 * j;
        src[j] = r < rows ? r : -1;
        if (MAP && r < rows) src[j] = source_row(row_map, map_div, source_rows, r);
    }
    uint32_t bytes = 0;  // of the four rows
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += kRows) {
        if (own >= 0 && own != j0 / kRows) continue;
        Oct<true> o[kRows][kParts];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if constexpr (ALIGNED) {
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    if (src[j0 + u] >= 0) o[u][q].load(base + src[j0 + u] * cols, c + 8 * q, cols);
                    else o[u][q].zero();
                }
            } else if (src[j0 + u] >= 0) {
                load_block(base + src[j0 + u] * cols + c, static_cast<int>(min(cols - c, static_cast<int64_t>(64))), o[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int j = j0 + u;
            const bool row = r0 + 32 * j < rows && c < 2 * ld;
            if (src[j] < 0) {  // a row of zeros, or none
                if (row) *reinterpret_cast<uint4 *>(out + 32 * j * ld) = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            Oct<true>::Max top = Oct<true>::kNone;
#pragma unroll
            for (int q = 0; q < kParts; ++q) o[u][q].template top<RELU2>(top);
            const uint32_t sb = scale_byte(top_bits<RELU2>(top));
            const float inv = scale_inverse(sb);
            uint32_t v4[kParts];
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                float v[8];
                o[u][q].template scaled<RELU2>(inv, v);
                v4[q] = sb == 255u ? 0u : e2m1x8<RELU2>(v);
            }
            if (row) *reinterpret_cast<uint4 *>(out + 32 * j * ld) = make_uint4(v4[0], v4[1], v4[2], v4[3]);
            bytes |= sb << (8 * j);
        }
    }
    // byte j of lane b -> byte b of lane j, within four lanes
    uint32_t t = __shfl_xor_sync(0xffffffffu, bytes, 1);
    bytes = (lane & 1) ? __byte_perm(bytes, t, 0x3715) : __byte_perm(bytes, t, 0x6240);
    t = __shfl_xor_sync(0xffffffffu, bytes, 2);
    bytes = (lane & 2) ? __byte_perm(bytes, t, 0x3276) : __byte_perm(bytes, t, 0x5410);
    if (own < 0 || own == (lane & 3) / kRows)
        *reinterpret_cast<uint32_t *>(scales + (static_cast<int64_t>(tile) * col_tiles + col_tile) * 512 + rr * 16 +
                                      (lane & 3) * 4) = bytes;
}

// Two neighbouring values of a source row, columns c and c + 1 (0 at and behind
// `width`), as loaded.  VEC: width is even, so a pair is one aligned access.
template <bool BF16>
struct Pair;
template <>
struct Pair<true> {
    uint32_t w;
    template <bool VEC>
    __device__ __forceinline__ void load(const uint16_t *row, int64_t c, int64_t width) {
        if (VEC) {
            w = c < width ? __ldg(reinterpret_cast<const uint32_t *>(row + c)) : 0u;
        } else {
            const uint32_t lo = c < width ? __ldg(row + c) : 0u, hi = c + 1 < width ? __ldg(row + c + 1) : 0u;
            w = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ void zero() { w = 0u; }
    __device__ __forceinline__ float lo() const { return bf16_lo(w); }
    __device__ __forceinline__ float hi() const { return bf16_hi(w); }
};
template <>
struct Pair<false> {
    float2 f;
    template <bool VEC>
    __device__ __forceinline__ void load(const float *row, int64_t c, int64_t width) {
        f = make_float2(0.0f, 0.0f);
        if (VEC) {
            if (c < width) f = __ldg(reinterpret_cast<const float2 *>(row + c));
        } else {
            if (c < width) f.x = __ldg(row + c);
            if (c + 1 < width) f.y = __ldg(row + c + 1);
        }
    }
    __device__ __forceinline__ void zero() { f = make_float2(0.0f, 0.0f); }
    __device__ __forceinline__ float lo() const { return f.x; }
    __device__ __forceinline__ float hi() const { return f.y; }
};

// The two columns' blocks of 32 values: their codes and scale bytes.
template <bool BF16, bool RELU2>
__device__ __forceinline__ void quantize_pairs(const Pair<BF16> (&p)[32], uint4 &qa, uint4 &qb, uint32_t &sa, uint32_t &sb) {
    uint32_t ta, tb;  // bits of the columns' largest |v|, or squared
    if constexpr (BF16) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = RELU2 ? max_signed_bf16x2(m, p[i].w) : max_abs_bf16x2(m, p[i].w);
        ta = top_bits<RELU2>(bf16_lo(RELU2 ? m : m & 0x7FFF7FFFu));
        tb = top_bits<RELU2>(bf16_hi(RELU2 ? m : m & 0x7FFF7FFFu));
    } else {
        float ma = 0.0f, mb = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            ma = RELU2 ? max_signed(ma, p[i].lo()) : max_abs(ma, p[i].lo());
            mb = RELU2 ? max_signed(mb, p[i].hi()) : max_abs(mb, p[i].hi());
        }
        ta = top_bits<RELU2>(ma);
        tb = top_bits<RELU2>(mb);
    }
    sa = scale_byte(ta);
    sb = scale_byte(tb);
    const float ia = scale_inverse(sa), ib = scale_inverse(sb);
    uint32_t wa[4], wb[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float va[8], vb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (BF16 && !RELU2) {
                const uint32_t u = mul_bf16x2(p[8 * g + i].w, (__float_as_uint(ia) >> 16) | (__float_as_uint(ib) & 0xFFFF0000u));
                va[i] = bf16_lo(u);
                vb[i] = bf16_hi(u);
            } else {
                const float a = p[8 * g + i].lo(), b = p[8 * g + i].hi();
                va[i] = (RELU2 ? a * fabsf(a) : a) * ia;
                vb[i] = (RELU2 ? b * fabsf(b) : b) * ib;
            }
        }
        wa[g] = sa == 255u ? 0u : e2m1x8<RELU2>(va);
        wb[g] = sb == 255u ? 0u : e2m1x8<RELU2>(vb);
    }
    qa = make_uint4(wa[0], wa[1], wa[2], wa[3]);
    qb = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

// Blocks along the source's columns: Q = x^T, Q's rows are x's columns.  A CTA
// takes 64 columns and 256 rows of x; warp w holds rows 32w .. 32w + 31 of it, two
// columns a lane, so a block is one lane's 32 values, kept as they were loaded (pairs of
// bf16 in one register).  The codes cross shared memory to leave as 128 consecutive
// bytes a row of Q.
constexpr int kTCols = 64;              // x's columns of a CTA (Q's rows)
constexpr int kTPitch = 128 + 16;       // bytes of a Q row in shared memory

// MAP: 0 no row map, 1 a map that only says which rows are live, 2 one that gathers.
template <bool BF16, bool VEC, bool RELU2, int MAP>
__global__ void __launch_bounds__(kThreads, BF16 ? 3 : 2)
quantize_cols_kernel(const void *__restrict__ x, const int *__restrict__ row_map, int map_div, int source_rows, int64_t rows,
                     int64_t cols, int row_tiles, int chunks, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales) {
    using T = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ __align__(16) uint8_t sc[kTCols][kTPitch];
    __shared__ __align__(8) uint8_t ss[kTCols][8];
    griddep_enter();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t ld = fp4_row_bytes(cols);
    const int halves = row_tiles * 2;  // 64-row parts of the scale tiles of one matrix
    const int mat = static_cast<int>(blockIdx.x) / halves;
    const int half = static_cast<int>(blockIdx.x) - mat * halves;
    const int64_t r0 = static_cast<int64_t>(half) * kTCols;  // Q's first row
    const int64_t col = r0 + 2 * lane;                       // x's column
    const T *base = static_cast<const T *>(x) + mat * rows * cols;
    auto live_at = [&](int64_t chunk) {  // this thread's row of x of a chunk
        const int64_t own = chunk * 256 + threadIdx.x;
        return own < cols && row_map[own] >= 0;
    };
    bool live_here = MAP != 0 && live_at(blockIdx.y);
    for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
        const int64_t c0 = static_cast<int64_t>(chunk) * 256 + wid * 32;  // Q's first column of this warp: x's row
        if (MAP != 0) {
            // padding alone (an expert's segment is mostly that where its rows are few):
            // zeros without the way through shared memory.  The barrier is also the one
            // between the chunk before and the writes below.
            const bool any = __syncthreads_or(live_here);
            live_here = live_at(chunk + static_cast<int64_t>(gridDim.y));
            if (!any) {
#pragma unroll
                for (int h = 0; h < kTCols * 8 / kThreads; ++h) {
                    const int q = threadIdx.x + h * kThreads;
                    const int64_t at = static_cast<int64_t>(chunk) * 128 + (q & 7) * 16;
                    if (r0 + (q >> 3) < rows && at < ld)
                        *reinterpret_cast<uint4 *>(codes + (mat * rows + r0 + (q >> 3)) * ld + at) = make_uint4(0u, 0u, 0u, 0u);
                }
                if (threadIdx.x < kTCols * 2) {
                    const int rt = (half & 1) * 64 + (threadIdx.x >> 1);
                    const int64_t tile = static_cast<int64_t>(mat) * row_tiles + half / 2;
                    *reinterpret_cast<uint32_t *>(scales + ((tile * chunks + chunk) * 2 + (threadIdx.x & 1)) * 512 + (rt % 32) * 16 +
                                                  (rt / 32) * 4) = 0u;
                }
                continue;
            }
        }
        Pair<BF16> p[32];
        bool none = false;  // no row of x is live: zeros without the arithmetic
        if (MAP == 2) {
            const int64_t own = c0 + lane;
            const int mine = own < cols ? source_row(row_map, map_div, source_rows, own) : -1;
            none = !__any_sync(0xffffffffu, mine >= 0);
            if (!none) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int src = __shfl_sync(0xffffffffu, mine, i);
                    p[i].template load<VEC>(base + (src < 0 ? 0 : src) * rows, src < 0 ? rows : col, rows);
                }
            }
        } else if (MAP == 1) {
            const int64_t own = c0 + lane;
            const unsigned live = __ballot_sync(0xffffffffu, own < cols && row_map[own < cols ? own : 0] >= 0);
            const T *row = base + c0 * rows;
            none = live == 0u;
            if (live == 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < 32; ++i, row += rows) p[i].template load<VEC>(row, col, rows);
            } else if (!none) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const bool in = live >> i & 1u;
                    p[i].template load<VEC>(in ? row + i * rows : base, in ? col : rows, rows);
                }
            }
        } else if (c0 + 32 <= cols) {
            const T *row = base + c0 * rows;
#pragma unroll
            for (int i = 0; i < 32; ++i, row += rows) p[i].template load<VEC>(row, col, rows);
        } else {
            const T *row = base + c0 * rows;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const bool in = c0 + i < cols;
                p[i].template load<VEC>(in ? row + i * rows : base, in ? col : rows, rows);
            }
        }
        uint32_t sa = 0, sb = 0;
        uint4 qa = make_uint4(0u, 0u, 0u, 0u), qb = qa;
        if (MAP == 0 || !none) quantize_pairs<BF16, RELU2>(p, qa, qb, sa, sb);
        *reinterpret_cast<uint4 *>(&sc[2 * lane][wid * 16]) = qa;
        *reinterpret_cast<uint4 *>(&sc[2 * lane + 1][wid * 16]) = qb;
        ss[2 * lane][wid] = static_cast<uint8_t>(sa);
        ss[2 * lane + 1][wid] = static_cast<uint8_t>(sb);
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kTCols * 8 / kThreads; ++h) {
            const int q = threadIdx.x + h * kThreads;
            const int r = q >> 3, blk = q & 7;
            const int64_t at = static_cast<int64_t>(chunk) * 128 + blk * 16;
            if (r0 + r < rows && at < ld)
                *reinterpret_cast<uint4 *>(codes + (mat * rows + r0 + r) * ld + at) =
                    *reinterpret_cast<const uint4 *>(&sc[r][blk * 16]);
        }
        if (threadIdx.x < kTCols * 2) {
            const int r = threadIdx.x >> 1, g = threadIdx.x & 1;  // row, 4-block group
            const int64_t tile = static_cast<int64_t>(mat) * row_tiles + half / 2;
            const int rt = (half & 1) * 64 + r;  // row of the scale tile
            *reinterpret_cast<uint32_t *>(scales + ((tile * chunks + chunk) * 2 + g) * 512 + (rt % 32) * 16 + (rt / 32) * 4) =
                *reinterpret_cast<const uint32_t *>(&ss[r][g * 4]);
        }
        if (MAP == 0) __syncthreads();
    }
}

// 8 codes -> their values in bf16 (exact), the first in the lowest half.  A code's three low
// bits select the two bytes of its size from tables (four codes a byte permutation); the
// fourth, that permutation's sign mode, makes a byte of ones of a set sign byte.
__device__ __forceinline__ void decode8(uint32_t u, uint32_t (&v)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = h == 0 ? u : u >> 16, size = c & 0x7777u;
        const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, size);  // 0 .5 1 1.5 | 2 3 4 6
        uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, size);
        uint32_t sign;  // 0x80 or, of a negative code, 0xFF
        asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(c));
        hi |= (sign << 7) & 0x80808080u;
        v[2 * h] = __byte_perm(lo, hi, 0x5140);
        v[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
    }
}

// A scale in bf16, in both halves.
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
    const uint32_t m = byte == 255u ? 0x7FC0u : (byte == 0u ? 0x0040u : byte << 7);
    return m | (m << 16);
}

// A warp takes CHUNKS pieces of 256 values, numbered along the rows, with the pieces'
// loads in flight together: a lane 8 values of each, 4 bytes of codes and their
// block's scale byte.  bf16 rows of whole 16-byte accesses are stored from registers.
// float32 values, and rows of any length, cross shared memory, so that neighbouring
// lanes store neighbouring words (two float4 stores 32 bytes apart take 51 us where this
// takes 36, 192 MB of values; bf16 rows of 4097: 66, instruction issue).
template <bool BF16, bool ALIGNED, int WARPS, int CHUNKS>
__global__ void __launch_bounds__(32 * WARPS)
dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows, int64_t cols,
                  int row_tiles, int pieces, uint32_t all_pieces, void *__restrict__ y) {
    using T = typename std::conditional<BF16, uint16_t, float>::type;
    constexpr bool kTurn = !(BF16 && ALIGNED);
    __shared__ __align__(16) T turn[kTurn ? WARPS : 1][kTurn ? 256 : 8];
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const uint32_t p0 = (blockIdx.x * static_cast<uint32_t>(WARPS) + (threadIdx.x >> 5)) * CHUNKS;
    if (p0 >= all_pieces) return;
    const int64_t ld = fp4_row_bytes(cols);
    const int64_t tile_row = fp4_col_tiles(cols) * kFp4TileBytes;  // bytes of a row of scale tiles
    uint32_t row = p0 / pieces;
    uint32_t piece = p0 - row * pieces;
    uint32_t mat = row / static_cast<uint32_t>(rows), r = row - mat * static_cast<uint32_t>(rows);
    const uint8_t *in, *sc;  // of the row, this lane's
    T *out;                  // the row's
    auto start_row = [&]() {
        in = codes + row * ld + lane * 4;
        sc = scales + (static_cast<int64_t>(mat) * row_tiles + (r >> 7)) * tile_row + (lane >> 4) * kFp4TileBytes +
             (r & 31) * 16 + (r >> 5 & 3) * 4 + ((lane >> 2) & 3);
        out = static_cast<T *>(y) + row * cols;
    };
    start_row();
    T *to[CHUNKS];      // the piece's first value
    int count[CHUNKS];  // of its values
    uint32_t u[CHUNKS], sb[CHUNKS];
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        to[j] = out + static_cast<int64_t>(piece) * 256;
        count[j] = p0 + j < all_pieces ? static_cast<int>(min(cols - static_cast<int64_t>(piece) * 256, static_cast<int64_t>(256))) : 0;
        u[j] = sb[j] = 0u;
        if (lane * 8 < count[j]) {
            u[j] = __ldg(reinterpret_cast<const uint32_t *>(in + static_cast<int64_t>(piece) * 128));
            sb[j] = __ldg(sc + static_cast<int64_t>(piece) * (2 * kFp4TileBytes));
        }
        if (++piece == static_cast<uint32_t>(pieces)) {
            piece = 0;
            ++row;
            if (++r == static_cast<uint32_t>(rows)) {
                r = 0;
                ++mat;
            }
            start_row();
        }
    }
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        const int n = count[j];
        if (n == 0) break;
        // the products are exact: a power of two times at most two bits, down to 2^-128
        uint32_t v[4];
        decode8(u[j], v);
        const uint32_t scale = scale_pair(sb[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(v[i], scale);
        if (!kTurn) {
            if (lane * 8 < n) *reinterpret_cast<uint4 *>(to[j] + lane * 8) = make_uint4(v[0], v[1], v[2], v[3]);
            continue;
        }
        T *mine = turn[kTurn ? threadIdx.x >> 5 : 0];
        if constexpr (BF16) {
            *reinterpret_cast<uint4 *>(mine + lane * 8) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
            *reinterpret_cast<float4 *>(mine + lane * 8) = make_float4(bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1]));
            *reinterpret_cast<float4 *>(mine + lane * 8 + 4) = make_float4(bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3]));
        }
        __syncwarp();
        if constexpr (BF16) {
            // pairs from the first 4-byte boundary on
            const uint32_t *words = reinterpret_cast<const uint32_t *>(mine);
            const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(to[j]) >> 1 & 1);
            if (odd && lane == 0) to[j][0] = mine[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 32 * i + lane, c = 2 * k + odd;
                uint32_t w = words[k];
                if (odd) w = __funnelshift_r(w, words[k < 127 ? k + 1 : k], 16);
                if (c + 1 < n) *reinterpret_cast<uint32_t *>(to[j] + c) = w;
                else if (c < n) to[j][c] = static_cast<uint16_t>(w & 0xFFFFu);
            }
        } else if (ALIGNED) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (128 * i + lane * 4 < n)
                    *reinterpret_cast<float4 *>(to[j] + 128 * i + lane * 4) = *reinterpret_cast<const float4 *>(mine + 128 * i + lane * 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (32 * i + lane < n) to[j][32 * i + lane] = mine[32 * i + lane];
        }
        __syncwarp();
    }
}

int sm_total() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 1;
}

// CTAs along the second axis (up to `most` pieces of work) beside x CTAs along the
// first: about 32 CTAs an SM in all.
dim3 grid_for(int64_t x, int64_t most) {
    int64_t y = (static_cast<int64_t>(sm_total()) * 32 + x - 1) / x;
    if (y > most) y = most;
    if (y > 65535) y = 65535;
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < 1 ? 1 : y));
}

// Where there are at most this many warps an SM, quantize_blocks_kernel deals a warp's four
// rows out to two (bf16 from L2, 2048 x 2048: 5.8 us with one warp and 3.5 with two, 4096 x
// 4096: 6.8 and 6.2; 8192 x 16384 from HBM, ReLU^2: 53 and 57, in CTAs of eight warps).
constexpr int64_t kHalfWarps = 32;

// Warps of a CTA for quantize_blocks_kernel, whose warps are independent: kBlockWarps, fewer
// where that spreads few warps over the SMs (118 x 6624: 2.7 us, with CTAs of eight 3.5).
int warps_per_cta(int64_t warps) {
    const int sms = sm_total();
    int w = 1;
    while (w < kBlockWarps && warps > static_cast<int64_t>(sms) * w) w *= 2;
    return w;
}

template <bool BF16, bool RELU2, int MAP>
int quantize_typed(const void *x, const int *row_map, int map_div, int source_rows, int64_t rows, int64_t cols, int batch,
                   bool transposed, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int row_tiles = static_cast<int>((rows + 127) / 128), chunks = static_cast<int>((cols + 255) / 256);
    if (transposed) {
        auto kern = rows % 2 == 0 ? quantize_cols_kernel<BF16, true, RELU2, MAP> : quantize_cols_kernel<BF16, false, RELU2, MAP>;
        return launch_pdl(kern, grid_for(static_cast<int64_t>(row_tiles) * 2 * batch, chunks), dim3(kThreads), 0, s, x,
                          row_map, map_div, source_rows, rows, cols, row_tiles, chunks, codes, scales);
    }
    if constexpr (BF16) {
        int64_t warps = static_cast<int64_t>(row_tiles) * batch * 4 * chunks * 2;
        const int halves = warps <= static_cast<int64_t>(sm_total()) * kHalfWarps ? 2 : 1;
        warps *= halves;
        const int w = warps_per_cta(warps);
        auto kern = halves == 2 ? (cols % 8 == 0 ? quantize_blocks_kernel<RELU2, MAP != 0, true, 2> : quantize_blocks_kernel<RELU2, MAP != 0, false, 2>)
                                : (cols % 8 == 0 ? quantize_blocks_kernel<RELU2, MAP != 0, true, 1> : quantize_blocks_kernel<RELU2, MAP != 0, false, 1>);
        return launch_pdl(kern, dim3(static_cast<unsigned>((warps + w - 1) / w)), dim3(32 * w), 0, s,
                          static_cast<const uint16_t *>(x), row_map, map_div, source_rows, rows, cols, row_tiles, chunks * 2,
                          static_cast<uint32_t>(warps), codes, scales);
    } else {
        auto kern = cols % 4 == 0 ? quantize_rows_kernel<true, RELU2, MAP != 0> : quantize_rows_kernel<false, RELU2, MAP != 0>;
        return launch_pdl(kern, grid_for(static_cast<int64_t>(row_tiles) * 4 * batch, chunks), dim3(kThreads), 0, s,
                          static_cast<const float *>(x), row_map, map_div, source_rows, rows, cols, row_tiles, chunks, codes, scales);
    }
}

template <bool BF16>
int quantize_dtype(const void *x, const int *row_map, int map_div, int source_rows, int64_t rows, int64_t cols, int batch,
                   bool transposed, bool relu2, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
#define MLPBLK_Q(R, M) return quantize_typed<BF16, R, M>(x, row_map, map_div, source_rows, rows, cols, batch, transposed, codes, scales, s)
#define MLPBLK_QM(R)                          \
    {                                         \
        if (!row_map) MLPBLK_Q(R, 0);         \
        if (map_div == 0) MLPBLK_Q(R, 1);     \
        MLPBLK_Q(R, 2);                       \
    }
    if (relu2) MLPBLK_QM(true)
    MLPBLK_QM(false)
#undef MLPBLK_QM
#undef MLPBLK_Q
}

template <bool BF16>
int dequantize_typed(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, int batch, void *y,
                     cudaStream_t s) {
    const int row_tiles = static_cast<int>((rows + 127) / 128);
    const bool aligned = cols * (BF16 ? 2 : 4) % 16 == 0;
    const int pieces = static_cast<int>((cols + 255) / 256);
    const int64_t all = rows * batch * pieces;
    // more pieces a warp as there are more warps than the SMs hold (float32, from L2: 8 x 4096
    // 1.7 us with four pieces, 1.2 with one; 1031 x 4095 5.1 and 4.5 with two; 4096 x 4096
    // 10.8, 11.5 with two)
    const int64_t sms = sm_total();
#define MLPBLK_DEQ(W, N)                                                                                              \
    return launch_pdl(aligned ? dequantize_kernel<BF16, true, W, N> : dequantize_kernel<BF16, false, W, N>,           \
                      dim3(static_cast<unsigned>((all + W * N - 1) / (W * N))), dim3(32 * W), 0, s, codes, scales,     \
                      rows, cols, row_tiles, pieces, static_cast<uint32_t>(all), y)
    if (all <= 8 * sms) MLPBLK_DEQ(1, 1);
    if (all <= 192 * sms) MLPBLK_DEQ(4, 2);
    MLPBLK_DEQ(4, 4);
#undef MLPBLK_DEQ
}

}  // namespace

int launch_fp4_quantize(int dtype, const void *x, const int *row_map, int map_div, int source_rows, int64_t rows,
                        int64_t cols, int batch, bool transposed, bool relu2, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    return dtype == MLPBLK_BF16
               ? quantize_dtype<true>(x, row_map, map_div, source_rows, rows, cols, batch, transposed, relu2, codes, scales, s)
               : quantize_dtype<false>(x, row_map, map_div, source_rows, rows, cols, batch, transposed, relu2, codes, scales, s);
}

int launch_fp4_dequantize(int dtype, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                          int batch, void *y, cudaStream_t s) {
    return dtype == MLPBLK_BF16 ? dequantize_typed<true>(codes, scales, rows, cols, batch, y, s)
                                : dequantize_typed<false>(codes, scales, rows, cols, batch, y, s);
}

}  // namespace mlpblk
