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
__device__ __forceinline__ int source_row(const int *row_map, int map_div, int64_t r) {
    const int m = row_map[r];
    return m < 0 ? -1 : (map_div > 0 ? m / map_div : static_cast<int>(r));
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
    __device__ __forceinline__ void load_shared(const uint16_t *p) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
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

// Blocks along the source's rows.  A CTA takes 8 values of r % 32 of one 128-row scale
// tile, a warp the rows r, r + 32, r + 64, r + 96, 256 columns at a time: a lane holds
// 8 consecutive values of each row, a block is four lanes, and the four rows'
// scales of 4 blocks are 16 consecutive bytes of a tile (one store), with the next
// row's beside them.  The four rows' loads are in flight together.
template <bool BF16, bool VEC, bool RELU2, bool MAP>
__global__ void __launch_bounds__(kThreads, BF16 && VEC ? (RELU2 ? 4 : 5) : 3)
quantize_rows_kernel(const void *__restrict__ x, const int *__restrict__ row_map, int map_div, int64_t rows,
                     int64_t cols, int row_tiles, int chunks, uint8_t *__restrict__ codes,
                     uint8_t *__restrict__ scales) {
    using T = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ __align__(16) T turn[VEC ? 1 : kWarps][4][VEC ? 8 : 256];
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const int64_t ld = fp4_row_bytes(cols);
    const int tile = static_cast<int>(blockIdx.x >> 2);  // of the whole batch
    const int mat = tile / row_tiles;
    const int rr = static_cast<int>(blockIdx.x & 3) * 8 + (threadIdx.x >> 5);
    const int64_t r0 = static_cast<int64_t>(tile - mat * row_tiles) * 128 + rr;
    const T *src[4];
    bool live[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + 32 * j;
        int64_t at = r < rows ? r : -1;
        if (MAP && r < rows) at = source_row(row_map, map_div, r);
        live[j] = at >= 0;
        src[j] = static_cast<const T *>(x) + (mat * rows + (at < 0 ? 0 : at)) * cols;
    }
    uint8_t *out = codes + (mat * rows + r0) * ld;
    for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
        const int64_t c = static_cast<int64_t>(chunk) * 256 + lane * 8;
        Oct<BF16> o[4];
        if (VEC) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (live[j]) o[j].load(src[j], c, cols);
                else o[j].zero();
            }
        } else {
            T *mine = &turn[VEC ? 0 : threadIdx.x >> 5][0][0];
            const int64_t c0 = static_cast<int64_t>(chunk) * 256 + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) mine[j * 256 + 32 * i + lane] = live[j] && c0 + 32 * i < cols ? __ldg(src[j] + c0 + 32 * i) : T(0);
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
            typename Oct<BF16>::Max top = Oct<BF16>::kNone;
            o[j].template top<RELU2>(top);
            uint32_t m = top_bits<RELU2>(top);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t sb = scale_byte(m);
            o[j].template scaled<RELU2>(scale_inverse(sb), v);
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

// Blocks along the source's rows, rows of 768 columns and more in 16-byte accesses: a
// lane holds a whole block (its 16-byte loads 64 or 128 bytes from its neighbour's; the
// sectors' other halves come from L1), so a block's maximum needs no shuffle and its
// codes are one 16-byte store.  A warp takes 1024 columns of the rows r, r + 32, r + 64,
// r + 96 of a scale tile, two rows in flight; four lanes then transpose their 4 x 4
// scale bytes and store 16 consecutive bytes of a tile.  8192 x 16384 bf16: 61 us with the
// kernel above, 56 with this one (6.06 TB/s); below 24 blocks a row too many lanes idle.
template <bool BF16, bool RELU2, bool MAP>
__global__ void __launch_bounds__(kThreads, BF16 && !RELU2 ? 3 : 2)
quantize_blocks_kernel(const void *__restrict__ x, const int *__restrict__ row_map, int map_div, int64_t rows,
                       int64_t cols, int row_tiles, int chunks, uint8_t *__restrict__ codes,
                       uint8_t *__restrict__ scales) {
    using T = typename std::conditional<BF16, uint16_t, float>::type;
    constexpr int kParts = 4;                    // Octs of a block
    constexpr int kRows = BF16 ? 2 : 1;          // rows in flight
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const int64_t ld = fp4_row_bytes(cols);
    const int col_tiles = chunks * 2;
    const int tile = static_cast<int>(blockIdx.x >> 2);  // of the whole batch
    const int mat = tile / row_tiles;
    const int rr = static_cast<int>(blockIdx.x & 3) * 8 + (threadIdx.x >> 5);
    const int64_t r0 = static_cast<int64_t>(tile - mat * row_tiles) * 128 + rr;
    int64_t src[4];  // source rows, -1: zeros
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + 32 * j;
        src[j] = r < rows ? r : -1;
        if (MAP && r < rows) src[j] = source_row(row_map, map_div, r);
    }
    const T *base = static_cast<const T *>(x) + static_cast<int64_t>(mat) * rows * cols;
    uint8_t *out = codes + (mat * rows + r0) * ld;
    uint8_t *st = scales + static_cast<int64_t>(tile) * col_tiles * 512 + rr * 16 + (lane & 3) * 4;
    for (int64_t blk = static_cast<int64_t>(blockIdx.y) * 32 + lane; blk - lane < col_tiles * 4;
         blk += static_cast<int64_t>(gridDim.y) * 32) {
        const int64_t c = blk * 32;
        uint32_t bytes = 0;  // of the four rows
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += kRows) {
            Oct<BF16> o[kRows][kParts];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    if (src[j0 + u] >= 0) o[u][q].load(base + src[j0 + u] * cols, c + 8 * q, cols);
                    else o[u][q].zero();
                }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int j = j0 + u;
                const bool row = r0 + 32 * j < rows && c < 2 * ld;
                if (src[j] < 0) {  // a row of zeros, or none
                    if (row) *reinterpret_cast<uint4 *>(out + 32 * j * ld + c / 2) = make_uint4(0u, 0u, 0u, 0u);
                    continue;
                }
                typename Oct<BF16>::Max top = Oct<BF16>::kNone;
#pragma unroll
                for (int q = 0; q < kParts; ++q) o[u][q].template top<RELU2>(top);
                const uint32_t sb = scale_byte(top_bits<RELU2>(top));
                const float inv = scale_inverse(sb);
                uint32_t w[kParts];
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    float v[8];
                    o[u][q].template scaled<RELU2>(inv, v);
                    w[q] = sb == 255u ? 0u : e2m1x8<RELU2>(v);
                }
                if (row) *reinterpret_cast<uint4 *>(out + 32 * j * ld + c / 2) = make_uint4(w[0], w[1], w[2], w[3]);
                bytes |= sb << (8 * j);
            }
        }
        // byte j of lane b -> byte b of lane j, within four lanes
        uint32_t t = __shfl_xor_sync(0xffffffffu, bytes, 1);
        bytes = (lane & 1) ? __byte_perm(bytes, t, 0x3715) : __byte_perm(bytes, t, 0x6240);
        t = __shfl_xor_sync(0xffffffffu, bytes, 2);
        bytes = (lane & 2) ? __byte_perm(bytes, t, 0x3276) : __byte_perm(bytes, t, 0x5410);
        if (blk < col_tiles * 4) *reinterpret_cast<uint32_t *>(st + (blk >> 2) * 512) = bytes;
    }
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
quantize_cols_kernel(const void *__restrict__ x, const int *__restrict__ row_map, int map_div, int64_t rows,
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
    for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
        const int64_t c0 = static_cast<int64_t>(chunk) * 256 + wid * 32;  // Q's first column of this warp: x's row
        Pair<BF16> p[32];
        if (MAP == 2) {
            const int64_t own = c0 + lane;
            const int mine = own < cols ? source_row(row_map, map_div, own) : -1;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int src = __shfl_sync(0xffffffffu, mine, i);
                p[i].template load<VEC>(base + (src < 0 ? 0 : src) * rows, src < 0 ? rows : col, rows);
            }
        } else if (MAP == 1) {
            const int64_t own = c0 + lane;
            const unsigned live = __ballot_sync(0xffffffffu, own < cols && row_map[own < cols ? own : 0] >= 0);
            const T *row = base + c0 * rows;
            if (live == 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < 32; ++i, row += rows) p[i].template load<VEC>(row, col, rows);
            } else {
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
        uint32_t sa, sb;
        uint4 qa, qb;
        quantize_pairs<BF16, RELU2>(p, qa, qb, sa, sb);
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

// A warp per row, 1024 columns at a time: a lane takes 8 values of each 256, 4 bytes of
// codes and their block's scale byte, with four of them in flight.
constexpr int kDeqChunks = 4;

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows, int64_t cols,
                  int64_t all_rows, int row_tiles, int chunks, void *__restrict__ y) {
    using T = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ __align__(16) float turn[VEC ? 1 : kWarps][VEC ? 4 : 256];
    griddep_enter();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= all_rows) return;
    const int64_t mat = row / rows, r = row - mat * rows, ld = fp4_row_bytes(cols);
    const uint8_t *in = codes + row * ld + lane * 4;
    const uint8_t *sc = scales + (mat * row_tiles + r / 128) * chunks * 1024 + (lane >> 4) * 512 + (r % 32) * 16 +
                        (r % 128) / 32 * 4 + ((lane >> 2) & 3);
    T *out = static_cast<T *>(y) + row * cols;
    for (int g = blockIdx.y * kDeqChunks; g < chunks; g += gridDim.y * kDeqChunks) {
        uint32_t u[kDeqChunks], sb[kDeqChunks];
#pragma unroll
        for (int j = 0; j < kDeqChunks; ++j) {
            const int64_t c = static_cast<int64_t>(g + j) * 256 + lane * 8;
            u[j] = sb[j] = 0u;
            if (c < cols) {
                u[j] = __ldg(reinterpret_cast<const uint32_t *>(in + static_cast<int64_t>(g + j) * 128));
                sb[j] = __ldg(sc + static_cast<int64_t>(g + j) * 1024);
            }
        }
#pragma unroll
        for (int j = 0; j < kDeqChunks; ++j) {
            const int64_t c = static_cast<int64_t>(g + j) * 256 + lane * 8;
            if (g + j >= chunks) break;
            if (!VEC) {
                // rows of any length: through shared memory, so that neighbouring lanes
                // store neighbouring columns
                float v[8];
                decode8(u[j], scale_value(sb[j]), v);
                float *mine = &turn[VEC ? 0 : threadIdx.x >> 5][0];
                *reinterpret_cast<float4 *>(mine + lane * 8) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(mine + lane * 8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
                __syncwarp();
                const int64_t c0 = static_cast<int64_t>(g + j) * 256 + lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = mine[32 * i + lane];
                    if (c0 + 32 * i < cols) {
                        if (BF16) reinterpret_cast<uint16_t *>(out)[c0 + 32 * i] = static_cast<uint16_t>(pack2(f, 0.0f) & 0xFFFFu);
                        else reinterpret_cast<float *>(out)[c0 + 32 * i] = f;
                    }
                }
                __syncwarp();
                continue;
            }
            if (c >= cols) continue;
            float v[8];
            decode8(u[j], scale_value(sb[j]), v);
            if (BF16) {
                *reinterpret_cast<uint4 *>(out + c) =
                    make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
            } else {
                *reinterpret_cast<float4 *>(out + c) = make_float4(v[0], v[1], v[2], v[3]);
                if (c + 4 < cols) *reinterpret_cast<float4 *>(out + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
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

template <bool BF16, bool RELU2, int MAP>
int quantize_typed(const void *x, const int *row_map, int map_div, int64_t rows, int64_t cols, int batch,
                   bool transposed, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    const int row_tiles = static_cast<int>((rows + 127) / 128), chunks = static_cast<int>((cols + 255) / 256);
    if (transposed) {
        auto kern = rows % 2 == 0 ? quantize_cols_kernel<BF16, true, RELU2, MAP> : quantize_cols_kernel<BF16, false, RELU2, MAP>;
        return launch_pdl(kern, grid_for(static_cast<int64_t>(row_tiles) * 2 * batch, chunks), dim3(kThreads), 0, s, x,
                          row_map, map_div, rows, cols, row_tiles, chunks, codes, scales);
    }
    if (cols * (BF16 ? 2 : 4) % 16 == 0 && cols >= 768)
        return launch_pdl(quantize_blocks_kernel<BF16, RELU2, MAP != 0>,
                          grid_for(static_cast<int64_t>(row_tiles) * 4 * batch, (chunks + 3) / 4), dim3(kThreads), 0, s, x, row_map,
                          map_div, rows, cols, row_tiles, chunks, codes, scales);
    auto kern = cols * (BF16 ? 2 : 4) % 16 == 0 ? quantize_rows_kernel<BF16, true, RELU2, MAP != 0>
                                                : quantize_rows_kernel<BF16, false, RELU2, MAP != 0>;
    return launch_pdl(kern, grid_for(static_cast<int64_t>(row_tiles) * 4 * batch, chunks), dim3(kThreads), 0, s, x,
                      row_map, map_div, rows, cols, row_tiles, chunks, codes, scales);
}

template <bool BF16>
int quantize_dtype(const void *x, const int *row_map, int map_div, int64_t rows, int64_t cols, int batch,
                   bool transposed, bool relu2, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
#define MLPBLK_Q(R, M) return quantize_typed<BF16, R, M>(x, row_map, map_div, rows, cols, batch, transposed, codes, scales, s)
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
    const int row_tiles = static_cast<int>((rows + 127) / 128), chunks = static_cast<int>((cols + 255) / 256);
    const int64_t all = rows * batch;
    auto kern = cols * (BF16 ? 2 : 4) % 16 == 0 ? dequantize_kernel<BF16, true> : dequantize_kernel<BF16, false>;
    return launch_pdl(kern, grid_for((all + kWarps - 1) / kWarps, (chunks + kDeqChunks - 1) / kDeqChunks), dim3(kThreads), 0,
                      s, codes, scales, rows, cols, all, row_tiles, chunks, y);
}

}  // namespace

int launch_fp4_quantize(int dtype, const void *x, const int *row_map, int map_div, int64_t rows, int64_t cols,
                        int batch, bool transposed, bool relu2, uint8_t *codes, uint8_t *scales, cudaStream_t s) {
    return dtype == MLPBLK_BF16
               ? quantize_dtype<true>(x, row_map, map_div, rows, cols, batch, transposed, relu2, codes, scales, s)
               : quantize_dtype<false>(x, row_map, map_div, rows, cols, batch, transposed, relu2, codes, scales, s);
}

int launch_fp4_dequantize(int dtype, const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                          int batch, void *y, cudaStream_t s) {
    return dtype == MLPBLK_BF16 ? dequantize_typed<true>(codes, scales, rows, cols, batch, y, s)
                                : dequantize_typed<false>(codes, scales, rows, cols, batch, y, s);
}

}  // namespace mlpblk
