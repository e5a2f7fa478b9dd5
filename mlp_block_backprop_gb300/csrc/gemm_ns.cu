// gemm_ns.cu -- the products of a Newton-Schulz step on the tensor cores (tcgen05.mma
// kind::f16: fp16 operands, fp32 accumulator in TMEM):
//
//   G  = X X^T  (X wide)  or  X^T X  (X tall)
//   P  = b G + c G G
//   X' = a X + P X        or  a X + X P
//
// and, where X's long side is at least twice the short one (of 512 or more), two steps at a time with one product
// on X for both: with the first step's P1, G becomes (a1 I + P1) G (a1 I + P1), its own P2 follows, and
// X' = (a2 I + P2)(a1 I + P1) X = a1 a2 X + S X.  That trades a G and an update (3 m^2 n) for three
// more products of the short side (m^3 each, half of them mirrored): 16384 x 4096 takes 28% fewer
// operations.  G's own rounding errors then go through a second step, so it stays at two.  S cancels most of a1 a2 X on
// strong directions (-11 of 12), so what S X leaves out of X's low part counts eleven times: S's diagonal is kept out of
// the product, whole and in float32, and meets both parts of X with a1 a2 (one entry in 512 x 2560: off by 4.7e-3 with
// the diagonal in S, 1.2e-3 so; Gaussian 1.6e-3 and 0.7e-3).
//
// Nothing is transposed in memory: each operand is read K-major or MN-major as it lies,
// and a tall X is worked on from its right.  G and P are symmetric: only tiles on and
// above the diagonal are computed, the others are written as their mirror images.
//
// fp16, not bf16: the tensor cores run both at the same rate, and the values' range is
// known (X's singular values stay below about 1.2, so X is kept times sqrt of its long
// side, entries near 1; G and P, whose errors count against the identity's 1, as they are).
// Rounding is 2^-11 instead of 2^-8, which the polynomial amplifies: on momentum with a few
// strong directions the bf16 form is off by 1e-2 to 1e-1, this one by 1e-3 to 2e-3.  Two places get
// more than fp16:
//   - a X, which carries a weak direction (amplified by a = 3.4 a step) unchanged, takes X
//     as the sum of two fp16 values in all but the last step;
//   - P's diagonal, next to which its other entries are small, leaves what its rounding took
//     in float32 (`diag`), and the update adds it to a.
//
// ns_small: one CTA, 128 x 128 tiles, or 128 x 64 where those fit one round of the SMs; K can be split over a
//   cluster whose parts meet in distributed shared memory in rank order.
// ns_pair: two CTAs on two SMs, 256 x 256 tiles (cta_group::2).
// ns_fused: all steps of a small matrix in one launch of a cluster.
// Bound by the tensor cores at large sizes (16384 x 4096: 508 of 512 clocks a stage of K), by the copies from L2 where
// tiles are small, by launches and K's latency at the smallest.
#include <type_traits>

#include "gemm_tc.cuh"
#include "ortho.h"

namespace mlpblk {

namespace {

constexpr int kNsK = 64;                // K values of a stage: 128 bytes

struct NsArgs {
    int op;
    int rows, cols;                     // of D
    int mt, nt;                         // tiles
    int per;                            // tiles of one matrix (on and above the diagonal, or all)
    int tiles;                          // of the batch
    int kblocks;
    int group_m;
    int pitch;                          // elements of a row of out, aux
    int64_t matrix;                     // elements of a matrix of out, aux
    const __half *aux, *aux2;           // [rows][cols]: Y or X; X's low part (or NULL), or P (kNsJoin)
    const float *diag, *diag2;          // [batch][diag_pitch]
    float *diag_out;
    int diag_pitch;                     // a multiple of 64
    bool diag_col;                      // kNsUpdate: diag goes by column (tall)
    __half *out, *out_lo;
    uint16_t *o;                        // bf16 [batch][rows][cols]
    bool o_tma;                         // rows of o are whole 16-byte pieces
    float alpha, a, b, c;
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4)                                   // D format: f32 (A, B: f16 is code 0)
           | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16)
           | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// One lane of the warp, the same one each time: the issuing roles run their loops with the
// whole warp, so that addresses and descriptors stay in uniform registers.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  elect.sync _|p, 0xffffffff;\n"
        "  selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void mbar_expect_relaxed(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "  selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// mbar_wait for a barrier that other CTAs of the cluster arrive on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            record_device_error(MLPBLK_ETIMEOUT);
            return false;
        }
    }
}

// Before a producer leaves: waits (bounded) for the copies that it issued into the S stages,
// the next of which would be `stage` in phase `phase`, so that none writes shared memory after
// a run that gave up.
__device__ __forceinline__ void await_copies(uint64_t *bars, int S, int stage, uint32_t phase) {
    const uint64_t t0 = global_timer_ns();
    for (int s = 0; s < S; ++s)
        while (!mbar_try_wait(&bars[s], s < stage ? phase : phase ^ 1u) && global_timer_ns() - t0 <= kWaitLimitNs) {
        }
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void tma_load_4d(const CUtensorMap *map, uint64_t *bar, void *dst, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(const CUtensorMap *map, uint32_t bar_cluster_addr, void *dst, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// ------------------------------------------------------------------- the work

// One output tile: its matrix, origin, and whether its mirror image is written too.
struct NsTile {
    int batch, m0, n0;
    bool mirror;
};

template <int TM, int TN, bool SYM>
__device__ __forceinline__ NsTile ns_tile(const NsArgs &a, int t) {
    NsTile w;
    w.batch = t / a.per;
    const int r = t - w.batch * a.per;
    int mi, ni;
    if (SYM) {
        // column ni holds the tiles (0 .. ni, ni): ni (ni + 1) / 2 tiles lie before it
        ni = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
        while (ni * (ni + 1) / 2 > r) --ni;
        while ((ni + 1) * (ni + 2) / 2 <= r) ++ni;
        mi = r - ni * (ni + 1) / 2;
    } else {
        raster_tile(r, a.mt, a.nt, a.group_m, mi, ni);
    }
    w.m0 = mi * TM;
    w.n0 = ni * TN;
    w.mirror = SYM && mi != ni;
    return w;
}

// Loads of one operand's stage: ROWS rows (or, MN-major, columns) from `row` on, K block kb, in boxes of BOX.
template <bool MN, int ROWS = 128, int BOX = 128>
__device__ __forceinline__ void load_operand(const CUtensorMap *map, uint64_t *bar, uint8_t *dst, int kb, int row, int batch) {
#pragma unroll
    for (int i = 0; i < ROWS; i += BOX, row += BOX, dst += BOX * 128) {
        if (MN) tma_load_4d(map, bar, dst, 0, kb * kNsK, row / 64, batch);
        else tma_load_3d(map, bar, dst, kb * kNsK, row, batch);
    }
}
template <bool MN>
__device__ __forceinline__ void load_operand_pair(const CUtensorMap *map, uint32_t bar, void *dst, int kb, int row, int batch) {
    if (MN) tma_load_4d_pair(map, bar, dst, 0, kb * kNsK, row / 64, batch);
    else tma_load_3d_pair(map, bar, dst, kb * kNsK, row, batch);
}

// Descriptor of an operand's stage, and its step for the next 16 values of K.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(const void *s) {
    return MN ? smem_desc_sw128(smem_u32(s), 64 * 128, 1024) : smem_desc_sw128(smem_u32(s), 16, 1024);
}
template <bool MN>
constexpr uint64_t kOperandStep = MN ? (16 * 128) >> 4 : 32 >> 4;

// ---------------------------------------------------------------- the epilogue

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

template <int OP>
constexpr bool kNsOne = OP != kNsGram;                      // reads a tile besides the accumulator
template <int OP>
constexpr bool kNsTwo = OP == kNsUpdate || OP == kNsJoin;   // two tiles
template <int OP>
constexpr bool kNsScaled = OP == kNsUpdate || OP == kNsApply || OP == kNsJoin;   // (a + diag) times the first

// The step's arithmetic on a pair of columns (col, col + 1) of a row: v the accumulators, p and q the first and
// second tile's values, d the row's diag, dc the columns' (tall updates, kNsJoin's diag2).
template <int OP>
__device__ __forceinline__ float2 ns_combine(const NsArgs &a, float2 v, float2 p, float2 q, float d, float2 dc, int row, int col) {
    if (OP == kNsGram) return make_float2(a.alpha * v.x, a.alpha * v.y);
    if (OP == kNsSquare) return make_float2(a.b * p.x + a.c * v.x, a.b * p.y + a.c * v.y);
    if (OP == kNsApply) return make_float2((a.a + d) * p.x + v.x, (a.a + d) * p.y + v.y);
    if (OP == kNsJoin) {
        float2 r = make_float2((a.a + d) * p.x + (a.b + dc.x) * q.x + v.x, (a.a + d) * p.y + (a.b + dc.y) * q.y + v.y);
        if (col == row) r.x += (a.a + d) * dc.x + a.b * d;
        if (col + 1 == row) r.y += (a.a + d) * dc.y + a.b * d;
        return r;
    }
    const float d0 = a.diag_col ? dc.x : d, d1 = a.diag_col ? dc.y : d;
    return make_float2((a.a + d0) * (p.x + q.x) + v.x, (a.a + d1) * (p.y + q.y) + v.y);
}

// Tensor maps of the epilogue: chunks of 32 rows x 64 columns (128 bytes, swizzled) or 32 (64 bytes,
// swizzled) of what it reads and writes, and of its mirror image (32 columns, as they lie).
struct NsMaps {
    CUtensorMap aux, aux2, out, out_lo, mirror;
};
struct NsMapRefs {
    const CUtensorMap *aux, *aux2, *out, *out_lo, *mirror;
    __device__ __forceinline__ NsMapRefs() {}
    __device__ __forceinline__ NsMapRefs(const NsMaps &m) : aux(&m.aux), aux2(&m.aux2), out(&m.out), out_lo(&m.out_lo), mirror(&m.mirror) {}
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

constexpr int kNsChunkBytes = 32 * 128;
constexpr int kNsStaging = 2 * kNsChunkBytes;   // a warp's: the first tile's chunk, in whose place the output is
                                                // staged, and the second one's, or the output's low part, or the image

// One warp's part of a tile: rows [row0, row0 + 32), chunks of CC columns (64 or 32) from col0 on.
// buf0, buf1: its staging; bar, phase: the barrier of its loads.
template <int OP, int CC = 64>
struct NsEpilogue {
    static constexpr int kBytes = 32 * CC * 2;      // of a chunk
    static constexpr int kRow = CC * 2;
    const NsArgs &a;
    const NsMapRefs maps;
    uint8_t *buf0, *buf1;
    uint64_t *bar;
    volatile int *abort;
    int lane;
    uint32_t phase;

    __device__ __forceinline__ bool on(const NsTile &, int row0, int col0) const { return row0 < a.rows && col0 < a.cols; }
    __device__ __forceinline__ bool second() const { return OP == kNsJoin || (OP == kNsUpdate && a.aux2 != nullptr); }

    // What the swizzle of a row's 16-byte pieces is: of 128-byte rows, or of 64-byte ones.
    static __device__ __forceinline__ int swizzle(int row) { return CC == 64 ? row & 7 : row >> 1 & 3; }

    // Asks for a chunk's tiles, once the stores from the same place have read it.
    __device__ __forceinline__ void load(const NsTile &w, int row0, int col0) {
        if (!kNsOne<OP> || !on(w, row0, col0)) return;
        if (lane == 0) {
            bulk_wait_group_read<0>();
            mbar_expect_relaxed(bar, second() ? 2 * kBytes : kBytes);
            tma_load_3d(maps.aux, bar, buf0, col0, row0, w.batch);
            if (second()) tma_load_3d(maps.aux2, bar, buf1, col0, row0, w.batch);
        }
        __syncwarp();
    }

    // The chunk from its accumulators v (row `lane`, CC columns).  The whole warp calls it.
    __device__ __forceinline__ bool finish(const NsTile &w, int row0, int col0, float (&v)[CC]) {
        if (!on(w, row0, col0)) return true;
        const int row = row0 + lane;
        const uint32_t at0 = smem_u32(buf0) + lane * kRow, at1 = smem_u32(buf1) + lane * kRow;
        const uint32_t sw = static_cast<uint32_t>(swizzle(lane));
        if (kNsOne<OP>) {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase, abort));
            phase ^= 1u;
            if (!ok) return false;
        } else {
            if (lane == 0) bulk_wait_group_read<0>();   // the staging is free again
            __syncwarp();
        }
        const int64_t dat = static_cast<int64_t>(w.batch) * a.diag_pitch;
        const float d = kNsScaled<OP> && !a.diag_col && row < a.rows ? __ldcg(a.diag + dat + row) : 0.0f;
        const float *by_col = OP == kNsJoin ? a.diag2 : (OP == kNsUpdate && a.diag_col ? a.diag : nullptr);
        const bool two = second();
#pragma unroll
        for (int j = 0; j < CC / 8; ++j) {   // eight columns: 16 bytes of each tile
            const uint32_t off = (static_cast<uint32_t>(j) ^ sw) << 4;
            uint4 x = make_uint4(0, 0, 0, 0), y = make_uint4(0, 0, 0, 0);
            if (kNsOne<OP>) x = ld_shared_v4(at0 + off);
            if (kNsTwo<OP> && two) y = ld_shared_v4(at1 + off);
            float4 c0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), c1 = c0;
            if (kNsTwo<OP> && by_col) {   // (the pitch is a multiple of 64)
                c0 = __ldcg(reinterpret_cast<const float4 *>(by_col + dat + col0 + 8 * j));
                c1 = __ldcg(reinterpret_cast<const float4 *>(by_col + dat + col0 + 8 * j + 4));
            }
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
            const float2 cs[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 8 * j + 2 * i;
                const float2 r = ns_combine<OP>(a, make_float2(v[k], v[k + 1]), unpack_half2(xs[i]), unpack_half2(ys[i]), d, cs[i], row, col0 + k);
                v[k] = r.x;
                v[k + 1] = r.y;
            }
        }
        if ((OP == kNsSquare || OP == kNsJoin) && row0 < col0 + CC && col0 < row0 + 32) {
            // the chunk lies on the diagonal: what rounding takes from the lane's value there (kNsJoin: all of it)
            const int at = row - col0;
            float x = 0.0f;
#pragma unroll
            for (int k = 0; k < CC; ++k) {
                x = k == at ? v[k] : x;
                if (OP == kNsJoin) v[k] = k == at ? 0.0f : v[k];
            }
            if (at >= 0 && at < CC && row < a.rows) a.diag_out[dat + row] = OP == kNsJoin ? x : x - __half2float(__float2half_rn(x));
        }
        if (OP == kNsUpdate && a.o) {
#pragma unroll
            for (int j = 0; j < CC / 8; ++j) {
                const float *e = &v[8 * j];
                st_shared_v4(at0 + ((static_cast<uint32_t>(j) ^ sw) << 4), pack_bf16x2(a.alpha * e[0], a.alpha * e[1]), pack_bf16x2(a.alpha * e[2], a.alpha * e[3]),
                             pack_bf16x2(a.alpha * e[4], a.alpha * e[5]), pack_bf16x2(a.alpha * e[6], a.alpha * e[7]));
            }
            if (!a.o_tma) {
                // rows of any length: a row a step, neighbouring lanes neighbouring columns
                __syncwarp();
                const int n_rows = min(32, a.rows - row0);
                uint16_t *o = a.o + (static_cast<int64_t>(w.batch) * a.rows + row0) * a.cols + col0 + lane;
                const bool in0 = col0 + lane < a.cols, in1 = CC == 64 && col0 + lane + 32 < a.cols;
                for (int r = 0; r < n_rows; ++r, o += a.cols) {
                    const uint8_t *from = buf0 + r * kRow;
                    const int b0 = 2 * lane, b1 = b0 + 64;
                    if (in0) o[0] = *reinterpret_cast<const uint16_t *>(from + ((((b0 >> 4) ^ swizzle(r)) << 4) | (b0 & 15)));
                    if (in1) o[32] = *reinterpret_cast<const uint16_t *>(from + ((((b1 >> 4) ^ swizzle(r)) << 4) | (b1 & 15)));
                }
                __syncwarp();
                return true;
            }
        } else {
#pragma unroll
            for (int j = 0; j < CC / 8; ++j) {
                const float *e = &v[8 * j];
                const uint32_t off = (static_cast<uint32_t>(j) ^ sw) << 4;
                const uint32_t h[4] = {pack_half2(e[0], e[1]), pack_half2(e[2], e[3]), pack_half2(e[4], e[5]), pack_half2(e[6], e[7])};
                st_shared_v4(at0 + off, h[0], h[1], h[2], h[3]);
                if (OP == kNsUpdate && a.out_lo) {
                    uint32_t l[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 p = unpack_half2(h[i]);
                        l[i] = pack_half2(e[2 * i] - p.x, e[2 * i + 1] - p.y);
                    }
                    st_shared_v4(at1 + off, l[0], l[1], l[2], l[3]);
                }
            }
            if (OP != kNsUpdate && w.mirror) {
                if (kNsTwo<OP>) __syncwarp();   // every lane has read its row of the second tile
                // the image's row j holds this chunk's column j: 32 values, 64 bytes; two lanes swap every
                // other value, so that a store is a pair
                const int odd = lane & 1;
                uint32_t to = smem_u32(buf1) + odd * 64 + (lane - odd) * 2;
#pragma unroll
                for (int j = 0; j < CC; j += 2) {
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                    const uint32_t u = odd ? pack_half2(got, v[j + 1]) : pack_half2(v[j], got);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(u) : "memory");
                    to += 128;
                }
            }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(maps.out, buf0, col0, row0, w.batch);
            if (OP == kNsUpdate && a.out_lo && !a.o) tma_store_3d(maps.out_lo, buf1, col0, row0, w.batch);
            if (OP != kNsUpdate && w.mirror) tma_store_3d(maps.mirror, buf1, row0, col0, w.batch);
            bulk_commit_group();
        }
        __syncwarp();
        return true;
    }
};

// A warp's accumulators of 64 or 32 columns.
__device__ __forceinline__ void ns_accumulators(uint32_t at, float (&v)[64]) {
    tmem_load_64cols(at, *reinterpret_cast<float(*)[32]>(&v[0]), *reinterpret_cast<float(*)[32]>(&v[32]));
}
__device__ __forceinline__ void ns_accumulators(uint32_t at, float (&v)[32]) { tmem_load_32cols(at, v); }

// ------------------------------------------------------------------- ns_small

// SPLIT (G alone): K is split over a cluster; the parts meet in `dump`, and a CTA finishes some of the
// tile's rows, 16 neighbouring threads a row, straight to global memory.  No mirror images there:
// a split is for products that leave SMs idle, so every tile is computed.
template <bool SPLIT_, int BN_ = 128>
struct NsSmall {
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int BN = BN_;                  // columns of a tile
    static constexpr int kEpiWarps = 8;             // two a lane quarter: half of the columns each
    static constexpr int kCols = BN / 2;            // a chunk's
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kABytes = 128 * 128, kBBytes = BN * 128;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static_assert(!SPLIT || BN == 128, "the cluster's sum");
    static constexpr int kDumpPitch = 132;          // floats of a row: 16-byte accesses of eight rows meet in no bank
    static constexpr int kDumpBytes = SPLIT ? 128 * kDumpPitch * 4 : kEpiWarps * kNsStaging;
    static constexpr int kCtrlBytes = 1024;
    static constexpr int kFit = (kSmemLimit - 1024 - kCtrlBytes - kDumpBytes) / kStageBytes, kStages = kFit < 8 ? kFit : 8;
    static constexpr int kSmemBytes = 1024 + kCtrlBytes + kDumpBytes + kStages * kStageBytes;
    static_assert(kStages >= 4, "pipeline");
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr) : "memory");
    return v;
}

// Eight columns from col on of a row of G, whose sums are v: the split kernel's epilogue.
__device__ __forceinline__ void ns_finish_eight(const NsArgs &a, const NsTile &w, int row, int col, const float (&v)[8]) {
    if (row >= a.rows || col >= a.cols) return;
    // (the pitch is a multiple of 64: what lies behind the last column is nobody's)
    *reinterpret_cast<uint4 *>(a.out + w.batch * a.matrix + static_cast<int64_t>(row) * a.pitch + col) =
        make_uint4(pack_half2(a.alpha * v[0], a.alpha * v[1]), pack_half2(a.alpha * v[2], a.alpha * v[3]), pack_half2(a.alpha * v[4], a.alpha * v[5]),
                   pack_half2(a.alpha * v[6], a.alpha * v[7]));
}

template <class C, int OP, bool AMN, bool BMN>
__global__ void __launch_bounds__(C::kThreads, 1)
ns_small_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const __grid_constant__ NsMaps maps, const NsArgs args) {
    constexpr bool SYM = OP != kNsUpdate && !C::SPLIT && C::BN == 128;
    constexpr int S = C::kStages, BN = C::BN;
    static_assert(!C::SPLIT || OP == kNsGram, "the cluster's sum");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *a_s = smem, *b_s = a_s + S * C::kABytes;
    uint8_t *staging = b_s + S * C::kBBytes;                 // the epilogue warps' chunks, or
    float *dump = reinterpret_cast<float *>(staging);        // [row][column], pitch kDumpPitch
    uint8_t *ctrl = staging + C::kDumpBytes;
    uint64_t *full_bar = reinterpret_cast<uint64_t *>(ctrl);
    uint64_t *empty_bar = full_bar + S;
    uint64_t *accf_bar = empty_bar + S;
    uint64_t *acce_bar = accf_bar + 2;
    uint64_t *part_full = acce_bar + 2;   // every CTA of the cluster has its part in `dump`
    uint64_t *part_empty = part_full + 1; // every CTA has read this CTA's part
    uint64_t *aux_bar = part_empty + 1;   // a warp's chunk has been loaded
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 512);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 516);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int cs = C::SPLIT ? static_cast<int>(cluster_nctarank()) : 1;
    const int rank = C::SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    const int worker = static_cast<int>(blockIdx.x) / cs, workers = static_cast<int>(gridDim.x) / cs;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], C::kEpiWarps);
        }
        mbar_init(part_full, cs);
        mbar_init(part_empty, cs);
        for (int b = 0; b < C::kEpiWarps; ++b) mbar_init(&aux_bar[b], 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (cs > 1) cluster_sync();  // the peers' barriers exist before anyone arrives on them
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    griddep_launch_dependents();
    int t = worker;
    NsTile w = {};
    if (t < args.tiles) w = ns_tile<128, BN, SYM>(args, t);
    auto next = [&]() {
        t += workers;
        if (t < args.tiles) w = ns_tile<128, BN, SYM>(args, t);
    };
    const int k0 = args.kblocks * rank / cs, k1 = args.kblocks * (rank + 1) / cs;
    griddep_wait();

    if (warp == 0) {
        const bool issue = elect_lane();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < args.tiles; next()) {
            for (int kb = k0; kb < k1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                if (issue) {
                    mbar_expect_relaxed(&full_bar[stage], C::kStageBytes);
                    load_operand<AMN, 128, BN>(&tmA, &full_bar[stage], a_s + stage * C::kABytes, kb, w.m0, w.batch);
                    load_operand<BMN, BN, BN>(&tmB, &full_bar[stage], b_s + stage * C::kBBytes, kb, w.n0, w.batch);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        await_copies(full_bar, S, stage, phase);
        __syncwarp();
    } else if (warp == 1) {
        const bool issue = elect_lane();
        const uint64_t a0 = operand_desc<AMN>(a_s), b0 = operand_desc<BMN>(b_s);
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < args.tiles; next(), ++it) {
            const int buf = it & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[buf], ((it >> 1) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            tc_fence_after_sync();
            for (int kb = k0; kb < k1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t ad = a0 + stage * (C::kABytes >> 4), bd = b0 + stage * (C::kBBytes >> 4);
                if (issue) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_bf16(tmem_base + buf * BN, ad + j * kOperandStep<AMN>, bd + j * kOperandStep<BMN>,
                                  idesc_f16_f32(128, BN, AMN, BMN), (kb > k0 || j > 0) ? 1u : 0u);
                    umma_commit(&empty_bar[stage]);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if (issue) umma_commit(&accf_bar[buf]);
            __syncwarp();
        }
        __syncwarp();
    } else if constexpr (!C::SPLIT) {
        const int q = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
        uint8_t *st = staging + ew * kNsStaging;
        NsEpilogue<OP, C::kCols> epi = {args, NsMapRefs(maps), st, st + kNsChunkBytes, &aux_bar[ew], abort_flag, lane, 0};
        auto place = [&](const NsTile &x, int &row, int &col) { row = x.m0 + 32 * q, col = x.n0 + C::kCols * half; };
        int it = 0, row, col;
        if (t < args.tiles) {
            place(w, row, col);
            epi.load(w, row, col);
        }
        while (t < args.tiles) {
            place(w, row, col);
            const int buf = it & 1;
            bool ok = __all_sync(0xffffffffu, mbar_wait(&accf_bar[buf], (it >> 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after_sync();
            float v[C::kCols];
            ns_accumulators(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * BN + C::kCols * half, v);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(&acce_bar[buf]);
            if (!epi.finish(w, row, col, v)) break;
            next();
            ++it;
            if (t < args.tiles) {
                place(w, row, col);
                epi.load(w, row, col);
            }
        }
        if (lane == 0) {
            bulk_wait_group<0>();
            if (*abort_flag) mbar_drain(&aux_bar[ew], epi.phase);   // a load may still be on its way
        }
        __syncwarp();
    } else {
        // A warp that gave up on a wait keeps walking (its waits then return at once), so that
        // the barriers of the cluster's sum stay in step.
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int i = 32 * q + lane, tid = static_cast<int>(threadIdx.x) - 64;
        constexpr int kEpiThreads = 32 * C::kEpiWarps;
        const int rows = 128 / cs, first = rank * rows;      // this CTA's rows of the tile
        int it = 0;
        for (; t < args.tiles; next(), ++it) {
            const bool some = k1 > k0;
            const int buf = it & 1;
            const int r0 = tid >> 4, c0 = (tid & 15) * 8;
            bool ok = mbar_wait(&accf_bar[buf], (it >> 1) & 1, abort_flag);
            tc_fence_after_sync();
            ok = mbar_wait_cluster(part_empty, (it & 1) ^ 1u, abort_flag) && ok;
            ok = __all_sync(0xffffffffu, ok);
            for (int c = half * 64; c < half * 64 + 64; c += 32) {
                float v[32];
                if (some && ok) {
                    tmem_load_32cols(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * 128 + c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<float4 *>(dump + i * C::kDumpPitch + c + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(&acce_bar[buf]);
            named_barrier_sync(1, kEpiThreads);
            if (tid < cs) mbar_arrive_cluster(mapa_shared(smem_u32(part_full), tid));
            ok = mbar_wait_cluster(part_full, it & 1, abort_flag) && ok;
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                for (int r = r0; r < rows; r += kEpiThreads / 16) {
                    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                    const uint32_t from = smem_u32(dump + (first + r) * C::kDumpPitch + c0);
#pragma unroll 4
                    for (int k = 0; k < cs; ++k) {
                        const uint32_t at = mapa_shared(from, k);
                        const float4 p = ld_cluster_v4(at), u = ld_cluster_v4(at + 16);
                        sum[0] += p.x; sum[1] += p.y; sum[2] += p.z; sum[3] += p.w;
                        sum[4] += u.x; sum[5] += u.y; sum[6] += u.z; sum[7] += u.w;
                    }
                    ns_finish_eight(args, w, w.m0 + first + r, w.n0 + c0, sum);
                }
            }
            named_barrier_sync(1, kEpiThreads);
            if (tid < cs) mbar_arrive_cluster(mapa_shared(smem_u32(part_empty), tid));
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (cs > 1) cluster_sync();  // no CTA leaves while its part may be read
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, 256);
    }
}

// -------------------------------------------------------------------- ns_pair

struct NsPair {
    static constexpr int kEpiWarps = 16;            // four a lane quarter: 64 columns each, in two chunks
    static constexpr int kCols = 32;                // of a chunk
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kOpBytes = 128 * 128;      // 128 rows of A or B a CTA
    static constexpr int kStageBytes = 2 * kOpBytes;
    static constexpr int kCtrlBytes = 1024;
    static constexpr int kWarpStaging = 2 * 32 * kCols * 2, kStagingBytes = kEpiWarps * kWarpStaging;
    static constexpr int kStages = (kSmemLimit - 1024 - kCtrlBytes - kStagingBytes) / kStageBytes;
    static constexpr int kSmemBytes = 1024 + kCtrlBytes + kStagingBytes + kStages * kStageBytes;
    static_assert(kStages >= 4, "pipeline");
};

template <int OP, bool AMN, bool BMN>
__global__ void __launch_bounds__(NsPair::kThreads, 1)
ns_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const __grid_constant__ NsMaps maps, const NsArgs args) {
    using P = NsPair;
    constexpr bool SYM = OP != kNsUpdate;
    constexpr int S = P::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *a_s = smem, *b_s = a_s + S * P::kOpBytes;
    uint8_t *staging = b_s + S * P::kOpBytes;
    uint8_t *ctrl = staging + P::kStagingBytes;
    uint64_t *full_bar = reinterpret_cast<uint64_t *>(ctrl);
    uint64_t *empty_bar = full_bar + S;
    uint64_t *accf_bar = empty_bar + S;
    uint64_t *acce_bar = accf_bar + 2;
    uint64_t *aux_bar = acce_bar + 2;     // a warp's chunk has been loaded
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 512);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 516);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full_bar[s], 1);   // the leader's collects both CTAs' bytes
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], 2 * P::kEpiWarps);  // both CTAs' epilogue warps (the leader's barrier counts)
        }
        for (int b = 0; b < P::kEpiWarps; ++b) mbar_init(&aux_bar[b], 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    cluster_sync();
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_alloc_permit_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    griddep_launch_dependents();
    int t = worker;
    NsTile w = {};
    if (t < args.tiles) w = ns_tile<256, 256, SYM>(args, t);
    auto next = [&]() {
        t += workers;
        if (t < args.tiles) w = ns_tile<256, 256, SYM>(args, t);
    };
    griddep_wait();

    if (warp == 0) {
        const bool issue = elect_lane();
        const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < args.tiles; next()) {
            const int ar = w.m0 + static_cast<int>(rank) * 128, br = w.n0 + static_cast<int>(rank) * 128;
            for (int kb = 0; kb < args.kblocks; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                if (issue) {
                    uint8_t *da = a_s + stage * P::kOpBytes, *db = b_s + stage * P::kOpBytes;
                    if (leader) {
                        mbar_expect_relaxed(&full_bar[stage], 2 * P::kStageBytes);
                        load_operand<AMN>(&tmA, &full_bar[stage], da, kb, ar, w.batch);
                        load_operand<BMN>(&tmB, &full_bar[stage], db, kb, br, w.batch);
                    } else {
                        load_operand_pair<AMN>(&tmA, full0 + stage * 8, da, kb, ar, w.batch);
                        load_operand_pair<BMN>(&tmB, full0 + stage * 8, db, kb, br, w.batch);
                    }
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // the leader's barriers collect the other CTA's operands too, which leaves no earlier
        if (leader) await_copies(full_bar, S, stage, phase);
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const bool issue = elect_lane();
            const uint64_t a0 = operand_desc<AMN>(a_s), b0 = operand_desc<BMN>(b_s);
            int stage = 0, it = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (; ok && t < args.tiles; t += workers, ++it) {
                const int buf = it & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[buf], ((it >> 1) & 1) ^ 1u, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                for (int kb = 0; kb < args.kblocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t ad = a0 + stage * (P::kOpBytes >> 4), bd = b0 + stage * (P::kOpBytes >> 4);
                    if (issue) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma_bf16_pair(tmem_base + buf * 256, ad + j * kOperandStep<AMN>, bd + j * kOperandStep<BMN>,
                                           idesc_f16_f32(256, 256, AMN, BMN), (kb > 0 || j > 0) ? 1u : 0u);
                        umma_commit_pair(&empty_bar[stage], 3);
                    }
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (issue) umma_commit_pair(&accf_bar[buf], 3);
                __syncwarp();
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, part = (warp - 2) >> 2, ew = warp - 2;
        constexpr int CC = P::kCols;
        const uint32_t acce0 = mapa_shared(smem_u32(&acce_bar[0]), 0);
        uint8_t *st = staging + ew * P::kWarpStaging;
        NsEpilogue<OP, CC> epi = {args, NsMapRefs(maps), st, st + P::kWarpStaging / 2, &aux_bar[ew], abort_flag, lane, 0};
        auto place = [&](const NsTile &x, int &row, int &col) { row = x.m0 + static_cast<int>(rank) * 128 + 32 * q, col = x.n0 + 64 * part; };
        int it = 0, row, col;
        if (t < args.tiles) {
            place(w, row, col);
            epi.load(w, row, col);
        }
        while (t < args.tiles) {
            place(w, row, col);
            const int buf = it & 1;
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * 256 + 64 * part;
            bool ok = __all_sync(0xffffffffu, mbar_wait(&accf_bar[buf], (it >> 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                float v[CC];
                ns_accumulators(t_row + CC * c, v);
                if (c == 1) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive_relaxed(&acce_bar[buf]);
                        else mbar_arrive_cluster_relaxed(acce0 + buf * 8);
                    }
                }
                ok = epi.finish(w, row, col + CC * c, v);
                if (!ok) break;
                if (c == 0) epi.load(w, row, col + CC);
            }
            if (!ok) break;
            next();
            ++it;
            if (t < args.tiles) {
                place(w, row, col);
                epi.load(w, row, col);
            }
        }
        if (lane == 0) {
            bulk_wait_group<0>();
            if (*abort_flag) mbar_drain(&aux_bar[ew], epi.phase);   // a load may still be on its way
        }
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the pair's MMAs may touch it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ------------------------------------------------------------------- ns_fused

// All steps of a small matrix in one launch: a cluster of up to eight CTAs a matrix, whose products
// follow one another between cluster barriers instead of launches (256 x 256, five steps: 51 us, 58 by launches).
// A product's tiles are dealt out to the CTAs; between products everything goes through L2, by
// the copies of the asynchronous proxy on both sides (but the diagonal's remainders).
struct NsFusedArgs {
    int m, rows, cols;                 // the short side; X
    int x_pitch, g_pitch;
    int steps;
    float *diag;
    uint16_t *o;                       // NULL: the last X stays in x[steps & 1]
    float sx;
    float coef[MLPBLK_ORTHO_MAX_STEPS][3];
};
// Operands (K-major, MN-major) and chunks of the epilogue.
struct NsFusedMaps {
    CUtensorMap x_k[2], x_mn[2], g, p;
    CUtensorMap x_chunk[2], lo_chunk, g_chunk, p_chunk, o_chunk;
};

constexpr int kFusedCtas = 8;          // of a cluster, at most

struct NsFused {
    using C = NsSmall<false, 64>;
    uint8_t *a_s, *b_s, *staging;
    uint64_t *full_bar, *empty_bar, *accf_bar, *acce_bar, *aux_bar;
    volatile int *abort;
    uint32_t tmem;
    int warp, lane, rank, ctas;
    int stage = 0, it = 0;             // of this warp's role, through all products
    uint32_t phase = 0;                // an epilogue warp: of its loads

    // One product of the cluster.
    template <int OP, bool AMN, bool BMN>
    __device__ __forceinline__ void product(const CUtensorMap *mA, const CUtensorMap *mB, const NsMapRefs &maps, const NsArgs &a, int batch) {
        constexpr int S = C::kStages;
        const int tiles = a.mt * a.nt;
        int t = rank;
        auto tile = [&]() {
            NsTile w = {};
            w.batch = batch;
            w.m0 = t % a.mt * 128;
            w.n0 = t / a.mt * C::BN;
            return w;
        };
        if (warp == 0) {
            const bool issue = elect_lane();
            if (issue) fence_proxy_async_global();
            bool ok = true;
            for (; ok && t < tiles; t += ctas) {
                const NsTile w = tile();
                for (int kb = 0; kb < a.kblocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort));
                    if (!ok) break;
                    if (issue) {
                        mbar_expect_relaxed(&full_bar[stage], C::kStageBytes);
                        load_operand<AMN, 128, C::BN>(mA, &full_bar[stage], a_s + stage * C::kABytes, kb, w.m0, batch);
                        load_operand<BMN, C::BN, C::BN>(mB, &full_bar[stage], b_s + stage * C::kBBytes, kb, w.n0, batch);
                    }
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp == 1) {
            const bool issue = elect_lane();
            const uint64_t a0 = operand_desc<AMN>(a_s), b0 = operand_desc<BMN>(b_s);
            bool ok = true;
            for (; ok && t < tiles; t += ctas, ++it) {
                const int buf = it & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[buf], ((it >> 1) & 1) ^ 1u, abort));
                if (!ok) break;
                tc_fence_after_sync();
                for (int kb = 0; kb < a.kblocks; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t ad = a0 + stage * (C::kABytes >> 4), bd = b0 + stage * (C::kBBytes >> 4);
                    if (issue) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma_bf16(tmem + buf * C::BN, ad + j * kOperandStep<AMN>, bd + j * kOperandStep<BMN>,
                                      idesc_f16_f32(128, C::BN, AMN, BMN), (kb > 0 || j > 0) ? 1u : 0u);
                        umma_commit(&empty_bar[stage]);
                    }
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (issue) umma_commit(&accf_bar[buf]);
                __syncwarp();
            }
        } else {
            const int q = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
            uint8_t *st = staging + ew * kNsStaging;
            NsEpilogue<OP, C::kCols> epi = {a, maps, st, st + kNsChunkBytes, &aux_bar[ew], abort, lane, phase};
            if (lane == 0) fence_proxy_async_global();
            if (t < tiles) epi.load(tile(), t % a.mt * 128 + 32 * q, t / a.mt * C::BN + C::kCols * half);
            while (t < tiles) {
                const NsTile w = tile();
                const int buf = it & 1;
                const bool ok = __all_sync(0xffffffffu, mbar_wait(&accf_bar[buf], (it >> 1) & 1, abort));
                if (!ok) break;
                tc_fence_after_sync();
                float v[C::kCols];
                ns_accumulators(tmem + (static_cast<uint32_t>(32 * q) << 16) + buf * C::BN + C::kCols * half, v);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(&acce_bar[buf]);
                if (!epi.finish(w, w.m0 + 32 * q, w.n0 + C::kCols * half, v)) break;
                t += ctas;
                ++it;
                if (t < tiles) epi.load(tile(), t % a.mt * 128 + 32 * q, t / a.mt * C::BN + C::kCols * half);
            }
            if (lane == 0) {
                bulk_wait_group<0>();
                if (*abort) mbar_drain(&aux_bar[ew], epi.phase);   // a load may still be on its way
            }
            __syncwarp();
            phase = epi.phase;
        }
        cluster_sync();
    }
};

template <bool TALL>
__global__ void __launch_bounds__(NsFused::C::kThreads, 1)
ns_fused_kernel(const __grid_constant__ NsFusedMaps maps, const __grid_constant__ NsFusedArgs args) {
    using C = NsSmall<false, 64>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    NsFused f;
    f.a_s = smem;
    f.b_s = f.a_s + S * C::kABytes;
    f.staging = f.b_s + S * C::kBBytes;
    uint8_t *ctrl = f.staging + C::kDumpBytes;
    f.full_bar = reinterpret_cast<uint64_t *>(ctrl);
    f.empty_bar = f.full_bar + S;
    f.accf_bar = f.empty_bar + S;
    f.acce_bar = f.accf_bar + 2;
    f.aux_bar = f.acce_bar + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 512);
    f.abort = reinterpret_cast<volatile int *>(ctrl + 516);
    f.warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    f.lane = threadIdx.x & 31;
    f.rank = static_cast<int>(cluster_ctarank());
    f.ctas = static_cast<int>(cluster_nctarank());
    const int batch = static_cast<int>(blockIdx.x) / f.ctas;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&f.full_bar[s], 1);
            mbar_init(&f.empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&f.accf_bar[b], 1);
            mbar_init(&f.acce_bar[b], C::kEpiWarps);
        }
        for (int b = 0; b < C::kEpiWarps; ++b) mbar_init(&f.aux_bar[b], 1);
        *f.abort = 0;
        fence_barrier_init();
        for (int i = 0; i < 2; ++i) {
            prefetch_tensormap(&maps.x_k[i]);
            prefetch_tensormap(&maps.x_mn[i]);
            prefetch_tensormap(&maps.x_chunk[i]);
        }
        prefetch_tensormap(&maps.g);
        prefetch_tensormap(&maps.p);
        prefetch_tensormap(&maps.g_chunk);
        prefetch_tensormap(&maps.p_chunk);
        prefetch_tensormap(&maps.lo_chunk);
    }
    if (f.warp == 1) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    f.tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();

    NsArgs sq = {};                    // G and P
    sq.rows = sq.cols = args.m;
    sq.mt = (args.m + 127) / 128;
    sq.nt = (args.m + C::BN - 1) / C::BN;
    sq.diag_pitch = args.g_pitch;
    sq.diag = sq.diag_out = args.diag;
    sq.alpha = 1.0f / (args.sx * args.sx);
    NsArgs up = {};                    // X
    up.rows = args.rows;
    up.cols = args.cols;
    up.mt = (args.rows + 127) / 128;
    up.nt = (args.cols + C::BN - 1) / C::BN;
    up.diag_pitch = args.g_pitch;
    up.diag = args.diag;
    up.diag_col = TALL;
    up.o_tma = args.cols % 8 == 0;
    up.alpha = 1.0f / args.sx;
    const int n_blocks = ((TALL ? args.rows : args.cols) + kNsK - 1) / kNsK, m_blocks = (args.m + kNsK - 1) / kNsK;
    // (what is set but not read by an epilogue only has to be there)
    NsMapRefs to_g, to_p, to_x;
    to_g.aux = to_g.aux2 = to_g.out_lo = to_g.mirror = nullptr;
    to_g.out = &maps.g_chunk;
    to_p = to_g;
    to_p.aux = &maps.g_chunk;
    to_p.out = &maps.p_chunk;
    to_x = to_g;
    to_x.aux2 = to_x.out_lo = &maps.lo_chunk;
    __half *const some = reinterpret_cast<__half *>(args.diag);
#pragma unroll 1
    for (int i = 0; i < args.steps; ++i) {
        const int from = i & 1;
        sq.kblocks = n_blocks;
        if (TALL) f.product<kNsGram, true, true>(&maps.x_mn[from], &maps.x_mn[from], to_g, sq, batch);
        else f.product<kNsGram, false, false>(&maps.x_k[from], &maps.x_k[from], to_g, sq, batch);
        sq.kblocks = m_blocks;
        sq.b = args.coef[i][1];
        sq.c = args.coef[i][2];
        f.product<kNsSquare, false, false>(&maps.g, &maps.g, to_p, sq, batch);
        const bool last = i + 1 == args.steps;
        up.kblocks = m_blocks;
        up.a = args.coef[i][0];
        up.aux2 = last ? nullptr : some;                  // there are low parts (the map says where)
        up.out_lo = i + 2 < args.steps ? some : nullptr;
        up.o = last ? args.o : nullptr;
        to_x.aux = &maps.x_chunk[from];
        to_x.out = up.o ? &maps.o_chunk : &maps.x_chunk[from ^ 1];
        if (TALL) f.product<kNsUpdate, false, false>(&maps.x_k[from], &maps.p, to_x, up, batch);
        else f.product<kNsUpdate, false, true>(&maps.p, &maps.x_mn[from], to_x, up, batch);
    }
    if (f.warp == 0) {
        await_copies(f.full_bar, S, f.stage, f.phase);
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (f.warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(f.tmem, 256);
    }
}

// ------------------------------------------------------------------------ host

// A batch of fp16 matrices [rows][cols], rows of `pitch` elements.  K-major: boxes of 64
// columns x 128 (or 64) rows.  MN-major: K runs over the rows; a box is 64 rows of two blocks (or
// one) of 64 columns (the map's third dimension walks the blocks, up to the pitch).
bool ns_map(CUtensorMap *m, const __half *p, bool mn, int64_t rows, int64_t cols, int64_t pitch, int batch, uint32_t box_rows = 128) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t R = static_cast<cuuint64_t>(rows), line = static_cast<cuuint64_t>(pitch) * 2, B = static_cast<cuuint64_t>(batch);
    cuuint32_t estr[4] = {1, 1, 1, 1};
    if (mn) {
        cuuint64_t dims[4] = {64, R, static_cast<cuuint64_t>(pitch / 64), B};
        cuuint64_t strides[3] = {line, 128, R * line};
        cuuint32_t box[4] = {64, kNsK, box_rows / 64, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<__half *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), R, B};
    cuuint64_t strides[2] = {line, R * line};
    cuuint32_t box[3] = {kNsK, box_rows, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of `box_cols` (64 or 32) x `box_rows` for the epilogue, of 16-bit values (fp16, or o's bf16); a mirror
// image's are not swizzled.
bool ns_chunk_map(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t pitch, int batch, uint32_t box_cols, uint32_t box_rows, bool swizzle = true) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t line = static_cast<cuuint64_t>(pitch) * 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[2] = {line, line * dims[1]};
    cuuint32_t box[3] = {box_cols, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? (box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps that the epilogue of `a` uses, in chunks of `cols` columns.
bool ns_epilogue_maps(NsMaps *m, const NsArgs &a, int batch, uint32_t cols = 64) {
    bool ok = true;
    if (a.aux) ok &= ns_chunk_map(&m->aux, a.aux, a.rows, a.cols, a.pitch, batch, cols, 32);
    if (a.aux2) ok &= ns_chunk_map(&m->aux2, a.aux2, a.rows, a.cols, a.pitch, batch, cols, 32);
    if (a.o) {
        if (a.o_tma) ok &= ns_chunk_map(&m->out, a.o, a.rows, a.cols, a.cols, batch, cols, 32);
    } else {
        ok &= ns_chunk_map(&m->out, a.out, a.rows, a.cols, a.pitch, batch, cols, 32);
        if (a.out_lo) ok &= ns_chunk_map(&m->out_lo, a.out_lo, a.rows, a.cols, a.pitch, batch, cols, 32);
    }
    if (a.op != kNsUpdate) ok &= ns_chunk_map(&m->mirror, a.out, a.rows, a.cols, a.pitch, batch, 32, cols, false);
    return ok;
}

// Cluster size 1: no cluster attribute.
template <class K>
int launch_ns(K kernel, int threads, int smem, int grid, int cluster, const CUtensorMap &mA, const CUtensorMap &mB, const NsMaps &maps,
              const NsArgs &a, int *attr_set, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    if (!attr_set[dev]) {
        const int rc = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        if (rc != MLPBLK_OK) return rc;
        attr_set[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, mA, mB, maps, a));
}

int64_t tiles_of(const NsArgs &a, int ts, bool sym) {
    const int64_t mt = (a.rows + ts - 1) / ts, nt = (a.cols + ts - 1) / ts;
    return sym ? mt * (mt + 1) / 2 : mt * nt;
}

// One operand: a batch of matrices as they lie.
struct NsOperand {
    const __half *p;
    int64_t rows, cols;
};

template <int OP, bool AMN, bool BMN>
int run_ns(NsArgs a, const NsOperand &A, const NsOperand &B, int batch, int sms, cudaStream_t s) {
    constexpr bool SYM = OP != kNsUpdate;
    const int64_t pair_tiles = tiles_of(a, 256, SYM) * batch, tiles = tiles_of(a, 128, SYM) * batch;
    const int pairs = sms / 2;
    if (tiles > INT32_MAX) return MLPBLK_EINVAL;
    NsMaps maps = {};
    CUtensorMap mA, mB;
    auto operands = [&](uint32_t box) {
        return ns_map(&mA, A.p, AMN, A.rows, A.cols, ortho_pitch(A.cols), batch, box) && ns_map(&mB, B.p, BMN, B.rows, B.cols, ortho_pitch(B.cols), batch, box);
    };
    // Rounds of tiles, each with its stages of K and the part of its epilogue that nothing hides (us,
    // measured): a pair's 256 x 256 tile 0.3 a stage and 2.4, and 4.5 for the clusters' start and last epilogue, a CTA's
    // 128 x 128 one 0.22 and 2.2.  (X X^T of 8 x 1024 x 2048: 80 pair tiles on 76 pairs 31 us, 288
    // small ones 23; X' 39 and 45.  16 x 512 x 512: 14 and 12; 3 x 1300 x 1300: 17 and 18, X' 27 and 23.)
    const int64_t pair_rounds = pairs >= 1 ? (pair_tiles + pairs - 1) / pairs : 0, rounds = (tiles + sms - 1) / sms;
    if (pairs >= 1 && 4.5 + pair_rounds * (0.3 * a.kblocks + 2.4) < rounds * (0.22 * a.kblocks + 2.2)) {
        static int attr_set[64] = {0};
        a.mt = (a.rows + 255) / 256;
        a.nt = (a.cols + 255) / 256;
        a.per = static_cast<int>(pair_tiles / batch);
        a.tiles = static_cast<int>(pair_tiles);
        a.group_m = 8;
        const int workers = a.tiles < pairs ? a.tiles : pairs;
        if (!operands(128) || !ns_epilogue_maps(&maps, a, batch, NsPair::kCols)) return MLPBLK_ECUDA;
        return launch_ns(ns_pair_kernel<OP, AMN, BMN>, NsPair::kThreads, NsPair::kSmemBytes, 2 * workers, 2, mA, mB, maps, a, attr_set, s);
    }
    a.mt = (a.rows + 127) / 128;
    a.nt = (a.cols + 127) / 128;
    a.group_m = 8;
    if constexpr (OP == kNsGram) {
        const int64_t every = static_cast<int64_t>(a.mt) * a.nt * batch;   // a split computes the images too
        // K is split where that saves more than the cluster's sum costs: a stage takes 0.155 us with
        // few CTAs at work, the sum some 5.5 and 0.3 a part (X X^T of 256 x 8192: 27.2 us whole, 22.4, 17.9 and 18.0
        // in two, four and eight; of 512 x 2048: 13.0, 14.3, 14.3, 25.6).  Clusters of eight find room on some two thirds
        // of the SMs at once (500 x 16000, sixteen tiles: 31 us in eight, 19.5 in four).  The other products' K is the
        // short side: where it has the 58 stages that this takes, there are hundreds of tiles.
        int split = 1;
        double best = 0.155 * a.kblocks;
        for (int k = 2; k <= 8; k *= 2) {
            const double cost = 0.155 * a.kblocks / k + 5.5 + 0.3 * k;
            if (every * k <= (k == 8 ? sms * 2 / 3 : sms * 5 / 6) && a.kblocks >= 2 * k && cost < best) best = cost, split = k;
        }
        if (split > 1) {
            a.per = a.mt * a.nt;
            a.tiles = static_cast<int>(every);
            if (!operands(128)) return MLPBLK_ECUDA;
            static int attr_set[64] = {0};
            return launch_ns(ns_small_kernel<NsSmall<true>, OP, AMN, BMN>, NsSmall<true>::kThreads, NsSmall<true>::kSmemBytes, a.tiles * split,
                             split, mA, mB, maps, a, attr_set, s);
        }
    }
    // Tiles of 64 columns where they fit in one round: half the MMAs and half the epilogue of each (five
    // steps of 512 x 512 65 us, 97 by 128 columns; 250 x 2000 76 and 104).
    const int64_t halves = static_cast<int64_t>(a.mt) * ((a.cols + 63) / 64) * batch;
    if (halves <= sms) {
        using C = NsSmall<false, 64>;
        a.nt = (a.cols + 63) / 64;
        a.per = a.mt * a.nt;
        a.tiles = static_cast<int>(halves);
        if (!operands(64) || !ns_epilogue_maps(&maps, a, batch, C::kCols)) return MLPBLK_ECUDA;
        static int attr_set[64] = {0};
        return launch_ns(ns_small_kernel<C, OP, AMN, BMN>, C::kThreads, C::kSmemBytes, a.tiles, 1, mA, mB, maps, a, attr_set, s);
    }
    a.per = static_cast<int>(tiles / batch);
    a.tiles = static_cast<int>(tiles);
    if (!operands(128) || !ns_epilogue_maps(&maps, a, batch)) return MLPBLK_ECUDA;
    static int attr_set[64] = {0};
    return launch_ns(ns_small_kernel<NsSmall<false>, OP, AMN, BMN>, NsSmall<false>::kThreads, NsSmall<false>::kSmemBytes, a.tiles < sms ? a.tiles : sms, 1,
                     mA, mB, maps, a, attr_set, s);
}

}  // namespace

int launch_ns_product(const NsProduct &p, int sms, cudaStream_t s) {
    const int64_t m = p.tall ? p.cols : p.rows;   // the short side
    const int64_t x_pitch = ortho_pitch(p.cols), g_pitch = ortho_pitch(m);
    NsArgs a = {};
    a.op = p.op;
    a.alpha = p.alpha;
    a.a = p.a;
    a.b = p.b;
    a.c = p.c;
    a.diag = p.diag;
    a.diag2 = p.diag2;
    a.diag_out = p.diag_out;
    a.diag_pitch = static_cast<int>(g_pitch);
    a.out = p.out;
    a.out_lo = p.out_lo;
    a.o = static_cast<uint16_t *>(p.o);
    a.o_tma = p.cols % 8 == 0;
    a.kblocks = static_cast<int>((m + kNsK - 1) / kNsK);
    const NsOperand X = {p.x, p.rows, p.cols}, Y = {p.y, m, m}, P = {p.p, m, m};
    if (p.op == kNsUpdate) {
        a.rows = static_cast<int>(p.rows);
        a.cols = static_cast<int>(p.cols);
        a.pitch = static_cast<int>(x_pitch);
        a.matrix = p.rows * x_pitch;
        a.aux = p.x;
        a.aux2 = p.x_lo;
        a.diag_col = p.tall;
        return p.tall ? run_ns<kNsUpdate, false, false>(a, X, P, p.batch, sms, s) : run_ns<kNsUpdate, false, true>(a, P, X, p.batch, sms, s);
    }
    a.rows = a.cols = static_cast<int>(m);
    a.pitch = static_cast<int>(g_pitch);
    a.matrix = m * g_pitch;
    if (p.op == kNsGram) {
        const int64_t n = p.tall ? p.rows : p.cols;
        a.kblocks = static_cast<int>((n + kNsK - 1) / kNsK);
        return p.tall ? run_ns<kNsGram, true, true>(a, X, X, p.batch, sms, s) : run_ns<kNsGram, false, false>(a, X, X, p.batch, sms, s);
    }
    a.aux = p.y;
    if (p.op == kNsJoin) a.aux2 = p.p;
    if (p.op == kNsSquare) return run_ns<kNsSquare, false, false>(a, Y, Y, p.batch, sms, s);
    if (p.op == kNsApply) return run_ns<kNsApply, false, false>(a, P, Y, p.batch, sms, s);
    return run_ns<kNsJoin, false, false>(a, P, Y, p.batch, sms, s);
}

// CTAs of a matrix: one a tile of X, up to eight.
static int ns_fused_ctas(int64_t rows, int64_t cols) {
    const int64_t tiles = (rows + 127) / 128 * ((cols + NsFused::C::BN - 1) / NsFused::C::BN);
    int c = 1;
    while (c < kFusedCtas && c < tiles) c *= 2;
    return c;
}

// One launch where a CTA has one tile of X and all matrices run at once; clusters of more than two
// CTAs find room for some two thirds of the SMs (us, one launch and several: 256 x 256 51 and 58, 128 x 512
// 50 and 56, 200 x 400 60 and 60, 250 x 1000 79 and 67; 12 of 256 x 256 54 and 61, 16 100 and 64).
bool ns_fused_fits(int64_t rows, int64_t cols, int batch, int sms) {
    const int64_t tiles = (rows + 127) / 128 * ((cols + NsFused::C::BN - 1) / NsFused::C::BN);
    const int64_t ctas = static_cast<int64_t>(batch) * ns_fused_ctas(rows, cols);
    return tiles <= kFusedCtas && ctas <= (tiles <= 2 ? sms : sms * 2 / 3);
}

int launch_ns_fused(const NsFusedProblem &p, cudaStream_t s) {
    const bool tall = p.rows > p.cols;
    const int64_t m = tall ? p.cols : p.rows, x_pitch = ortho_pitch(p.cols), g_pitch = ortho_pitch(m);
    NsFusedArgs a = {};
    a.m = static_cast<int>(m);
    a.rows = static_cast<int>(p.rows);
    a.cols = static_cast<int>(p.cols);
    a.x_pitch = static_cast<int>(x_pitch);
    a.g_pitch = static_cast<int>(g_pitch);
    a.steps = p.steps;
    a.diag = p.diag;
    a.o = static_cast<uint16_t *>(p.o);
    a.sx = p.sx;
    for (int i = 0; i < p.steps; ++i)
        for (int j = 0; j < 3; ++j) a.coef[i][j] = p.coefficients[i][j];
    NsFusedMaps maps = {};
    bool ok = ns_map(&maps.g, p.g, false, m, m, g_pitch, p.batch, NsFused::C::BN) && ns_map(&maps.p, p.p, false, m, m, g_pitch, p.batch, NsFused::C::BN) &&
              ns_chunk_map(&maps.g_chunk, p.g, m, m, g_pitch, p.batch, NsFused::C::kCols, 32) && ns_chunk_map(&maps.p_chunk, p.p, m, m, g_pitch, p.batch, NsFused::C::kCols, 32) &&
              ns_chunk_map(&maps.lo_chunk, p.lo, p.rows, p.cols, x_pitch, p.batch, NsFused::C::kCols, 32);
    if (p.o && p.cols % 8 == 0) ok = ok && ns_chunk_map(&maps.o_chunk, p.o, p.rows, p.cols, p.cols, p.batch, NsFused::C::kCols, 32);
    for (int i = 0; i < 2; ++i)
        ok = ok && ns_map(&maps.x_k[i], p.x[i], false, p.rows, p.cols, x_pitch, p.batch, NsFused::C::BN) && ns_map(&maps.x_mn[i], p.x[i], true, p.rows, p.cols, x_pitch, p.batch, NsFused::C::BN) &&
             ns_chunk_map(&maps.x_chunk[i], p.x[i], p.rows, p.cols, x_pitch, p.batch, NsFused::C::kCols, 32);
    if (!ok) return MLPBLK_ECUDA;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    static int attr_set[2][64] = {};
    void (*const kernel)(NsFusedMaps, NsFusedArgs) = tall ? ns_fused_kernel<true> : ns_fused_kernel<false>;
    if (!attr_set[tall][dev]) {
        const int rc = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NsFused::C::kSmemBytes));
        if (rc != MLPBLK_OK) return rc;
        attr_set[tall][dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    const int ctas = ns_fused_ctas(p.rows, p.cols);
    cfg.gridDim = dim3(static_cast<unsigned>(p.batch * ctas));
    cfg.blockDim = dim3(NsFused::C::kThreads);
    cfg.dynamicSmemBytes = NsFused::C::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, maps, a));
}

int take_device_error_gemm_ns() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return MLPBLK_ECUDA;
    if (v != 0) cudaMemcpyToSymbol(g_device_error, &z, sizeof(int));
    return v;
}

}  // namespace mlpblk
