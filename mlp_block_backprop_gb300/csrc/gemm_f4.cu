// gemm_f4.cu -- products of MXFP4 matrices, C[m,n] = A[m,k] . B[n,k]^T, on the tensor
// cores' block-scaled path (tcgen05.mma kind::mxf4: E2M1 operands, one E8M0 scale
// per 32 values of K, fp32 accumulator in TMEM).
//
// A stage row is 128 bytes, 256 values of K, in the 128-byte swizzle; one MMA takes
// 32 bytes (64 values) of it.  The scales lie in global memory in the order in which
// tcgen05.cp wants them (include/mlpblk.h: 512-byte tiles of 128 rows x 128 values
// of K).  In TMEM a tile is four columns, lane l of column j holding the scales of row
// 32j + l, the same in all four lane quarters: four warps read a stage's tiles from
// shared memory, 16 bytes a lane, and store them with tcgen05.st, one quarter each.
// tcgen05.cp would do it without them, but it runs in the MMAs' pipe (8192 x 16384 x
// 4096: 226 us with it, 172 without; one token x 16384 x 4096: 10.5 us and 8.9).
//
// f4_small: one CTA computes a 128 x 128 tile with B's rows (C's columns) on the 128
//   lanes and A's rows (tokens) on the columns, so that few tokens cost few
//   columns (32 or 64): at one token the kernel streams the weights.  C leaves straight from
//   registers: 32 lanes are 32 consecutive elements of a row of C, whatever n is.
//   K can be split over a cluster; the parts meet in distributed shared memory and
//   are added in rank order.
// f4_pair: two CTAs on two SMs compute a 256 x 256 tile (cta_group::2), A's rows on the
//   lanes; each CTA stages 128 rows of A and of B, and the scales of its A rows and
//   of all 256 columns.
#include <limits.h>

#include <type_traits>

#include "fp4_layout.h"
#include "gemm_tc.cuh"

namespace mlpblk {

namespace {

constexpr int kF4MaxExperts = 256;
constexpr int kF4KB = 256;              // K values of a stage
constexpr int kF4PrefetchStages = 8;    // stages of B that f4_small asks into L2 ahead (136 KB a CTA)

struct F4Args {
    int mode;                           // Fp4Mode
    int64_t m, n;                       // C (per expert when K-grouped)
    int mt, nt;                         // tiles along m (but when grouped by rows) and n
    int kblocks;                        // stages along all of K
    int experts;
    int64_t max_rows;
    const uint8_t *sa, *sb;             // scales
    int64_t row_tile_bytes;             // of one 128-row strip of scale tiles (A and B share K)
    int group_m;                        // raster: this many tiles of A sweep B together
    const int *count, *seg;
    void *c;
};

// ------------------------------------------------------------------------- PTX

// Instruction descriptor of kind::mxf4: E2M1 A and B (code 1), E8M0 scales, K = 64;
// the scale ids (0 or 2) say which two of a TMEM word's four scale bytes an MMA reads.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf) {
    return (static_cast<uint32_t>(sf) << 4)           // B scale id
           | (1u << 7) | (1u << 10)                    // A, B: E2M1
           | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
           | (1u << 23)                                // scales: E8M0
           | (static_cast<uint32_t>(M >> 7) << 27)     // M / 128
           | (static_cast<uint32_t>(sf) << 29);        // A scale id
}

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  setp.ne.b32 p, %6, 0;\n"
        "  tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// Four columns of scales of this warp's lane quarter from registers.
__device__ __forceinline__ void tmem_store_4cols(uint32_t taddr, uint4 v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of the warp, the same one each time.  The roles that issue copies and MMAs
// run their loops with the whole warp and let this lane issue: addresses and
// descriptors are then warp-uniform and live in uniform registers.  With the loop
// inside `if (lane == 0)` every operand crosses from vector registers, and a stage cost
// the issuing thread some 680 cycles, more than its MMAs take.
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

// mbar_arrive_expect_tx without its release: the producer's own accesses need no
// ordering (the copies it issues signal the barrier by themselves).
__device__ __forceinline__ void mbar_expect_relaxed(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

// Asks L2 to fetch a box of a 2-D tensor map.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1)
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

// Before a producer leaves: waits for the copies that it issued into the S stages, the next
// of which would be `stage` in phase `phase`.  A run that went well finds them landed; one
// that gave up must not leave while a copy may still write its shared memory.  Bounded over
// all stages together.
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

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// ------------------------------------------------------------------- the work

// The experts' segments in shared memory and the tiles before each expert.
struct F4Groups {
    int seg[kF4MaxExperts + 1];
    int count[kF4MaxExperts];
    int before[kF4MaxExperts + 1];
    int warp_tiles[kF4MaxExperts / 32];
};

// One output tile: rows m0 .. m0 + m_valid of A, columns n0 .. n0 + n_valid of C.
struct F4Tile {
    int a_row, b_row;          // rows of the code matrices (TMA coordinates)
    const uint8_t *sa, *sb;    // scale tiles of those rows at k-block 0
    int kb0, kb1;              // k-blocks
    int sa_tile, sb_tile;      // the same as row indices of the scale arrays
    int64_t c_row;             // C's row of the tile's first A row, counted through all of C
    int c_local, c_mat;        // the same as a row of one matrix of C, and which
    int n0, m_valid, n_valid;
};

// Tiles of TM rows that `rows` take (up to 2^31 - 1: the sum needs 32 unsigned bits).
template <int TM>
__device__ __forceinline__ int f4_row_tiles(int rows) {
    return static_cast<int>((static_cast<unsigned>(rows) + (TM - 1)) / TM);
}

// Fills `g` (the whole CTA, a thread an expert) for tiles of TM rows; returns the number
// of tiles.  Values that a plan of another shape would give are cut to the arrays, so
// no access leaves them.
template <int TM>
__device__ __forceinline__ int f4_groups(const F4Args &a, F4Groups *g) {
    const int e = static_cast<int>(threadIdx.x), lane = e & 31, warp = e >> 5;
    // (whole stages of the largest K end at 2^31, behind what a segment can name)
    const int limit = static_cast<int>(a.mode == kFp4GroupRows ? a.m : min(static_cast<int64_t>(a.kblocks) * kF4KB, static_cast<int64_t>(INT_MAX)));
    int tiles = 0;
    if (e < a.experts) {
        const int s0 = min(max(a.seg[e], 0), limit), s1 = min(max(a.seg[e + 1], 0), limit);
        g->seg[e] = s0;
        if (e == a.experts - 1) g->seg[a.experts] = s1;
        if (a.mode == kFp4GroupRows) {
            int c = max(min(a.count[e], s1 - s0), 0);
            if (a.max_rows > 0) c = static_cast<int>(min(static_cast<int64_t>(c), a.max_rows));
            g->count[e] = c;
            tiles = f4_row_tiles<TM>(c) * a.nt;
        } else {
            tiles = a.mt * a.nt;
        }
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (warp < kF4MaxExperts / 32 && lane == 31) g->warp_tiles[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int v = 0; v < kF4MaxExperts / 32; ++v) {
        const int c = v * 32 < a.experts ? g->warp_tiles[v] : 0;
        before += v < warp ? c : 0;
        all += c;
    }
    if (e < a.experts) g->before[e] = before + incl - tiles;
    if (e == 0) g->before[a.experts] = all;
    __syncthreads();
    return all;
}

// Tile t.  Dense tiles are rastered with A's tiles fastest within a group of
// group_m (raster_tile); an expert's likewise over its own rows.
template <int TM, int TN>
__device__ __forceinline__ F4Tile f4_tile(const F4Args &a, const F4Groups *g, int t, int group_m) {
    F4Tile w;
    int e = 0;
    if (a.mode != kFp4Dense) {
        int lo = 0, hi = a.experts;  // before[lo] <= t < before[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (g->before[mid] <= t) lo = mid;
            else hi = mid;
        }
        e = lo;
        t -= g->before[e];
    }
    const int rows = a.mode == kFp4GroupRows ? g->count[e] : static_cast<int>(a.m);
    int mi = 0, ni = 0;
    const int mt = f4_row_tiles<TM>(rows);
    if (mt == 1) ni = t;
    else raster_tile(t, mt, a.nt, group_m, mi, ni);
    const int first = a.mode == kFp4GroupRows ? g->seg[e] : 0;
    w.a_row = first + mi * TM;
    w.n0 = ni * TN;
    w.b_row = (a.mode == kFp4GroupRows ? e * static_cast<int>(a.n) : 0) + w.n0;
    w.sa_tile = w.a_row / 128;
    w.sb_tile = (a.mode == kFp4GroupRows ? e * static_cast<int>((a.n + 127) / 128) : 0) + w.n0 / 128;
    w.sa = a.sa + w.sa_tile * a.row_tile_bytes;
    w.sb = a.sb + w.sb_tile * a.row_tile_bytes;
    w.kb0 = 0;
    w.kb1 = a.kblocks;
    w.c_row = w.c_local = w.a_row;
    w.c_mat = 0;
    if (a.mode == kFp4GroupK) {
        w.c_mat = e;
        w.kb0 = g->seg[e] / kF4KB;
        w.kb1 = g->seg[e + 1] / kF4KB;
        w.c_row += e * a.m;
    }
    w.m_valid = min(TM, rows - mi * TM);
    w.n_valid = static_cast<int>(min(static_cast<int64_t>(TN), a.n - w.n0));
    return w;
}

// ------------------------------------------------------------------- f4_small

// 128 columns: a tile that has 32 or 64 rows of A at most loads and multiplies no more (a
// kernel with 32 columns and two CTAs an SM, four stages each, was slower everywhere: one
// token x 16384 x 4096 7.8 us and 6.1, 8 x 2048 x 2048 4.6 and 3.2).  SPLIT: K is split
// over a cluster, whose sum takes shared memory from the stages.
template <bool SPLIT_>
struct F4Small {
    static constexpr int BN = 128;
    static constexpr bool SPLIT = SPLIT_;
    static constexpr int kEpiWarps = 8;            // two a lane quarter: 64 columns each
    static constexpr int kEpiCols = 64;
    static constexpr int kThreads = 64 + 32 * kEpiWarps + 128 + 32;  // codes, MMA, epilogue, four scale warps, scale loads
    static constexpr int kScaleLoadWarp = kThreads / 32 - 1;
    static constexpr int kLBytes = 128 * 128;      // B's rows, on the lanes
    static constexpr int kRBytes = BN * 128;       // A's rows, on the columns
    static constexpr int kSfBytes = 1024;          // scales of 128 rows and a stage of K
    static constexpr int kStageBytes = kLBytes + kRBytes + 2 * kSfBytes;
    static constexpr int kDumpBytes = SPLIT ? BN * 128 * 4 : 0;  // an fp32 tile, for the cluster's sum
    static constexpr int kCtrlBytes = 4096;
    static constexpr int kStages = (kSmemLimit - 1024 - kCtrlBytes - kDumpBytes) / kStageBytes;
    static constexpr int kSmemBytes = 1024 + kCtrlBytes + kDumpBytes + kStages * kStageBytes;
    // TMEM: two accumulators, then each stage's scales (8 columns each operand)
    static constexpr int kSfCol = 2 * BN;
    static constexpr int kSfSet = 16;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kStages >= 3 && kSfCol + kStages * kSfSet <= 512, "pipeline");
    static_assert(sizeof(F4Groups) + 512 <= kCtrlBytes, "control block");
};

// Columns that a tile's loads and MMAs cover.
__device__ __forceinline__ int f4_width(const F4Tile &w) { return w.m_valid <= 32 ? 32 : (w.m_valid <= 64 ? 64 : 128); }

// 32 columns of a tile out of a lane's registers: column j goes to C's row row0 + j,
// lane i to its column col0 + i; `rows` of the columns and the lanes with `on` are stored.
// OUT: 0 bf16, 1 float32, 2 float32 +=.  bf16 with an even n: neighbouring lanes swap
// every other value, so that a store is a pair of columns.
template <int OUT>
__device__ __forceinline__ void store_columns(void *c, int64_t row0, int64_t n, int64_t col, const float (&v)[32], int rows,
                                              bool on) {
    const int lane = threadIdx.x & 31;
    if (OUT == 0 && (n & 1) == 0) {
        const int odd = lane & 1;
        uint16_t *p = static_cast<uint16_t *>(c) + (row0 + odd) * n + (col - odd);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const uint32_t w = odd ? pack_bf16x2(got, v[j + 1]) : pack_bf16x2(v[j], got);
            if (on && j + odd < rows) *reinterpret_cast<uint32_t *>(p) = w;
            p += 2 * n;
        }
    } else if (OUT == 0) {
        uint16_t *p = static_cast<uint16_t *>(c) + row0 * n + col;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (on && j < rows) *p = static_cast<uint16_t>(pack_bf16x2(v[j], 0.0f) & 0xFFFFu);
            p += n;
        }
    } else {
        float *p = static_cast<float *>(c) + row0 * n + col;
        float old[32];
        if (OUT == 2) {
#pragma unroll
            for (int j = 0; j < 32; ++j) old[j] = on && j < rows ? p[j * n] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (on && j < rows) *p = OUT == 2 ? old[j] + v[j] : v[j];
            p += n;
        }
    }
}

// Asks the first stages of a worker's B into L2 while the previous kernel (A's
// quantisation, as a rule) still runs: no data reaches this kernel before
// griddep_wait.  With few tokens the weights' way from HBM is most of the time: one token x
// 16384 x 4096 with the quantisation before it takes 9.3 us without and 9.2 with eight
// stages asked ahead where the weights are in L2, 25 and 22 alone with its host's calls
// where they are not; 16 stages 9.9 and 23 (L2 drops requests that come faster than it
// fetches).  Where the experts' segments decide the tiles it gained nothing.
template <class C>
__device__ __forceinline__ void f4_prefetch(const F4Args &a, const CUtensorMap *map, const F4Tile &w, int rank, int cs) {
    const int k0 = w.kb1 * rank / cs, k1 = min(w.kb1 * (rank + 1) / cs, k0 + kF4PrefetchStages);
    for (int kb = k0; kb < k1; ++kb) {
        tma_prefetch_2d(map, kb * 128, w.b_row);
        bulk_prefetch_l2(w.sb + static_cast<int64_t>(kb) * C::kSfBytes, C::kSfBytes);
    }
}

template <class C, int OUT>
__global__ void __launch_bounds__(C::kThreads, 1)
f4_small_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                const __grid_constant__ CUtensorMap tmB, const F4Args args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int S = C::kStages;
    uint8_t *lanes_s = smem;                                   // [S][128 rows][128 B]
    uint8_t *cols_s = lanes_s + S * C::kLBytes;                // [S][BN rows][128 B]
    uint8_t *sf_s = cols_s + S * C::kRBytes;                   // [S][2][1 KB]
    float *dump = reinterpret_cast<float *>(sf_s + S * 2 * C::kSfBytes);  // [BN][128]
    uint8_t *ctrl = reinterpret_cast<uint8_t *>(dump) + C::kDumpBytes;
    uint64_t *full_bar = reinterpret_cast<uint64_t *>(ctrl);
    uint64_t *empty_bar = full_bar + S;
    uint64_t *sf_bar = empty_bar + S;     // the stage's scales are in shared memory
    uint64_t *accf_bar = sf_bar + S;
    uint64_t *acce_bar = accf_bar + 2;
    uint64_t *part_full = acce_bar + 2;   // every CTA of the cluster has its part in `dump`
    uint64_t *part_empty = part_full + 1; // every CTA has read this CTA's part
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 384);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 388);
    F4Groups *groups = reinterpret_cast<F4Groups *>(ctrl + 512);
    static_assert((3 * S + 6) * 8 <= 384, "barriers");

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int cs = C::SPLIT ? static_cast<int>(cluster_nctarank()) : 1;
    const int rank = C::SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    const int worker = static_cast<int>(blockIdx.x) / cs, workers = static_cast<int>(gridDim.x) / cs;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full_bar[s], 1 + 4);  // the operands, and the scale warps
            mbar_init(&empty_bar[s], 1);
            mbar_init(&sf_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], C::kEpiWarps);
        }
        mbar_init(part_full, cs);
        mbar_init(part_empty, cs);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmA32);
        prefetch_tensormap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (cs > 1) cluster_sync();  // the peers' barriers exist before anyone arrives on them
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    griddep_launch_dependents();
    const bool dense = args.mode == kFp4Dense;
    int tiles = args.mt * args.nt;  // dense; grouped: from the segments, below
    int t = worker;                 // the tile at hand, the same walk in every role
    F4Tile w;
    if (dense && t < tiles) w = f4_tile<C::BN, 128>(args, groups, t, args.group_m);
    if (dense && t < tiles && warp == 2 && lane == 0) f4_prefetch<C>(args, &tmB, w, rank, cs);
    __syncwarp();
    griddep_wait();
    if (!dense) {
        tiles = f4_groups<C::BN>(args, groups);
        if (t < tiles) w = f4_tile<C::BN, 128>(args, groups, t, args.group_m);
    }
    auto next = [&]() {
        t += workers;
        if (t < tiles) w = f4_tile<C::BN, 128>(args, groups, t, args.group_m);
    };

    if (warp == 0 || warp == C::kScaleLoadWarp) {
        // ----------------------------------------------------- TMA producers
        // One warp for the codes, one for the scales: a thread issues a copy in some 70
        // ns, and four a stage from one thread took longer than the stage (340 ns a
        // stage at one token x 16384 x 4096).
        const bool issue = elect_lane();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < tiles; next()) {
            const int nk = w.kb1 - w.kb0;
            const int k0 = w.kb0 + nk * rank / cs, k1 = w.kb0 + nk * (rank + 1) / cs;
            const int wide = f4_width(w);
            for (int kb = k0; kb < k1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                if (issue) {
                    if (warp == 0) {
                        uint64_t *bar = &full_bar[stage];
                        uint8_t *cols = cols_s + stage * C::kRBytes;
                        mbar_expect_relaxed(bar, C::kLBytes + wide * 128);
                        tma_load_2d(&tmB, bar, lanes_s + stage * C::kLBytes, kb * 128, w.b_row);
                        if (wide == C::BN) {
                            tma_load_2d(&tmA, bar, cols, kb * 128, w.a_row);
                        } else {
                            tma_load_2d(&tmA32, bar, cols, kb * 128, w.a_row);
                            if (wide > 32) tma_load_2d(&tmA32, bar, cols + 32 * 128, kb * 128, w.a_row + 32);
                        }
                    } else {
                        uint64_t *bar = &sf_bar[stage];
                        uint8_t *sf = sf_s + stage * 2 * C::kSfBytes;
                        mbar_expect_relaxed(bar, 2 * C::kSfBytes);
                        bulk_copy_g2s(sf, w.sb + static_cast<int64_t>(kb) * C::kSfBytes, C::kSfBytes, bar);
                        bulk_copy_g2s(sf + C::kSfBytes, w.sa + static_cast<int64_t>(kb) * C::kSfBytes, C::kSfBytes, bar);
                    }
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        await_copies(warp == 0 ? full_bar : sf_bar, S, stage, phase);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        const bool issue = elect_lane();
        const uint64_t l0 = smem_desc_sw128(smem_u32(lanes_s), 16, 1024), c0 = smem_desc_sw128(smem_u32(cols_s), 16, 1024);
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < tiles; next(), ++it) {
            const int nk = w.kb1 - w.kb0;
            const int k0 = w.kb0 + nk * rank / cs, k1 = w.kb0 + nk * (rank + 1) / cs;
            const int buf = it & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[buf], ((it >> 1) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + buf * C::BN;
            const uint32_t idesc = idesc_mxf4(128, f4_width(w), 0);
            for (int kb = k0; kb < k1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t ld = l0 + stage * (C::kLBytes >> 4), cd = c0 + stage * (C::kRBytes >> 4);
                const uint32_t sl = tmem_base + C::kSfCol + stage * C::kSfSet, sc = sl + 8;
                if (issue) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        umma_mxf4(d, ld + 2 * j, cd + 2 * j, (j & 1) ? idesc | idesc_mxf4(0, 0, 2) : idesc, sl + 4 * (j >> 1),
                                  sc + 4 * (j >> 1), (kb > k0 || j > 0) ? 1u : 0u);
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
    } else if (warp >= 2 + C::kEpiWarps) {
        // ------------------------------------------------------ scale warps
        // Shared memory to TMEM, as in f4_pair.
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < tiles; next()) {
            const int nk = w.kb1 - w.kb0;
            const int k0 = w.kb0 + nk * rank / cs, k1 = w.kb0 + nk * (rank + 1) / cs;
            for (int kb = k0; kb < k1; ++kb) {
                ok = mbar_wait(&sf_bar[stage], phase, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t sf = smem_u32(sf_s + stage * 2 * C::kSfBytes) + lane * 16;
                const uint32_t to = tmem_base + lanes + C::kSfCol + stage * C::kSfSet;
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = ld_shared_v4(sf + i * kFp4TileBytes);
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_store_4cols(to + 4 * i, v[i]);
                tmem_wait_store();
                tc_fence_before_sync();
                __syncwarp();
                // no memory access to release: wait::st has completed the TMEM writes
                if (lane == 0) mbar_arrive_relaxed(&full_bar[stage]);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // --------------------------------------------------------- epilogue
        // A warp that gave up on a wait keeps walking (its waits then return at
        // once), so that the barriers of the cluster's sum stay in step.
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int i = 32 * q + lane;  // lane of the tile: C's column n0 + i
        constexpr int kEpiThreads = 32 * C::kEpiWarps;
        int it = 0;
        for (; t < tiles; next(), ++it) {
            const int nk = w.kb1 - w.kb0;
            const bool some = nk * (rank + 1) / cs > nk * rank / cs;  // this CTA has a part of K
            const int buf = it & 1;
            bool ok = mbar_wait(&accf_bar[buf], (it >> 1) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after_sync();
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * C::BN;
            if (cs > 1) ok = mbar_wait_cluster(part_empty, (it & 1) ^ 1u, abort_flag) && ok;
            ok = __all_sync(0xffffffffu, ok);
            const int c_end = min(w.m_valid, (half + 1) * C::kEpiCols);
            for (int c0 = half * C::kEpiCols; c0 < c_end; c0 += 32) {
                float v[32];
                if (some && ok) {
                    tmem_load_32cols(t_row + c0, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                }
                if (cs > 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) dump[(c0 + j) * 128 + i] = v[j];
                } else {
                    store_columns<OUT>(args.c, w.c_row + c0, args.n, w.n0 + i, v, w.m_valid - c0,
                                       ok && i < w.n_valid && (OUT != 2 || some));
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(&acce_bar[buf]);
            if (cs > 1) {
                named_barrier_sync(1, kEpiThreads);
                if (threadIdx.x >= 64 && threadIdx.x < 64 + cs)
                    mbar_arrive_cluster(mapa_shared(smem_u32(part_full), threadIdx.x - 64));
                ok = mbar_wait_cluster(part_full, it & 1, abort_flag) && ok;
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    // columns rank, rank + cs, ...: eight at a time, their remote loads in flight together
                    constexpr int kCols = 8;
                    constexpr int kHalves = C::kEpiWarps / 4;
                    const int c_all = OUT == 2 && nk == 0 ? 0 : w.m_valid;  // 0: nothing to add
                    for (int c0 = rank + half * kCols * cs; c0 < c_all; c0 += kHalves * kCols * cs) {
                        float sum[kCols];
                        const int64_t at = (w.c_row + c0) * args.n + w.n0 + i;
#pragma unroll
                        for (int u = 0; u < kCols; ++u) sum[u] = 0.0f;
                        for (int r = 0; r < cs; ++r) {
                            const uint32_t from = mapa_shared(smem_u32(dump + i), r);
                            float part[kCols];
#pragma unroll
                            for (int u = 0; u < kCols; ++u)  // past the tile: column 0 instead, not stored
                                part[u] = ld_cluster_f32(from + (c0 + u * cs < w.m_valid ? c0 + u * cs : 0) * 512);
#pragma unroll
                            for (int u = 0; u < kCols; ++u) sum[u] += part[u];
                        }
#pragma unroll
                        for (int u = 0; u < kCols; ++u) {
                            if (i >= w.n_valid || c0 + u * cs >= w.m_valid) continue;
                            const int64_t o = at + static_cast<int64_t>(u * cs) * args.n;
                            if (OUT == 0) {
                                static_cast<uint16_t *>(args.c)[o] = static_cast<uint16_t>(pack_bf16x2(sum[u], 0.0f) & 0xFFFFu);
                            } else {
                                float *p = static_cast<float *>(args.c) + o;
                                *p = OUT == 2 ? *p + sum[u] : sum[u];
                            }
                        }
                    }
                }
                named_barrier_sync(1, kEpiThreads);
                if (threadIdx.x >= 64 && threadIdx.x < 64 + cs)
                    mbar_arrive_cluster(mapa_shared(smem_u32(part_empty), threadIdx.x - 64));
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (cs > 1) cluster_sync();  // no CTA leaves while its part may be read
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

// --------------------------------------------------------------------- f4_pair

__device__ __forceinline__ void umma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  setp.ne.b32 p, %6, 0;\n"
        "  tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// C's lines are the first to leave L2, so that the operands' stay (16384 x 8192 x 2048
// bf16: 91 -> 87 us).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int32_t c0, int32_t c1, int32_t c2) {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "l"(pol)
                 : "memory");
}

__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap *map, const void *src, int32_t c0, int32_t c1,
                                                  int32_t c2) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// TMEM of a pair tile: the two accumulators overlap in 128 columns, which leaves 128
// for the scales: accumulator 0 at 0, accumulator 1 at 128, the scales of each of the
// five stages (A: 8 columns, B: 16) from 384 on.  The epilogue drains the shared
// columns first and tells the MMA so; only then may the next tile start, and it does
// while the rest drains.
struct F4Pair {
    static constexpr int kThreads = 480;           // codes, MMA, eight epilogue warps, four scale warps, scale loads
    static constexpr int kScaleLoadWarp = kThreads / 32 - 1;
    static constexpr int kOpBytes = 128 * 128;     // 128 rows of A or B
    static constexpr int kSfABytes = 1024, kSfBBytes = 2048;
    static constexpr int kSfBytes = kSfABytes + kSfBBytes;
    static constexpr int kStageBytes = 2 * kOpBytes + kSfBytes;
    static constexpr int kStagingBytes = 8 * 4096; // 32 rows x 128 B an epilogue warp
    static constexpr int kCtrlBytes = 4096;
    static constexpr int kStages = (kSmemLimit - 1024 - kCtrlBytes - kStagingBytes) / kStageBytes;
    static constexpr int kSmemBytes = 1024 + kCtrlBytes + kStagingBytes + kStages * kStageBytes;
    static constexpr int kAcc1 = 128, kSfCol = 384, kSfSet = 24;
    static_assert(kStages >= 4 && kSfCol + kStages * kSfSet <= 512, "shared memory or TMEM over budget");
};

// OUT: 0 bf16, 1 float32, 2 float32 +=.  TMA_OUT: rows of C are a multiple of 16 bytes.
template <int OUT, bool TMA_OUT>
__global__ void __launch_bounds__(F4Pair::kThreads, 1)
f4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const __grid_constant__ CUtensorMap tmC, const F4Args args) {
    using P = F4Pair;
    constexpr int S = P::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *a_s = smem;                             // [S][128 rows][128 B]
    uint8_t *b_s = a_s + S * P::kOpBytes;            // [S][128 rows][128 B]
    uint8_t *staging = b_s + S * P::kOpBytes;        // [8 warps][32 rows][128 B]
    uint8_t *sf_s = staging + P::kStagingBytes;      // [S][A 1 KB, B 2 KB]
    uint8_t *ctrl = sf_s + S * P::kSfBytes;
    uint64_t *full_bar = reinterpret_cast<uint64_t *>(ctrl);
    uint64_t *empty_bar = full_bar + S;
    uint64_t *accf_bar = empty_bar + S;
    uint64_t *acce_bar = accf_bar + 2;   // accumulator drained
    uint64_t *ovl_bar = acce_bar + 2;    // the columns shared with the other accumulator drained
    uint64_t *sf_bar = ovl_bar + 1;      // this CTA's scales of a stage are in shared memory
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctrl + 384);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctrl + 388);
    F4Groups *groups = reinterpret_cast<F4Groups *>(ctrl + 512);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full_bar[s], 1 + 8);  // both CTAs' operands, and their scale warps
            mbar_init(&empty_bar[s], 1);
            mbar_init(&sf_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], 16);  // both CTAs' epilogue warps (the leader's barrier counts)
        }
        mbar_init(ovl_bar, 16);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmSA);
        prefetch_tensormap(&tmSB);
        if (TMA_OUT) prefetch_tensormap(&tmC);
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
    int tiles = args.mt * args.nt;  // dense; grouped: from the segments, below
    int t = worker;                 // the tile at hand, the same walk in every role
    F4Tile w;
    if (args.mode == kFp4Dense && t < tiles) w = f4_tile<256, 256>(args, groups, t, args.group_m);
    griddep_wait();
    if (args.mode != kFp4Dense) {
        tiles = f4_groups<256>(args, groups);
        if (t < tiles) w = f4_tile<256, 256>(args, groups, t, args.group_m);
    }
    auto next = [&]() {
        t += workers;
        if (t < tiles) w = f4_tile<256, 256>(args, groups, t, args.group_m);
    };

    if (warp == 0 || warp == P::kScaleLoadWarp) {
        // ------------------------------- TMA producers: the codes, the scales
        const bool issue = elect_lane();
        const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < tiles; next()) {
            const int a_row = w.a_row + static_cast<int>(rank) * 128, b_row = w.b_row + static_cast<int>(rank) * 128;
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                if (issue) {
                    if (warp != 0) {
                        uint8_t *sf = sf_s + stage * P::kSfBytes;
                        mbar_expect_relaxed(&sf_bar[stage], P::kSfBytes);
                        tma_load_2d(&tmSA, &sf_bar[stage], sf, kb * 256, w.sa_tile + static_cast<int>(rank));
                        tma_load_2d(&tmSB, &sf_bar[stage], sf + P::kSfABytes, kb * 256, w.sb_tile);
                    } else {
                        uint8_t *da = a_s + stage * P::kOpBytes, *db = b_s + stage * P::kOpBytes;
                        if (leader) {
                            // the leader's barrier collects both CTAs' operand bytes
                            uint64_t *bar = &full_bar[stage];
                            mbar_expect_relaxed(bar, 4 * P::kOpBytes);
                            tma_load_2d(&tmA, bar, da, kb * 128, a_row);
                            tma_load_2d(&tmB, bar, db, kb * 128, b_row);
                        } else {
                            tma_load_2d_pair(&tmA, full0 + stage * 8, da, kb * 128, a_row);
                            tma_load_2d_pair(&tmB, full0 + stage * 8, db, kb * 128, b_row);
                        }
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
        if (warp != 0) await_copies(sf_bar, S, stage, phase);
        else if (leader) await_copies(full_bar, S, stage, phase);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        if (leader) {
            const bool issue = elect_lane();
            const uint64_t a0 = smem_desc_sw128(smem_u32(a_s), 16, 1024), b0 = smem_desc_sw128(smem_u32(b_s), 16, 1024);
            int stage = 0, it = 0;
            uint32_t phase = 0;
            bool ok = true;
            auto next_k = [&]() {  // stages of the tile at hand, or of the next that has any
                for (; t < tiles; next())
                    if (w.kb0 < w.kb1) return w.kb1 - w.kb0;
                return 0;
            };
            int nk = next_k();
            while (ok && nk > 0) {
                const int now = nk;
                const int buf = it & 1;
                ok = mbar_wait(&acce_bar[buf], ((it >> 1) & 1) ^ 1u, abort_flag);
                if (ok && it > 0) ok = mbar_wait(ovl_bar, (it - 1) & 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + (buf ? P::kAcc1 : 0);
                for (int kb = 0; kb < now; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t ad = a0 + stage * (P::kOpBytes >> 4), bd = b0 + stage * (P::kOpBytes >> 4);
                    const uint32_t sa = tmem_base + P::kSfCol + stage * P::kSfSet, sb = sa + 8;
                    if (issue) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            umma_mxf4_pair(d, ad + 2 * j, bd + 2 * j, (j & 1) ? idesc_mxf4(256, 256, 2) : idesc_mxf4(256, 256, 0),
                                           sa + 4 * (j >> 1), sb + 8 * (j >> 1), (kb > 0 || j > 0) ? 1u : 0u);
                        umma_commit_pair(&empty_bar[stage], 3);
                    }
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (kb == 0) {  // while the first stage's MMAs run
                        next();
                        nk = next_k();
                    }
                }
                if (!ok) break;
                if (issue) umma_commit_pair(&accf_bar[buf], 3);
                __syncwarp();
                ++it;
            }
        }
        __syncwarp();
    } else if (warp >= 10) {
        // ------------------------------------------------------ scale warps
        // Shared memory to TMEM.  A stage's TMEM columns are free again once its shared
        // memory is (its MMAs have completed), so sf_bar's phase covers both.
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (; ok && t < tiles; next()) {
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                ok = mbar_wait(&sf_bar[stage], phase, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                // word 4l + j of a tile is row 32j + l's four scales: column j, lane l
                const uint32_t sf = smem_u32(sf_s + stage * P::kSfBytes) + lane * 16;
                const uint32_t to = tmem_base + lanes + P::kSfCol + stage * P::kSfSet;
                uint4 v[6];
#pragma unroll
                for (int i = 0; i < 6; ++i) v[i] = ld_shared_v4(sf + i * kFp4TileBytes);
                tmem_store_4cols(to, v[0]);       // A, K values 0-127 of the stage
                tmem_store_4cols(to + 4, v[1]);   // A, 128-255
                tmem_store_4cols(to + 8, v[2]);   // B rows 0-127, K 0-127
                tmem_store_4cols(to + 12, v[4]);  // B rows 128-255, K 0-127
                tmem_store_4cols(to + 16, v[3]);
                tmem_store_4cols(to + 20, v[5]);
                tmem_wait_store();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    // no memory access to release: wait::st has completed the TMEM writes
                    if (leader) mbar_arrive_relaxed(&full_bar[stage]);
                    else mbar_arrive_cluster_relaxed(full0 + stage * 8);
                }
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else {
        // --------------------------------------------------------- epilogue
        // Two warps a lane quarter; each drains 64 of the 128 columns that the other
        // accumulator shares, then 64 more.
        const int q = warp & 3, ew = warp - 2;
        const bool first = ew < 4;
        uint8_t *st = staging + ew * 4096;
        const uint32_t srow = smem_u32(st) + lane * 128;
        const uint32_t sw = static_cast<uint32_t>(lane & 7);
        const uint32_t ovl0 = mapa_shared(smem_u32(ovl_bar), 0), acce0 = mapa_shared(smem_u32(&acce_bar[0]), 0);
        int it = 0;
        for (; t < tiles; next()) {
            const bool some = w.kb0 < w.kb1;
            if (OUT == 2 && !some) continue;  // nothing to add
            const int buf = it & 1;
            if (some) {
                const bool ok = mbar_wait(&accf_bar[buf], (it >> 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after_sync();
            }
            const int rt = static_cast<int>(rank) * 128 + 32 * q;  // the warp's first row of the tile
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + (buf ? P::kAcc1 : 0);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int chunk = buf ? (first ? 0 : 1) + 2 * i : (first ? 2 : 3) - 2 * i;
                float v[2][32];
                if (some) {
                    tmem_load_64cols(t_row + 64 * chunk, v[0], v[1]);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        // the leader's MMA may overwrite what every warp has now read
                        if (i == 0) {
                            if (leader) mbar_arrive_relaxed(ovl_bar);
                            else mbar_arrive_cluster_relaxed(ovl0);
                        }
                        if (i == 1) {
                            if (leader) mbar_arrive_relaxed(&acce_bar[buf]);
                            else mbar_arrive_cluster_relaxed(acce0 + buf * 8);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[0][j] = v[1][j] = 0.0f;
                }
                const int col = w.n0 + 64 * chunk;
                if (rt >= w.m_valid || col >= args.n) continue;
                constexpr int kParts = OUT == 0 ? 1 : 2;  // 128-byte pieces of a row of the chunk
#pragma unroll
                for (int h = 0; h < kParts; ++h) {
                    constexpr int kCols = OUT == 0 ? 64 : 32;
                    const int c0 = col + h * kCols;
                    if (TMA_OUT) {
                        if (lane == 0) bulk_wait_group_read<0>();  // the staging rows are free again
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t at = srow + ((static_cast<uint32_t>(j) ^ sw) << 4);
                        if (OUT == 0) {
                            const float *e = j < 4 ? &v[0][8 * j] : &v[1][8 * (j - 4)];
                            st_shared_v4(at, pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                                         pack_bf16x2(e[6], e[7]));
                        } else {
                            const float *e = &v[h][4 * j];
                            st_shared_v4(at, __float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]),
                                         __float_as_uint(e[3]));
                        }
                    }
                    if (TMA_OUT) {
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0 && c0 < args.n) {
                            const int r = w.c_local + rt;
                            if (OUT == 2) tma_reduce_add_3d(&tmC, st, c0, r, w.c_mat);
                            else tma_store_3d(&tmC, st, c0, r, w.c_mat);
                            bulk_commit_group();
                        }
                    } else {
                        // rows of any length: eight rows at a time, neighbouring lanes neighbouring
                        // columns
                        __syncwarp();
                        const int n_rows = min(32, w.m_valid - rt);
                        using E = typename std::conditional<OUT == 0, uint16_t, float>::type;
                        E *out = static_cast<E *>(args.c) + (w.c_row + rt) * args.n + c0 + lane;
#pragma unroll 1
                        for (int r0 = 0; r0 < n_rows; r0 += 8, out += 8 * args.n) {
                            E e[8][kCols / 32];
                            float old[8];
#pragma unroll
                            for (int r = 0; r < 8; ++r)
#pragma unroll
                                for (int u = 0; u < kCols / 32; ++u) {
                                    const int byte = (lane + 32 * u) * static_cast<int>(sizeof(E));
                                    e[r][u] = *reinterpret_cast<const E *>(st + (r0 + r) * 128 + ((((byte >> 4) ^ r) << 4) | (byte & 15)));
                                }
                            if (OUT == 2) {
#pragma unroll
                                for (int r = 0; r < 8; ++r)
                                    old[r] = r0 + r < n_rows && c0 + lane < args.n ? static_cast<float>(out[r * args.n]) : 0.0f;
                            }
#pragma unroll
                            for (int r = 0; r < 8; ++r)
#pragma unroll
                                for (int u = 0; u < kCols / 32; ++u)
                                    if (r0 + r < n_rows && c0 + lane + 32 * u < args.n)
                                        out[r * args.n + 32 * u] = OUT == 2 ? static_cast<E>(old[r] + static_cast<float>(e[r][u])) : e[r][u];
                        }
                        __syncwarp();
                    }
                }
            }
            if (some) ++it;
        }
        if (TMA_OUT && lane == 0) bulk_wait_group<0>();
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

// A code matrix as a 2-D byte array: box of 128 bytes (a stage of K) x `box_rows` rows.
bool make_map_codes(CUtensorMap *m, const void *codes, int64_t rows, int64_t k, uint32_t box_rows) {
    return make_map_2d(m, codes, kMapU8, static_cast<uint64_t>(fp4_row_bytes(k)), static_cast<uint64_t>(rows), 128, box_rows);
}

template <class C, int OUT>
int run_small(F4Args a, const Fp4Product &p, int cs, int workers, cudaStream_t s) {
    a.group_m = 8;
    a.mt = static_cast<int>((p.m + C::BN - 1) / C::BN);
    a.nt = static_cast<int>((p.n + 127) / 128);
    CUtensorMap mA, mA32, mB;
    const int64_t a_rows = p.m, b_rows = p.mode == kFp4GroupRows ? p.n * p.experts : p.n;
    // a map takes 0.2 us of host time: none that no tile's rows ask for (f4_width)
    const int64_t last = p.m % C::BN;
    const bool narrow = p.mode != kFp4Dense || (last != 0 && last <= 64), wide = p.mode != kFp4Dense || p.m > 64;
    if (!make_map_codes(&mB, p.b, b_rows, p.k, 128)) return MLPBLK_ECUDA;
    if (wide && !make_map_codes(&mA, p.a, a_rows, p.k, C::BN)) return MLPBLK_ECUDA;
    if (narrow && !make_map_codes(&mA32, p.a, a_rows, p.k, 32)) return MLPBLK_ECUDA;
    if (!wide) mA = mA32;
    if (!narrow) mA32 = mA;
    static int attr_set[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    if (!attr_set[dev]) {
        const int rc = cuda_status(cudaFuncSetAttribute(f4_small_kernel<C, OUT>,
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes));
        if (rc != MLPBLK_OK) return rc;
        attr_set[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(workers) * cs);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C::SPLIT ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, f4_small_kernel<C, OUT>, mA, mA32, mB, a));
}

// Scales as a 2-D array of words: a row is the tiles of 128 rows of the matrix, a
// stage's part of it 256 words.
bool make_map_scales(CUtensorMap *m, const void *scales, int64_t row_tiles, int64_t k, uint32_t box_rows) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t words = static_cast<cuuint64_t>(fp4_col_tiles(k)) * (kFp4TileBytes / 4);
    cuuint64_t dims[2] = {words, static_cast<cuuint64_t>(row_tiles)};
    cuuint64_t strides[1] = {words * 4};
    cuuint32_t box[2] = {256, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(scales), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// C as matrices of [m, n]: boxes of 32 rows x 128 bytes, 128-byte swizzle.
bool make_map_c(CUtensorMap *m, void *c, bool f32, int64_t mats, int64_t rows, int64_t cols) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t esz = f32 ? 4 : 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    cuuint64_t strides[2] = {dims[0] * esz, dims[0] * dims[1] * esz};
    cuuint32_t box[3] = {f32 ? 32u : 64u, 32u, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OUT, bool TMA_OUT>
int run_pair(F4Args a, const Fp4Product &p, int workers, cudaStream_t s) {
    a.group_m = 4;  // 8192 x 16384 x 4096: 157 us; 160 with 8, 162 with 16
    a.mt = static_cast<int>((p.m + 255) / 256);
    a.nt = static_cast<int>((p.n + 255) / 256);
    CUtensorMap mA, mB, mSA, mSB, mC;
    const bool rows_grouped = p.mode == kFp4GroupRows;
    const int64_t a_tiles = (p.m + 127) / 128, b_tiles = (p.n + 127) / 128 * (rows_grouped ? p.experts : 1);
    if (!make_map_codes(&mA, p.a, p.m, p.k, 128) || !make_map_codes(&mB, p.b, rows_grouped ? p.n * p.experts : p.n, p.k, 128) ||
        !make_map_scales(&mSA, p.sa, a_tiles, p.k, 1) || !make_map_scales(&mSB, p.sb, b_tiles, p.k, 2))
        return MLPBLK_ECUDA;
    if (TMA_OUT) {
        if (!make_map_c(&mC, p.c, OUT != 0, p.mode == kFp4GroupK ? p.experts : 1, p.m, p.n)) return MLPBLK_ECUDA;
    } else {
        mC = mA;
    }
    static int attr_set[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    if (!attr_set[dev]) {
        const int rc = cuda_status(cudaFuncSetAttribute(f4_pair_kernel<OUT, TMA_OUT>,
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, F4Pair::kSmemBytes));
        if (rc != MLPBLK_OK) return rc;
        attr_set[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * static_cast<unsigned>(workers));
    cfg.blockDim = dim3(F4Pair::kThreads);
    cfg.dynamicSmemBytes = F4Pair::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, f4_pair_kernel<OUT, TMA_OUT>, mA, mB, mSA, mSB, mC, a));
}

}  // namespace

Fp4Choice choose_fp4_matmul(const Fp4Product &p, int num_sms) {
    const bool f32 = p.out_dtype == MLPBLK_FP32;
    const int kblocks = static_cast<int>((p.k + kF4KB - 1) / kF4KB);
    int64_t rows = p.m;  // rows of one product, at most
    int64_t groups = 1;
    if (p.mode == kFp4GroupRows) {
        if (p.max_rows > 0 && p.max_rows < rows) rows = p.max_rows;
        groups = p.experts;
    } else if (p.mode == kFp4GroupK) {
        groups = p.experts;
    }
    Fp4Choice c = {};
    // 256 x 256 pair tiles where they occupy half of the SM pairs and, grouped by rows, an
    // expert has more than one 128-row tile on average (1500 tokens, top-4 of 60 experts
    // of 776 x 1000: 13.8 us in pair tiles, 8.4 in small ones).  A single round of them
    // needs 16 stages to make up for its longer start and end (2048 x 2048 x 1024 4.8 us
    // in small tiles, 5.8 in pair tiles; x 4096 9.3 and 9.3; x 8192 15.1 and 13.8), and
    // float32 rows that are not whole 16-byte pieces 6 (8192 x 4095 x 1024 33 and 41 us,
    // x 4096 63 and 55).
    const int pairs = num_sms / 2;
    const int64_t mean_rows = p.mode == kFp4GroupRows ? rows / p.experts : rows;
    const int64_t pair_tiles = p.mode == kFp4GroupRows ? ((mean_rows + 255) / 256) * p.experts * ((p.n + 255) / 256)
                                                       : (rows + 255) / 256 * groups * ((p.n + 255) / 256);
    c.tma = p.n * (f32 ? 4 : 2) % 16 == 0;
    const int stages_of_tile = p.mode == kFp4GroupK ? kblocks / p.experts : kblocks;
    const int least = pair_tiles <= pairs ? 16 : (f32 && !c.tma ? 6 : 0);
    if (pairs >= 1 && mean_rows > 128 && 2 * pair_tiles >= pairs && stages_of_tile >= least) {
        c.pair = true;
        c.workers = static_cast<int>(p.mode != kFp4GroupRows && pair_tiles < pairs ? pair_tiles : pairs);
        return c;
    }
    // K is split where that saves more of its stages than the cluster's sum costs: 4 us for
    // 128 columns, 1.5 for up to 32.  A stage takes 0.15 us, twice that where rows of codes
    // begin at no 128-byte line (each of its 256 rows is then two requests of the copies):
    // 128 x 128 x 8192 7.3 us whole and 7.8 split, x 16384 12.3 and 8.4; 118 x 192 x 6624
    // 11.3 and 8.9; one token x 1024 x 4096 4.3 and 4.7, x 8192 6.6 and 5.2.
    const int64_t tiles = (rows + 127) / 128 * ((p.n + 127) / 128) * groups;
    const int64_t stages = static_cast<int64_t>(kblocks) * (fp4_row_bytes(p.k) % 128 != 0 ? 2 : 1);
    c.split = 1;
    if (stages >= (rows <= 32 ? 32 : 40))
        while (c.split < 8 && tiles * c.split * 2 <= num_sms && stages >= 8 * c.split) c.split *= 2;
    int64_t workers = num_sms / c.split;
    if (workers < 1) workers = 1;
    if (p.mode != kFp4GroupRows && tiles < workers) workers = tiles;
    c.workers = static_cast<int>(workers);
    return c;
}

int launch_fp4_matmul(const Fp4Product &p, int num_sms, cudaStream_t s) {
    F4Args a = {};
    a.mode = p.mode;
    a.m = p.m;
    a.n = p.n;
    a.kblocks = static_cast<int>((p.k + kF4KB - 1) / kF4KB);
    a.experts = p.experts;
    a.max_rows = p.max_rows;
    a.sa = p.sa;
    a.sb = p.sb;
    a.row_tile_bytes = fp4_col_tiles(p.k) * kFp4TileBytes;
    a.count = p.count;
    a.seg = p.seg;
    a.c = p.c;
    const bool f32 = p.out_dtype == MLPBLK_FP32;
    const Fp4Choice ch = choose_fp4_matmul(p, num_sms);
    const int w = ch.workers;
    if (ch.pair) {
        if (!f32) return ch.tma ? run_pair<0, true>(a, p, w, s) : run_pair<0, false>(a, p, w, s);
        if (!p.accumulate) return ch.tma ? run_pair<1, true>(a, p, w, s) : run_pair<1, false>(a, p, w, s);
        return ch.tma ? run_pair<2, true>(a, p, w, s) : run_pair<2, false>(a, p, w, s);
    }
#define MLPBLK_SMALL(SPLIT)                                                           \
    {                                                                                 \
        if (!f32) return run_small<F4Small<SPLIT>, 0>(a, p, ch.split, w, s);          \
        if (!p.accumulate) return run_small<F4Small<SPLIT>, 1>(a, p, ch.split, w, s); \
        return run_small<F4Small<SPLIT>, 2>(a, p, ch.split, w, s);                    \
    }
    if (ch.split > 1) MLPBLK_SMALL(true)
    MLPBLK_SMALL(false)
#undef MLPBLK_SMALL
}

int take_device_error_gemm_f4() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return MLPBLK_ECUDA;
    if (v != 0) cudaMemcpyToSymbol(g_device_error, &z, sizeof(int));
    return v;
}

}  // namespace mlpblk
