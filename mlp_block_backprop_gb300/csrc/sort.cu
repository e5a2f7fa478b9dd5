// sort.cu -- tokens sorted by expert and back ("Nemotron Kernels From Inference To
// Backpropagation" -- "Kernel 4: Routed ReLU2 MoE": select, execute, weight and
// combine), as operators of their own: the plan, the two moves and their gradients.
//
//   plan       rank of entry i among the entries of its expert; pos[i] = seg + rank
//   permute    rows[pos[t,j]] = x[t]                dx[t] = sum_j d_rows[pos[t,j]]
//   unpermute  y[t] = residual[t] + sum_j w[t,j] * rows[pos[t,j]]
//              d_rows[pos[t,j]] = w[t,j] * dy[t],   dw[t,j] = <dy[t], rows[pos[t,j]]>
//
// The moves are bound by HBM.  All of them walk the tokens, not the sorted rows: a
// token's row is then read (or written) once for all of its slots.
#include <algorithm>

#include "mlpblk_internal.h"

namespace mlpblk {

namespace {

// ------------------------------------------------------------------- the plan

constexpr int kSortExperts = 256;
constexpr int kSortCluster = 8;        // CTAs of a large plan (the portable cluster size)
constexpr int64_t kSortOneCta = 4096;  // entries up to which one CTA makes the plan
constexpr int64_t kSortOneRows = 9216; // and sorted rows, most of which it only marks as empty (4096 entries of 128 experts
                                       // padded to 256: 10.3 us, with a cluster 6.2; 384 of 64 padded to 128: 4.6 and 5.0)
constexpr int64_t kSortSmallRows = 4096;
constexpr int64_t kSortSmall = 64;     // entries up to which that CTA has 8 warps, not 32 (16 entries: 3.6 us and 4.1;
                                       // 384 of 64 experts, whose padding is most of the work: 6.2 and 5.2)

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ int ld_cluster(const int *local, unsigned rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local)), r;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
    return v;
}

// One cluster makes the whole plan in one launch: CTA c of C takes a contiguous
// range of the entries, warp w a contiguous part of that, so ranks follow entry
// order.  A warp walks its part once: lanes with the same expert find each other by a
// ballot for each bit of the id (match_any does the same at one instruction in some 80
// cycles an SM: 24582 entries of 60 experts, 3.8 us for the ranks alone) and take the
// next ranks within the warp.  The counts' prefixes then run over
// the warps (a lane a warp) and over the CTAs through distributed shared memory, and an
// entry's row is its expert's first row, plus the entries before its CTA, its warp,
// and itself.  An entry's expert and rank stay in a register for parts of up to
// 32 * kSortKeep entries, plans of up to 131072 in eight CTAs (13.3 us, 8 experts); longer
// parts leave the rank in pos and read the id again (131074: 18.0, 262144: 29).
// Bound by latency: one pass over the ids, two cluster barriers.
constexpr int kSortKeep = 16;

template <int kSortWarps>
__global__ void __launch_bounds__(32 * kSortWarps)
sort_kernel(const int *__restrict__ idx, int64_t n, int experts, int pad, int64_t R, int64_t per_warp,
            int *__restrict__ count, int *__restrict__ seg, int *__restrict__ pos, int *__restrict__ row_map) {
    constexpr int kSortThreads = 32 * kSortWarps;
    __shared__ int wcnt[kSortExperts][kSortWarps + 1];  // entries of an expert in a warp, then in the warps before it
    __shared__ int ctot[kSortExperts];       // this CTA's entries per expert (read by the cluster)
    __shared__ int segs[kSortExperts + 1];
    __shared__ int first[kSortExperts];      // the row of this CTA's first entry of an expert
    __shared__ int live[kSortExperts];       // every CTA's entries per expert
    __shared__ int scan[kSortExperts / 32];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int C = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    const unsigned lt = (1u << lane) - 1u;
    for (int e = lane; e < experts; e += 32) wcnt[e][wid] = 0;
    __syncwarp();
    const int64_t w0 = (static_cast<int64_t>(c) * kSortWarps + wid) * per_warp;
    const int64_t w1 = min(n, w0 + per_warp);
    const bool keep = per_warp <= 32 * kSortKeep;
    const int bits = 32 - __clz(experts);  // of the ids 0 .. experts - 1 and of -1
    uint32_t kept[kSortKeep];  // rank in the warp << 9 | expert (511: none)
    griddep_wait();
    // the next rank of expert e within the warp, for the 32 lanes' entries in order
    auto rank_of = [&](int e) {
        unsigned peers = 0xffffffffu;  // lanes with the same id (-1 has every bit set)
        for (int b = 0; b < bits; ++b) {
            const bool set = e >> b & 1;
            const unsigned m = __ballot_sync(0xffffffffu, set);
            peers &= set ? m : ~m;
        }
        const int base = e >= 0 ? wcnt[e][wid] : 0;
        __syncwarp();
        if (e >= 0 && (peers & lt) == 0) wcnt[e][wid] = base + __popc(peers);
        __syncwarp();
        return base + __popc(peers & lt);
    };
    auto valid = [&](int e) { return e >= 0 && e < experts ? e : -1; };
    if (keep) {
#pragma unroll
        for (int g = 0; g < kSortKeep; ++g) {
            const int64_t i = w0 + 32 * g + lane;
            kept[g] = static_cast<uint32_t>(i < w1 ? valid(idx[i]) : -1);
        }
#pragma unroll
        for (int g = 0; g < kSortKeep; ++g) {
            if (w0 + 32 * g >= w1) break;
            const int e = static_cast<int>(kept[g]);
            const int r = rank_of(e);
            kept[g] = (static_cast<uint32_t>(r) << 9) | (e < 0 ? 511u : static_cast<uint32_t>(e));
        }
    } else {
        for (int64_t g = w0; g < w1; g += 32) {
            const int64_t i = g + lane;
            const int r = rank_of(i < w1 ? valid(idx[i]) : -1);
            if (i < w1) pos[i] = r;
        }
    }
    __syncthreads();
    // the warps before each warp: warp w takes experts w, w + kSortWarps, ..., a lane a warp
    for (int e = wid; e < experts; e += kSortWarps) {
        const int own = lane < kSortWarps ? wcnt[e][lane] : 0;
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane < kSortWarps) wcnt[e][lane] = incl - own;
        if (lane == 31) ctot[e] = incl;
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    int before = 0, all = 0, padded = 0, incl = 0;
    if (tid < kSortExperts) {
        if (tid < experts) {
            if (C > 1) {
#pragma unroll
                for (int r = 0; r < kSortCluster; ++r) {
                    const int v = r < C ? ld_cluster(&ctot[tid], r) : 0;
                    before += r < c ? v : 0;
                    all += v;
                }
            } else {
                all = ctot[tid];
            }
        }
        live[tid] = all;
        padded = (all + pad - 1) / pad * pad;
        incl = padded;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) scan[wid] = incl;
    }
    if (C > 1) cluster_arrive();  // this CTA has read the others' counts
    __syncthreads();
    if (tid < kSortExperts) {
        int off = 0;
#pragma unroll
        for (int w = 0; w < kSortExperts / 32; ++w) off += w < wid ? scan[w] : 0;
        segs[tid + 1] = off + incl;
        if (tid == 0) segs[0] = 0;
        first[tid] = off + incl - padded + before;
    }
    __syncthreads();
    if (c == 0) {
        if (tid < experts) count[tid] = live[tid];
        for (int e = tid; e <= experts; e += kSortThreads) seg[e] = segs[e];
    }
    auto place = [&](int64_t i, int e, int r) {
        const int p = e < 0 ? -1 : first[e] + wcnt[e][wid] + r;
        pos[i] = p;
        if (p >= 0) row_map[p] = static_cast<int>(i);
    };
    if (keep) {
#pragma unroll
        for (int g = 0; g < kSortKeep; ++g) {
            const int64_t i = w0 + 32 * g + lane;
            const uint32_t e = kept[g] & 511u;
            if (i < w1) place(i, e == 511u ? -1 : static_cast<int>(e), static_cast<int>(kept[g] >> 9));
        }
    } else {
        for (int64_t i = w0 + lane; i < w1; i += 32) place(i, valid(idx[i]), pos[i]);
    }
    // rows without an entry: the segments' padding and what lies behind them (64 bits: a
    // lane's row may lie behind the last int)
    if (pad > 1)
        for (int e = c * kSortWarps + wid; e < experts; e += C * kSortWarps)
            for (int64_t r = static_cast<int64_t>(segs[e]) + live[e] + lane; r < segs[e + 1]; r += 32) row_map[r] = -1;
    for (int64_t r = static_cast<int64_t>(segs[experts]) + c * kSortThreads + tid; r < R; r += C * kSortThreads)
        row_map[r] = -1;
    if (C > 1) cluster_wait();  // no CTA leaves while its counts are being read
}

// ------------------------------------------------------------------ the moves

// A row is `units` accesses of type U (16, 4 or 2 bytes: the widest that divides
// a row), a CTA kMoveThreads / TX rows of TX threads.  A thread holds several accesses
// at a time, TX apart: enough bytes in flight where they are short; TX (32, 64 or 128) is
// the least that covers a row so, that no thread's accesses lie behind it (16384 x 2048
// bf16, top-2, unpermute: 68 us with 128 threads, 46 with 64).  TX is a constant,
// so a row's addresses are one pointer and immediate offsets (64-bit indices throughout
// cost the plan, both moves and both gradients of 4097 x 1001 float32, top-6, 18 us beside
// 111, of 16384 x 4096 bf16, top-2, 17 beside 305).
constexpr int kMoveThreads = 128;  // 256: 4097 x 1001 float32 109 us, 107 so; 16384 x 2049 bf16 352 and 336
template <class U>
constexpr int kPerOf = sizeof(U) == 16 ? 4 : 8;  // permute
template <class U, bool RES>
constexpr int kPerUnOf = sizeof(U) == 16 && RES ? 2 : kPerOf<U>;  // unpermute, with and without a residual
constexpr int kSlots = 2;  // slots whose rows the gradient loads together
// unpermute's gradient (16384 tokens, top-2, bf16: x 4096 97 us; x 4098 104, with four
// slots of four accesses 114; x 2049 134 and 181)
template <class U>
constexpr int kPerBwdOf = sizeof(U) == 16 ? 2 : 8;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// The float values of one access, and back.
template <class U, bool BF16>
struct Vals;
template <>
struct Vals<uint4, true> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(uint4 u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[8]) {
        return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    }
};
template <>
struct Vals<uint32_t, true> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void get(uint32_t u, float (&v)[2]) {
        v[0] = __uint_as_float(u << 16);
        v[1] = __uint_as_float(u & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint32_t put(const float (&v)[2]) { return pack2(v[0], v[1]); }
};
template <>
struct Vals<uint16_t, true> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void get(uint16_t u, float (&v)[1]) {
        v[0] = __uint_as_float(static_cast<uint32_t>(u) << 16);
    }
    static __device__ __forceinline__ uint16_t put(const float (&v)[1]) {
        return static_cast<uint16_t>(pack2(v[0], 0.0f) & 0xFFFFu);
    }
};
template <>
struct Vals<uint4, false> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(uint4 u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Vals<uint32_t, false> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void get(uint32_t u, float (&v)[1]) { v[0] = __uint_as_float(u); }
    static __device__ __forceinline__ uint32_t put(const float (&v)[1]) { return __float_as_uint(v[0]); }
};

template <class U>
__device__ __forceinline__ U zero_unit() {
    U z;
    memset(&z, 0, sizeof(U));
    return z;
}

// An entry's row, -1 where it has none.  Positions of another plan than this shape's
// are taken as none, so no access leaves the R rows.
__device__ __forceinline__ int entry_row(const int *pos, int64_t i, int R) {
    const int r = pos[i];
    return static_cast<unsigned>(r) < static_cast<unsigned>(R) ? r : -1;
}

// An expert's padding rows are one range of bytes, cut into `slices` parts of whole rows;
// this CTA zeros part q % slices of expert q / slices, in 16-byte stores between the
// part's first and last 16-byte boundary, whatever a row's own access is.  (With a CTA
// for every two rows that might be padding, most of them without one, the gradient of 6
// tokens of 536 bf16, 201 experts padded to 256, took 33 us, with the parts 7.7.)
template <class U>
__device__ __forceinline__ void zero_padding(U *rows, int units, int64_t q, int slices, int experts, const int *count,
                                             const int *seg, int R) {
    const int e = static_cast<int>(q / slices), i = static_cast<int>(q % slices);
    if (e >= experts) return;
    const int64_t live = static_cast<int64_t>(seg[e]) + count[e];
    const int64_t end = min(seg[e + 1], R), n = end - live;
    if (live < 0 || n <= 0) return;
    U *p = rows + (live + n * i / slices) * units;
    const int64_t len = (n * (i + 1) / slices - n * i / slices) * units;
    const int64_t head = min(len, static_cast<int64_t>((-reinterpret_cast<uintptr_t>(p) & 15) / sizeof(U)));
    const int64_t body = (len - head) / (16 / sizeof(U)), tail = head + body * (16 / sizeof(U));
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    for (int64_t c = tid; c < head; c += kMoveThreads) p[c] = zero_unit<U>();
    uint4 *wide = reinterpret_cast<uint4 *>(p + head);
    for (int64_t c = tid; c < body; c += kMoveThreads) wide[c] = make_uint4(0, 0, 0, 0);
    for (int64_t c = tail + tid; c < len; c += kMoveThreads) p[c] = zero_unit<U>();
}

// rows[pos[t,j]] = x[t]; the blocks behind the tokens' zero the padding rows.
template <int TX, class U>
__global__ void __launch_bounds__(kMoveThreads)
permute_kernel(const U *__restrict__ x, const int *__restrict__ pos, const int *__restrict__ count,
               const int *__restrict__ seg, int64_t T, int k, int experts, int slices, int R, int units, int parts,
               int64_t token_blocks, U *__restrict__ rows) {
    constexpr int kPer = kPerOf<U>;
    griddep_enter();
    const int64_t b = blockIdx.x;
    if (b >= token_blocks) {
        zero_padding(rows, units, b - token_blocks, slices, experts, count, seg, R);
        return;
    }
    const int64_t t = static_cast<int64_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    if (t >= T) return;
    const int step = parts * kPer * TX;
    for (int c = static_cast<int>(blockIdx.x % parts) * kPer * TX + threadIdx.x; c < units; c += step) {
        const U *src = x + t * units + c;
        U v[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) v[u] = c + u * TX < units ? __ldg(src + u * TX) : zero_unit<U>();
        for (int j = 0; j < k; ++j) {
            const int64_t r = entry_row(pos, t * k + j, R);
            if (r < 0) continue;
            U *dst = rows + r * units + c;
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                if (c + u * TX < units) dst[u * TX] = v[u];
        }
    }
}

// y[t] = residual[t] + sum_j w[t,j] * rows[pos[t,j]], slot order, float32, rounded
// once.  Two slots' rows are loaded together, with the residual's.  What counts is loads in
// flight over all warps of an SM: 16384 x 4096 bf16, top-2, takes 81 us with two
// accesses of 16 bytes a thread and 32 warps an SM, 91 with four and 16 warps, 98 with four
// and 24 (spills), 153 with four slots at a time and 8; without a residual four accesses
// leave room for 24 warps (59 us, the bytes' floor).  Rows that arrive by bulk copies in a
// ring of shared-memory stages were no faster (91 us, half as fast on 1001-float rows).
// residual and y may be the same array: an element is read and written by the same
// thread.
template <int TX, class U, bool BF16, bool RES>
__global__ void __launch_bounds__(kMoveThreads, sizeof(U) == 16 && RES ? 8 : 6)
unpermute_kernel(const U *__restrict__ rows, const int *__restrict__ pos, const float *__restrict__ weights,
                 const U *residual, int64_t T, int k, int R, int units, int parts, U *y) {
    using V = Vals<U, BF16>;
    constexpr int kPer = kPerUnOf<U, RES>;
    griddep_enter();
    const int64_t t = static_cast<int64_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    if (t >= T) return;
    const float *wt = weights + t * k;
    const int step = parts * kPer * TX;
    for (int c = static_cast<int>(blockIdx.x % parts) * kPer * TX + threadIdx.x; c < units; c += step) {
        float acc[kPer][V::N];
        U res[kPer];
        const U *rp = residual + t * units + c;
#pragma unroll
        for (int u = 0; u < kPer; ++u) res[u] = RES && c + u * TX < units ? rp[u * TX] : zero_unit<U>();
        for (int j = 0; j < k; j += 2) {
            const int ra = entry_row(pos, t * k + j, R), rb = j + 1 < k ? entry_row(pos, t * k + j + 1, R) : -1;
            const float wa = weights ? wt[j] : 1.0f;
            const float wb = weights && j + 1 < k ? wt[j + 1] : 1.0f;
            const U *pa = rows + static_cast<int64_t>(ra < 0 ? 0 : ra) * units + c;
            const U *pb = rows + static_cast<int64_t>(rb < 0 ? 0 : rb) * units + c;
            U oa[kPer], ob[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                oa[u] = c + u * TX < units && ra >= 0 ? __ldg(pa + u * TX) : zero_unit<U>();
                ob[u] = c + u * TX < units && rb >= 0 ? __ldg(pb + u * TX) : zero_unit<U>();
            }
            if (j == 0) {
#pragma unroll
                for (int u = 0; u < kPer; ++u) V::get(res[u], acc[u]);
            }
            if (ra >= 0) {
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    float f[V::N];
                    V::get(oa[u], f);
#pragma unroll
                    for (int i = 0; i < V::N; ++i) acc[u][i] += wa * f[i];
                }
            }
            if (rb >= 0) {
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    float f[V::N];
                    V::get(ob[u], f);
#pragma unroll
                    for (int i = 0; i < V::N; ++i) acc[u][i] += wb * f[i];
                }
            }
        }
        U *yp = y + t * units + c;
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            if (c + u * TX < units) yp[u * TX] = V::put(acc[u]);
    }
}

// d_rows[pos[t,j]] = w[t,j] * dy[t] and dw[t,j] = <dy[t], rows[pos[t,j]]>.  The rows of
// kSlots slots are loaded together with dy; a dot product is summed over the row's
// threads by shuffles, then over its warps in warp order.  d_weights NULL skips the
// products and rows.
template <int TX, class U, bool BF16>
__global__ void __launch_bounds__(kMoveThreads)
unpermute_bwd_kernel(const U *__restrict__ dy, const U *__restrict__ rows, const int *__restrict__ pos,
                     const int *__restrict__ count, const int *__restrict__ seg, const float *__restrict__ weights,
                     int64_t T, int k, int experts, int slices, int R, int units, int parts, int64_t token_blocks,
                     U *__restrict__ d_rows, float *__restrict__ d_weights) {
    using V = Vals<U, BF16>;
    constexpr int kPerBwd = kPerBwdOf<U>;
    constexpr int kWarps = TX / 32;  // of a row
    __shared__ float part[2][kSlots][kMoveThreads / 32];
    griddep_enter();
    const int64_t b = blockIdx.x;
    if (b >= token_blocks) {
        zero_padding(d_rows, units, b - token_blocks, slices, experts, count, seg, R);
        return;
    }
    const int64_t t = static_cast<int64_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    const bool in = t < T;
    const int w0 = threadIdx.y * kWarps;
    for (int j0 = static_cast<int>(blockIdx.x % parts) * kSlots, group = 0; j0 < k; j0 += parts * kSlots, ++group) {
        float s[kSlots];
        int r[kSlots];
        float w[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const bool on = in && j0 + j < k;
            s[j] = 0.0f;
            r[j] = on ? entry_row(pos, t * k + j0 + j, R) : -1;
            w[j] = on && weights ? weights[t * k + j0 + j] : 1.0f;
        }
        for (int c = threadIdx.x; in && c < units; c += kPerBwd * TX) {
            const U *gp = dy + t * units + c;
            U g[kPerBwd], o[kSlots][kPerBwd];
#pragma unroll
            for (int u = 0; u < kPerBwd; ++u) g[u] = c + u * TX < units ? __ldg(gp + u * TX) : zero_unit<U>();
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                const U *rp = rows + static_cast<int64_t>(r[j] < 0 ? 0 : r[j]) * units + c;
                const bool use = d_weights && r[j] >= 0;
#pragma unroll
                for (int u = 0; u < kPerBwd; ++u) o[j][u] = use && c + u * TX < units ? __ldg(rp + u * TX) : zero_unit<U>();
            }
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (r[j] < 0) continue;
                U *dp = d_rows + static_cast<int64_t>(r[j]) * units + c;
#pragma unroll
                for (int u = 0; u < kPerBwd; ++u) {
                    float a[V::N], f[V::N];
                    V::get(g[u], a);
                    V::get(o[j][u], f);
#pragma unroll
                    for (int i = 0; i < V::N; ++i) {
                        s[j] += a[i] * f[i];
                        f[i] = a[i] * w[j];
                    }
                    if (c + u * TX < units) dp[u * TX] = V::put(f);
                }
            }
        }
        if (!d_weights) continue;
        const int buf = group & 1;
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
            if ((threadIdx.x & 31) == 0) part[buf][j][w0 + threadIdx.x / 32] = s[j];
        }
        __syncthreads();  // one barrier a group of slots: the next group writes the other half of `part`
        if (in && threadIdx.x < kSlots && j0 + threadIdx.x < k) {
            float d = 0.0f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) d += part[buf][threadIdx.x][w0 + q];
            d_weights[t * k + j0 + threadIdx.x] = d;
        }
    }
}

// The shape of a move: bytes of an access, accesses of a row, threads of a row, CTAs of
// the tokens (`parts` of them share a row's columns, or its slots) and of the padding.
struct MoveShape {
    int unit, units;
    int tx;
    int parts, slices;
    dim3 block;
    int64_t token_blocks, pad_blocks;
};

// Up to kFewBlocks CTAs, about one an SM, the columns (`slots` 0) or groups of slots of a
// row are dealt out to several, so that few tokens with long rows do not wait for one
// access after another (20 tokens of 3051 bf16, top-7: unpermute 26.5 -> 11.1 us, its
// gradient 34.3 -> 23.9).  A slice of padding has about kSliceBytes.
constexpr int64_t kFewBlocks = 152;
constexpr int64_t kSliceBytes = 32768;

MoveShape move_shape(int64_t T, int64_t width, int dtype, int experts, int pad, int per16, int per4, int per2, int step16,
                     int slots) {
    MoveShape m;
    const int64_t bytes = width * (dtype == MLPBLK_BF16 ? 2 : 4);
    m.unit = bytes % 16 == 0 ? 16 : (bytes % 4 == 0 ? 4 : 2);
    m.units = static_cast<int>(bytes / m.unit);
    const int p = m.unit == 16 ? per16 : (m.unit == 4 ? per4 : per2);
    m.tx = m.units <= 32 * p ? 32 : (m.units <= 64 * p ? 64 : 128);
    m.block = dim3(m.tx, kMoveThreads / m.tx, 1);
    const int64_t blocks = (T + m.block.y - 1) / m.block.y;
    const int64_t step = static_cast<int64_t>(m.tx) * (m.unit == 16 ? step16 : p);
    const int64_t steps = slots ? slots : (m.units + step - 1) / step;
    m.parts = static_cast<int>(std::max<int64_t>(1, std::min(steps, kFewBlocks / std::max<int64_t>(1, blocks))));
    m.token_blocks = blocks * m.parts;
    m.slices = pad > 1 ? static_cast<int>(std::min<int64_t>(pad - 1, ((pad - 1) * bytes + kSliceBytes - 1) / kSliceBytes)) : 0;
    m.pad_blocks = static_cast<int64_t>(experts) * m.slices;
    return m;
}

}  // namespace

int launch_sort(const int *idx, int64_t n, int experts, int pad, int64_t R, int *count, int *seg, int *pos,
                int *row_map, cudaStream_t s) {
    const int C = n <= kSortOneCta && R <= kSortOneRows ? 1 : kSortCluster;
    const int warps = n <= kSortSmall && R <= kSortSmallRows ? 8 : 32;
    int64_t per_warp = (n + static_cast<int64_t>(C) * warps - 1) / (static_cast<int64_t>(C) * warps);
    per_warp = (per_warp + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    auto kern = warps == 8 ? sort_kernel<8> : sort_kernel<32>;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, idx, n, experts, pad, R, per_warp, count, seg, pos, row_map));
}

int launch_permute(const void *x, const int *pos, const int *count, const int *seg, int64_t T, int64_t width,
                   int dtype, int k, int experts, int pad, int64_t R, void *rows, cudaStream_t s) {
    const MoveShape m = move_shape(T, width, dtype, experts, pad, kPerOf<uint4>, kPerOf<uint32_t>, kPerOf<uint16_t>, kPerOf<uint4>, 0);
    const dim3 grid(static_cast<unsigned>(m.token_blocks + m.pad_blocks));
#define MLPBLK_PERMUTE(U)                                                                                      \
    return launch_pdl(m.tx == 32 ? permute_kernel<32, U> : m.tx == 64 ? permute_kernel<64, U> : permute_kernel<128, U>, grid, m.block, 0, s,         \
                      static_cast<const U *>(x), pos, count, seg, T, k,                                        \
                      experts, m.slices, static_cast<int>(R), m.units, m.parts, m.token_blocks, static_cast<U *>(rows))
    if (m.unit == 16) MLPBLK_PERMUTE(uint4);
    if (m.unit == 4) MLPBLK_PERMUTE(uint32_t);
    MLPBLK_PERMUTE(uint16_t);
#undef MLPBLK_PERMUTE
}

int launch_unpermute(const void *rows, const int *pos, const float *weights, const void *residual, int64_t T,
                     int64_t width, int dtype, int k, int64_t R, void *y, cudaStream_t s) {
    const MoveShape m = move_shape(T, width, dtype, 1, 1, kPerOf<uint4>, kPerOf<uint32_t>, kPerOf<uint16_t>,
                                   residual ? kPerUnOf<uint4, true> : kPerUnOf<uint4, false>, 0);
    const dim3 grid(static_cast<unsigned>(m.token_blocks));
#define MLPBLK_UNPERMUTE_R(U, B, RES)                                                                        \
    return launch_pdl(m.tx == 32 ? unpermute_kernel<32, U, B, RES>                                           \
                      : m.tx == 64 ? unpermute_kernel<64, U, B, RES> : unpermute_kernel<128, U, B, RES>,     \
                      grid, m.block, 0, s, static_cast<const U *>(rows), pos, weights,                       \
                      static_cast<const U *>(residual), T, k, static_cast<int>(R), m.units, m.parts, static_cast<U *>(y))
#define MLPBLK_UNPERMUTE(U, B)                  \
    if (residual) MLPBLK_UNPERMUTE_R(U, B, true); \
    MLPBLK_UNPERMUTE_R(U, B, false)
    if (dtype == MLPBLK_BF16) {
        if (m.unit == 16) {
            MLPBLK_UNPERMUTE(uint4, true);
        }
        if (m.unit == 4) {
            MLPBLK_UNPERMUTE(uint32_t, true);
        }
        MLPBLK_UNPERMUTE(uint16_t, true);
    }
    if (m.unit == 16) {
        MLPBLK_UNPERMUTE(uint4, false);
    }
    MLPBLK_UNPERMUTE(uint32_t, false);
#undef MLPBLK_UNPERMUTE
#undef MLPBLK_UNPERMUTE_R
}

int launch_unpermute_bwd(const void *dy, const void *rows, const int *pos, const int *count, const int *seg,
                         const float *weights, int64_t T, int64_t width, int dtype, int k, int experts, int pad, int64_t R,
                         void *d_rows, float *d_weights, cudaStream_t s) {
    const MoveShape m = move_shape(T, width, dtype, experts, pad, kPerBwdOf<uint4>, kPerBwdOf<uint32_t>, kPerBwdOf<uint16_t>, kPerBwdOf<uint4>,
                                   (k + kSlots - 1) / kSlots);
    const dim3 grid(static_cast<unsigned>(m.token_blocks + m.pad_blocks));
#define MLPBLK_UNPERMUTE_BWD(U, B)                                                                               \
    return launch_pdl(m.tx == 32 ? unpermute_bwd_kernel<32, U, B>                                                \
                      : m.tx == 64 ? unpermute_bwd_kernel<64, U, B> : unpermute_bwd_kernel<128, U, B>,           \
                      grid, m.block, 0, s, static_cast<const U *>(dy),                                           \
                      static_cast<const U *>(rows), pos, count, seg, weights, T, k, experts, m.slices, static_cast<int>(R), m.units,  \
                      m.parts, m.token_blocks, static_cast<U *>(d_rows), d_weights)
    if (dtype == MLPBLK_BF16) {
        if (m.unit == 16) MLPBLK_UNPERMUTE_BWD(uint4, true);
        if (m.unit == 4) MLPBLK_UNPERMUTE_BWD(uint32_t, true);
        MLPBLK_UNPERMUTE_BWD(uint16_t, true);
    }
    if (m.unit == 16) MLPBLK_UNPERMUTE_BWD(uint4, false);
    MLPBLK_UNPERMUTE_BWD(uint32_t, false);
#undef MLPBLK_UNPERMUTE_BWD
}

}  // namespace mlpblk
