// api.cu -- the C ABI (include/mlpblk.h): argument checks, workspace layout and
// the order of kernels for one microbatch forward and backward.
//
// Forward  (bf16): fold gamma into W1 -> W1 GEMM (rstd prologue, h/a epilogue)
//                  -> W2 GEMM (residual epilogue)
// Backward (bf16): wgrad W2 GEMM (+=) -> dgrad-h GEMM (gate, dh_s = rstd*dh)
//                  -> dgrad-n GEMM (dn_s = rstd*dn, bf16) -> wgrad W1 GEMM (+= , gamma)
//                  -> RMSNorm backward rows (dx, dgamma partials) -> dgamma (+=)
//                  (d_model <= 768: the rows and the dgamma sum run on the
//                  wgrad-W1 GEMM's side warps)
// The fp32 element type runs the same sequence on CUDA cores.
#include <math.h>
#include <stdlib.h>

#include <initializer_list>
#include <new>

#include "fp4_layout.h"
#include "mlpblk_internal.h"
#include "ortho.h"

namespace mlpblk {
int launch_gemm_tc_fwd(int epi, int M, int N, int K, const void *A, const void *B, void *C0,
                       void *C1, const GemmArgs &extra, int num_sms, cudaStream_t s);
int launch_gemm_tc_bwd(int epi, int M, int N, int K, const void *A, const void *B, void *C0,
                       void *C1, const GemmArgs &extra, int num_sms, cudaStream_t s);
int take_device_error_gemm_fwd();
int take_device_error_gemm_bwd();
}  // namespace mlpblk

namespace mlpblk {
int g_last_cuda_error = 0;
}  // namespace mlpblk

using namespace mlpblk;

namespace {

constexpr int kMaxParts = 512;  // dgamma partial rows the workspace holds

int64_t align256(int64_t b) { return (b + 255) & ~static_cast<int64_t>(255); }

int check_desc(const mlpblk_desc *d) {
    if (!d) return MLPBLK_EINVAL;
    if (d->dtype != MLPBLK_BF16 && d->dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->tokens < 0 || d->d_model <= 0 || d->ffn <= 0) return MLPBLK_EINVAL;
    if (d->d_model % 8 != 0 || d->ffn % 8 != 0) return MLPBLK_ENOTSUP;
    if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return MLPBLK_EINVAL;
    const int64_t lim = static_cast<int64_t>(1) << 31;
    const int64_t wide = d->d_model > d->ffn ? d->d_model : d->ffn;
    if (d->ffn >= lim / d->d_model) return MLPBLK_EINVAL;
    if (d->tokens >= lim / wide) return MLPBLK_EINVAL;
    if (d->d_model > kMaxNormD) return MLPBLK_ENOTSUP;
    return MLPBLK_OK;
}

bool aligned16(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct WsLayout {
    int64_t w1g, dh, h, a, dn, part, sk_partial, sk_flags, total;
};

// Stream-K flag sets, one per tensor-core GEMM that can split a tile; each set
// is zeroed by the kernel launched just before that GEMM.
// kSetSide: the wgrad-W1 side warps' arrival count (its first word).
enum SkFlagSet : int { kSetFwdW1 = 0, kSetFwdW2 = 1, kSetDgradH = 2, kSetDgradN = 3, kSetSide = 4, kSkSets = 5 };

// Workspace regions.  W1*gamma (forward, and the recompute backward's first
// GEMM) shares its region with dh_s (backward).  `recompute` adds the T x F
// h and a that the recompute variant keeps in the workspace instead of saving.
WsLayout ws_layout(const mlpblk_desc *d, bool recompute) {
    const int64_t elt = d->dtype == MLPBLK_BF16 ? 2 : 4;
    const int64_t tf = align256(d->tokens * d->ffn * elt);
    const int64_t fd = align256(d->ffn * d->d_model * elt);
    WsLayout l;
    l.w1g = 0;
    l.dh = 0;
    int64_t off = recompute ? (tf > fd ? tf : fd) : tf;
    l.h = recompute ? off : -1;
    if (recompute) off += tf;
    l.a = recompute ? off : -1;
    if (recompute) off += tf;
    l.dn = off;
    l.part = l.dn + align256(d->tokens * d->d_model * elt);  // dn_s in the block dtype
    const int64_t bwd = l.part + align256(static_cast<int64_t>(kMaxParts) * d->d_model * 4);
    // the GEMMs' stream-K partial sums and flags, apart from everything above
    l.sk_partial = fd > bwd ? fd : bwd;
    l.sk_flags = l.sk_partial + align256(static_cast<int64_t>(kMaxSkSlots) * kSkSlotFloats * 4);
    l.total = l.sk_flags + align256(static_cast<int64_t>(kSkSets) * kSkFlagsPerSet * 4);
    return l;
}

// Workspace of the FP8-operand variant (forward and backward regions overlap
// where they are never live together).
struct WsLayoutF8 {
    int64_t t16;   // a (forward) or dh (backward), bf16 [T, F]
    int64_t dh8;   // dh in E4M3 [T, F]
    int64_t w1q;   // W1*gamma (forward) or W1 (backward) in E4M3 [F, d]
    int64_t w2q;   // W2 in E4M3 [d, F]
    int64_t dyq;   // dy in E4M3 [T, d]
    int64_t dn;    // dn_s fp32 [T, d]
    int64_t part;  // dgamma partials [kMaxParts, d]
    int64_t amax;  // per-CTA maxima of the amax passes
    int64_t scales;  // scale records: 0 W1, 1 W2, 2 dy, 3 dh
    int64_t sk_partial, sk_flags, total;
};

constexpr int kAmaxParts = 2048;
static_assert(kAmaxParts >= kMaxSkSlots * kMaxEpiWarps, "the GEMM epilogues' maxima fit the amax scratch");

WsLayoutF8 ws_layout_f8(const mlpblk_desc *dsc) {
    const int64_t T = dsc->tokens, d = dsc->d_model, F = dsc->ffn;
    WsLayoutF8 l;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = off;
        off += align256(bytes);
        return at;
    };
    l.t16 = take(T * F * 2);
    l.dh8 = take(T * F);
    l.w1q = take(F * d);
    l.w2q = take(d * F);
    l.dyq = take(T * d);
    l.dn = take(T * d * 4);
    l.part = take(static_cast<int64_t>(kMaxParts) * d * 4);
    l.amax = take(kAmaxParts * 4);
    l.scales = take(4 * 16);
    l.sk_partial = take(static_cast<int64_t>(kMaxSkSlots) * kSkSlotFloats * 4);
    l.sk_flags = take(static_cast<int64_t>(kSkSets) * kSkFlagsPerSet * 4);
    l.total = off;
    return l;
}

// Device properties, checked once per device: sm_103 and its SM count.
int device_sms(int *sms) {
    static int cached[64] = {0};  // 0 unknown, -1 unsupported, else SM count
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != MLPBLK_OK || dev < 0 || dev >= 64) return MLPBLK_ECUDA;
    if (cached[dev] == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return MLPBLK_ECUDA;
        cached[dev] = (major == 10 && minor == 3 && n > 0) ? n : -1;
    }
    if (cached[dev] < 0) return MLPBLK_ENODEV;
    // MLPBLK_MAX_SMS caps the SMs the GEMMs spread over (an even count, to leave
    // SMs to concurrent work); unset, they use every SM
    static int cap = -1;
    if (cap < 0) {
        const char *e = getenv("MLPBLK_MAX_SMS");
        const int v = e ? atoi(e) : 0;
        cap = v >= 2 ? (v & ~1) : 0;
    }
    *sms = (cap > 0 && cap < cached[dev]) ? cap : cached[dev];
    return MLPBLK_OK;
}

#define MLPBLK_TRY(expr)              \
    do {                              \
        const int rc_ = (expr);       \
        if (rc_ != MLPBLK_OK) return rc_; \
    } while (0)

// Launch trace (mlpblk_trace_begin/end): caller-owned events around each launch.
struct Trace {
    cudaEvent_t *events = nullptr;
    int *kinds = nullptr;
    int capacity = 0;
    int count = 0;
    bool on = false;
} g_trace;

}  // namespace

namespace mlpblk {
// Where the forward's RMSNorm statistic is computed (mlpblk_set_rmsnorm_mode);
// the environment variable MLPBLK_RMS_IN_GEMM=1 sets the initial mode.
int g_rms_mode = -1;

bool rms_in_gemm() {
    if (g_rms_mode < 0) {
        const char *e = getenv("MLPBLK_RMS_IN_GEMM");
        g_rms_mode = (e && e[0] == '1') ? MLPBLK_RMSNORM_IN_W1_PROLOGUE : MLPBLK_RMSNORM_STATS_PASS;
    }
    return g_rms_mode == MLPBLK_RMSNORM_IN_W1_PROLOGUE;
}
}  // namespace mlpblk

namespace {

// The bf16 backward runs the RMSNorm backward rows on the wgrad-W1 GEMM's side
// warps when d_model <= kSideNormMaxD, unless MLPBLK_SIDE_NORM=0 selects the
// separate row kernel (both paths are parity-tested).
bool side_norm(int64_t d) {
    static int v = -1;
    if (v < 0) {
        const char *e = getenv("MLPBLK_SIDE_NORM");
        v = (e && e[0] == '0') ? 0 : 1;
    }
    return v == 1 && d <= kSideNormMaxD;
}

// One-shot test fault (mlpblk_set_test_fault): consumed by the next bf16 forward.
int g_test_fault = 0;

int take_test_fault() {
    const int f = g_test_fault;
    g_test_fault = 0;
    return f == MLPBLK_TEST_FAULT_SKIP_LOADS ? 1 : 0;
}

// Runs one launcher, bracketed by the trace events when a trace is active.
template <class F>
int traced(int kind, cudaStream_t s, F &&launch) {
    if (!g_trace.on) return launch();
    const int i = g_trace.count++;
    const bool rec = i < g_trace.capacity;
    // under stream capture the records become external event nodes, which keep
    // their timestamps when the graph is replayed
    unsigned int flags = cudaEventRecordDefault;
    if (rec) {
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        MLPBLK_TRY(cuda_status(cudaStreamIsCapturing(s, &cs)));
        if (cs == cudaStreamCaptureStatusActive) flags = cudaEventRecordExternal;
        g_trace.kinds[i] = kind;
        MLPBLK_TRY(cuda_status(cudaEventRecordWithFlags(g_trace.events[2 * i], s, flags)));
    }
    MLPBLK_TRY(launch());
    if (rec) MLPBLK_TRY(cuda_status(cudaEventRecordWithFlags(g_trace.events[2 * i + 1], s, flags)));
    return MLPBLK_OK;
}

#define MLPBLK_LAUNCH(kind, stream, call) MLPBLK_TRY(traced(kind, stream, [&]() { return (call); }))


}  // namespace

extern "C" {

int mlpblk_version(void) { return 102; }

const char *mlpblk_strerror(int code) {
    switch (code) {
        case MLPBLK_OK: return "success";
        case MLPBLK_EINVAL: return "invalid argument (null or misaligned pointer, bad size or eps)";
        case MLPBLK_ENOTSUP: return "unsupported dtype or shape (d_model, ffn multiples of 8; d_model <= 4096)";
        case MLPBLK_EWORKSPACE: return "workspace smaller than mlpblk_workspace_size()";
        case MLPBLK_ECUDA: return "CUDA runtime error or kernel launch failure";
        case MLPBLK_ETIMEOUT: return "a device-side bounded wait gave up; outputs are invalid";
        case MLPBLK_ENODEV: return "current device is not sm_103 (GB300)";
        default: return "unknown mlpblk status code";
    }
}

size_t mlpblk_workspace_size(const mlpblk_desc *desc) {
    if (check_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(ws_layout(desc, false).total);
}

}  // extern "C"

namespace {

// The forward's launches.  h_out may be null on the bf16 path (a_only: the
// recompute variant's forward, whose W1 epilogue writes a alone).
// prefolded: w1g already holds W1 * gamma (mlpblk_fold_weights); gamma and w1
// are not read.
int forward_impl(const mlpblk_desc *desc, const void *x, const void *gamma, const void *w1,
                 const void *w2, void *y, void *h_out, void *a_out, float *rstd_saved, void *w1g,
                 float *sk_partial, int *sk_flags, int sms, cudaStream_t s, bool a_only,
                 bool prefolded = false) {
    const int64_t T = desc->tokens, d = desc->d_model, F = desc->ffn;
    const bool stats_in_gemm = desc->dtype == MLPBLK_BF16 && !a_only && rms_in_gemm();
    if (stats_in_gemm) {
        // rstd inside the W1 GEMM (whole tiles: no stream-K flags to clear)
        if (!prefolded)
            MLPBLK_LAUNCH(MLPBLK_KERNEL_FOLD_GAMMA, s,
                          launch_fold_gamma(desc->dtype, w1, gamma, w1g, F, d, nullptr, 0, s));
    } else {
        // rstd, and W1 * gamma unless it is given
        MLPBLK_LAUNCH(prefolded ? MLPBLK_KERNEL_RSTD : MLPBLK_KERNEL_FOLD_GAMMA, s,
                      launch_norm_prep(desc->dtype, x, rstd_saved, T, d, desc->eps, prefolded ? nullptr : w1,
                                       gamma, prefolded ? nullptr : w1g, prefolded ? 0 : F,
                                       sk_flags + kSetFwdW1 * kSkFlagsPerSet, kSkFlagsPerSet, s));
    }
    if (desc->dtype == MLPBLK_BF16) {
        GemmArgs g1 = {};
        if (stats_in_gemm) {
            g1.rstd_out = rstd_saved;
            g1.inv_k = 1.0f / static_cast<float>(d);
            g1.eps = desc->eps;
        } else {
            g1.rstd_in = rstd_saved;
        }
        g1.skip_loads = take_test_fault();
        g1.sk_partial = sk_partial;
        g1.sk_flags = sk_flags + kSetFwdW1 * kSkFlagsPerSet;
        g1.zero_flags = sk_flags + kSetFwdW2 * kSkFlagsPerSet;
        const int epi1 = a_only ? kEpiFwdW1A : (stats_in_gemm ? kEpiFwdW1 : kEpiFwdW1Pre);
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W1, s,
                      launch_gemm_tc_fwd(epi1, (int)T, (int)F, (int)d, x, w1g, a_only ? a_out : h_out,
                                         a_only ? nullptr : a_out, g1, sms, s));
        GemmArgs g2 = {};
        g2.aux = static_cast<const uint16_t *>(x);
        g2.ld_aux = (int)d;
        g2.sk_partial = sk_partial;
        g2.sk_flags = sk_flags + kSetFwdW2 * kSkFlagsPerSet;
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W2, s, launch_gemm_tc_fwd(kEpiFwdW2, (int)T, (int)d, (int)F, a_out, w2, y, nullptr, g2, sms, s));
    } else {
        const float *xf = static_cast<const float *>(x);
        SimtEpi e1 = {nullptr, rstd_saved, nullptr};
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W1, s, launch_gemm_simt(kEpiFwdW1, (int)T, (int)F, (int)d, xf, d, 1,
                                    static_cast<const float *>(w1g), d, 1,
                                    static_cast<float *>(h_out), static_cast<float *>(a_out), e1, s));
        SimtEpi e2 = {xf, nullptr, nullptr};
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W2, s, launch_gemm_simt(kEpiFwdW2, (int)T, (int)d, (int)F,
                                    static_cast<const float *>(a_out), F, 1,
                                    static_cast<const float *>(w2), F, 1, static_cast<float *>(y),
                                    nullptr, e2, s));
    }
    return MLPBLK_OK;
}

// The backward's launches, from saved (or recomputed) h and a.
int backward_impl(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                  const void *w1, const void *w2, const void *h_saved, const void *a_saved,
                  const float *rstd_saved, void *dx, float *dgamma, float *dw1, float *dw2,
                  void *dh_s, void *dn_s, float *part, float *sk_partial, int *sk_flags, int sms,
                  cudaStream_t s, bool overwrite) {
    const int64_t T = desc->tokens, d = desc->d_model, F = desc->ffn;
    int parts = 0;  // dgamma partial rows written by the norm kernel
    if (desc->dtype == MLPBLK_BF16) {
        // dW2 first: it needs no flags and zeroes the dgrad-h GEMM's.  The two
        // independent pairs (dW2, dh) and (dn, dW1) overlap at their boundary:
        // the second of each starts on the SMs the first frees without waiting
        // for all of it (kPdlDeferWait), which the first allows by launching it
        // only after its own predecessor has completed (kPdlWaitFirst)
        GemmArgs gw2 = {};
        gw2.zero_flags = sk_flags + kSetDgradH * kSkFlagsPerSet;
        gw2.pdl = kPdlWaitFirst;
        GemmArgs gd = {};
        gd.aux = static_cast<const uint16_t *>(h_saved);
        gd.ld_aux = (int)F;
        gd.rstd_in = rstd_saved;
        gd.sk_partial = sk_partial;
        gd.sk_flags = sk_flags + kSetDgradH * kSkFlagsPerSet;
        gd.zero_flags = sk_flags + kSetDgradN * kSkFlagsPerSet;
        gd.pdl = kPdlDeferWait;
        GemmArgs gn = {};
        gn.sk_partial = sk_partial;
        gn.sk_flags = sk_flags + kSetDgradN * kSkFlagsPerSet;
        gn.zero_flags = side_norm(d) ? sk_flags + kSetSide * kSkFlagsPerSet : nullptr;
        gn.pdl = kPdlWaitFirst;
        GemmArgs gw1 = {};
        gw1.colscale = static_cast<const uint16_t *>(gamma);
        gw1.pdl = kPdlDeferWait;
        const bool side = side_norm(d);
        if (side) {
            // the RMSNorm backward rows run on the wgrad-W1 GEMM's side warps,
            // one dgamma partial row per CTA of that launch, summed into dgamma
            // by the same warps once every CTA's row is complete
            gw1.side.x = static_cast<const uint16_t *>(x);
            gw1.side.dy = static_cast<const uint16_t *>(dy);
            gw1.side.gamma = static_cast<const uint16_t *>(gamma);
            gw1.side.dn_s = static_cast<const uint16_t *>(dn_s);
            gw1.side.rstd = rstd_saved;
            gw1.side.dx = static_cast<uint16_t *>(dx);
            gw1.side.part = part;
            gw1.side.dgamma = dgamma;
            gw1.side.arrive = sk_flags + kSetSide * kSkFlagsPerSet;
            gw1.side.T = T;
            gw1.side.d = (int)d;
            gw1.grid_out = &parts;
        }
        const int epi_w1 = side ? kEpiAccF32ColScaleNorm : kEpiAccF32ColScale;
        if (overwrite) {
            // = instead of +=: the weight-gradient GEMMs store every tile one
            // worker sums whole, and add the split tiles' parts into regions
            // that one small launch clears first (with dgamma, which the norm
            // backward then adds into).  It runs before dW2's GEMM, whose
            // completion dW1's GEMM follows through the chain of waits above.
            gw2.overwrite = 1;
            gw1.overwrite = 1;
            GemmArgs plan2 = {}, plan1 = {};
            GemmArgs q2 = gw2, q1 = gw1;
            q2.plan_out = &plan2;
            q1.plan_out = &plan1;
            MLPBLK_TRY(launch_gemm_tc_bwd(kEpiAccF32, (int)d, (int)F, (int)T, dy, a_saved, dw2, nullptr, q2, sms, s));
            MLPBLK_TRY(launch_gemm_tc_bwd(epi_w1, (int)F, (int)d, (int)T, dh_s, x, dw1, nullptr, q1, sms, s));
            MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s,
                          launch_zero_split_tiles(split_tiles_of(plan2, dw2, F), split_tiles_of(plan1, dw1, d),
                                                  dgamma, d, s));
        }
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W2, s, launch_gemm_tc_bwd(kEpiAccF32, (int)d, (int)F, (int)T, dy, a_saved, dw2, nullptr, gw2, sms, s));
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_H, s, launch_gemm_tc_bwd(kEpiDgradH, (int)T, (int)F, (int)d, dy, w2, dh_s, nullptr, gd, sms, s));
        // dn_s = rstd * dn stored in bf16 like dh_s (rstd rides in dh_s already)
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_N, s, launch_gemm_tc_bwd(kEpiStoreBf16, (int)T, (int)d, (int)F, dh_s, w1, dn_s, nullptr, gn, sms, s));
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W1, s, launch_gemm_tc_bwd(epi_w1, (int)F, (int)d, (int)T, dh_s, x, dw1, nullptr, gw1, sms, s));
        if (side) {
            if (parts <= 0 || parts > kMaxParts) return MLPBLK_ECUDA;
            return MLPBLK_OK;
        }
    } else {
        // CUDA-core path, = instead of +=: the gradients are cleared, then added into
        if (overwrite)
            MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s,
                          launch_grads(true, 0.0f, dgamma, d, dw1, F * d, dw2, d * F, s));
        const float *dyf = static_cast<const float *>(dy);
        const float *xf = static_cast<const float *>(x);
        const float *dhf = static_cast<const float *>(dh_s);
        SimtEpi ed = {static_cast<const float *>(h_saved), rstd_saved, nullptr};
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_H, s, launch_gemm_simt(kEpiDgradH, (int)T, (int)F, (int)d, dyf, d, 1,
                                    static_cast<const float *>(w2), 1, F, static_cast<float *>(dh_s),
                                    nullptr, ed, s));
        SimtEpi e0 = {nullptr, nullptr, nullptr};
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W2, s, launch_gemm_simt(kEpiAccF32, (int)d, (int)F, (int)T, dyf, 1, d,
                                    static_cast<const float *>(a_saved), 1, F, dw2, nullptr, e0, s));
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_N, s, launch_gemm_simt(kEpiStoreF32, (int)T, (int)d, (int)F, dhf, F, 1,
                                    static_cast<const float *>(w1), 1, d, static_cast<float *>(dn_s), nullptr, e0, s));
        SimtEpi ec = {nullptr, nullptr, static_cast<const float *>(gamma)};
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W1, s, launch_gemm_simt(kEpiAccF32ColScale, (int)F, (int)d, (int)T, dhf, 1, F, xf, 1, d,
                                    dw1, nullptr, ec, s));
    }
    MLPBLK_LAUNCH(MLPBLK_KERNEL_NORM_BWD, s, launch_rmsnorm_bwd(desc->dtype, x, dn_s, desc->dtype == MLPBLK_BF16, dy, rstd_saved, gamma, dx, part, T, d, kMaxParts, &parts, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_DGAMMA_REDUCE, s, launch_dgamma_finalize(part, parts, dgamma, d, s));
    return MLPBLK_OK;
}

}  // namespace

extern "C" {

int mlpblk_forward(const mlpblk_desc *desc, const void *x, const void *gamma, const void *w1,
                   const void *w2, void *y, void *h_saved, void *a_saved, float *rstd_saved,
                   void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(w1) || !aligned16(w2) || !aligned16(y) ||
        !aligned16(h_saved) || !aligned16(a_saved) || !aligned16(rstd_saved) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (y == x) return MLPBLK_EINVAL;
    const WsLayout l = ws_layout(desc, false);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return forward_impl(desc, x, gamma, w1, w2, y, h_saved, a_saved, rstd_saved, ws + l.w1g,
                        reinterpret_cast<float *>(ws + l.sk_partial), reinterpret_cast<int *>(ws + l.sk_flags),
                        sms, static_cast<cudaStream_t>(stream), false);
}

}  // extern "C"

namespace {

int backward_entry(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                   const void *w1, const void *w2, const void *h_saved, const void *a_saved,
                   const float *rstd_saved, void *dx, float *dgamma, float *dw1, float *dw2,
                   void *workspace, size_t workspace_bytes, void *stream, bool overwrite) {
    MLPBLK_TRY(check_desc(desc));
    if (desc->tokens == 0) {
        // no rows: += adds nothing; = leaves zero gradients
        if (!overwrite) return MLPBLK_OK;
        if (!aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2)) return MLPBLK_EINVAL;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const int64_t d = desc->d_model, F = desc->ffn;
        MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s, launch_grads(true, 0.0f, dgamma, d, dw1, F * d, dw2, d * F, s));
        return MLPBLK_OK;
    }
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(w1) || !aligned16(w2) ||
        !aligned16(h_saved) || !aligned16(a_saved) || !aligned16(rstd_saved) || !aligned16(dx) ||
        !aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (dx == dy || dx == x) return MLPBLK_EINVAL;
    const WsLayout l = ws_layout(desc, false);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return backward_impl(desc, dy, x, gamma, w1, w2, h_saved, a_saved, rstd_saved, dx, dgamma, dw1, dw2,
                         ws + l.dh, ws + l.dn, reinterpret_cast<float *>(ws + l.part),
                         reinterpret_cast<float *>(ws + l.sk_partial), reinterpret_cast<int *>(ws + l.sk_flags),
                         sms, static_cast<cudaStream_t>(stream), overwrite);
}

}  // namespace

extern "C" {

int mlpblk_backward(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                    const void *w1, const void *w2, const void *h_saved, const void *a_saved,
                    const float *rstd_saved, void *dx, float *dgamma, float *dw1, float *dw2,
                    void *workspace, size_t workspace_bytes, void *stream) {
    return backward_entry(desc, dy, x, gamma, w1, w2, h_saved, a_saved, rstd_saved, dx, dgamma, dw1, dw2,
                          workspace, workspace_bytes, stream, false);
}

int mlpblk_backward_overwrite(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                              const void *w1, const void *w2, const void *h_saved, const void *a_saved,
                              const float *rstd_saved, void *dx, float *dgamma, float *dw1, float *dw2,
                              void *workspace, size_t workspace_bytes, void *stream) {
    return backward_entry(desc, dy, x, gamma, w1, w2, h_saved, a_saved, rstd_saved, dx, dgamma, dw1, dw2,
                          workspace, workspace_bytes, stream, true);
}

int mlpblk_fold_weights(const mlpblk_desc *desc, const void *gamma, const void *w1, void *w1g,
                        void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (!aligned16(gamma) || !aligned16(w1) || !aligned16(w1g)) return MLPBLK_EINVAL;
    if (w1g == w1) return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_FOLD_GAMMA, s,
                  launch_fold_gamma(desc->dtype, w1, gamma, w1g, desc->ffn, desc->d_model, nullptr, 0, s));
    return MLPBLK_OK;
}

int mlpblk_forward_prefolded(const mlpblk_desc *desc, const void *x, const void *w1g, const void *w2,
                             void *y, void *h_saved, void *a_saved, float *rstd_saved, void *workspace,
                             size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(w1g) || !aligned16(w2) || !aligned16(y) || !aligned16(h_saved) ||
        !aligned16(a_saved) || !aligned16(rstd_saved) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (y == x) return MLPBLK_EINVAL;
    const WsLayout l = ws_layout(desc, false);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return forward_impl(desc, x, nullptr, nullptr, w2, y, h_saved, a_saved, rstd_saved, const_cast<void *>(w1g),
                        reinterpret_cast<float *>(ws + l.sk_partial), reinterpret_cast<int *>(ws + l.sk_flags),
                        sms, static_cast<cudaStream_t>(stream), false, true);
}

size_t mlpblk_workspace_size_recompute(const mlpblk_desc *desc) {
    if (check_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(ws_layout(desc, true).total);
}

int mlpblk_forward_recompute(const mlpblk_desc *desc, const void *x, const void *gamma,
                             const void *w1, const void *w2, void *y, float *rstd_saved,
                             void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(w1) || !aligned16(w2) || !aligned16(y) ||
        !aligned16(rstd_saved) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (y == x) return MLPBLK_EINVAL;
    const WsLayout l = ws_layout(desc, true);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    // bf16: the W1 epilogue writes a alone; fp32: h goes to scratch
    const bool bf16 = desc->dtype == MLPBLK_BF16;
    return forward_impl(desc, x, gamma, w1, w2, y, bf16 ? nullptr : ws + l.h, ws + l.a, rstd_saved,
                        ws + l.w1g, reinterpret_cast<float *>(ws + l.sk_partial),
                        reinterpret_cast<int *>(ws + l.sk_flags), sms, static_cast<cudaStream_t>(stream), bf16);
}

int mlpblk_backward_recompute(const mlpblk_desc *desc, const void *dy, const void *x,
                              const void *gamma, const void *w1, const void *w2,
                              const float *rstd_saved, void *dx, float *dgamma, float *dw1,
                              float *dw2, void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(w1) || !aligned16(w2) ||
        !aligned16(rstd_saved) || !aligned16(dx) || !aligned16(dgamma) || !aligned16(dw1) ||
        !aligned16(dw2) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (dx == dy || dx == x) return MLPBLK_EINVAL;
    const WsLayout l = ws_layout(desc, true);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t T = desc->tokens, d = desc->d_model, F = desc->ffn;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    void *w1g = ws + l.w1g;
    void *h = ws + l.h;
    void *a = ws + l.a;
    float *sk_partial = reinterpret_cast<float *>(ws + l.sk_partial);
    int *sk_flags = reinterpret_cast<int *>(ws + l.sk_flags);
    // h and a again, from x and the saved rstd: the forward's W1 GEMM (same
    // configuration and schedule, so the same bits)
    MLPBLK_LAUNCH(MLPBLK_KERNEL_FOLD_GAMMA, s,
                  launch_fold_gamma(desc->dtype, w1, gamma, w1g, F, d, sk_flags + kSetFwdW1 * kSkFlagsPerSet,
                                    kSkFlagsPerSet, s));
    if (desc->dtype == MLPBLK_BF16) {
        GemmArgs g1 = {};
        g1.rstd_in = rstd_saved;
        g1.sk_partial = sk_partial;
        g1.sk_flags = sk_flags + kSetFwdW1 * kSkFlagsPerSet;
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W1, s,
                      launch_gemm_tc_fwd(kEpiFwdW1Pre, (int)T, (int)F, (int)d, x, w1g, h, a, g1, sms, s));
    } else {
        SimtEpi e1 = {nullptr, rstd_saved, nullptr};
        MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W1, s,
                      launch_gemm_simt(kEpiFwdW1, (int)T, (int)F, (int)d, static_cast<const float *>(x), d, 1,
                                       static_cast<const float *>(w1g), d, 1, static_cast<float *>(h),
                                       static_cast<float *>(a), e1, s));
    }
    // dh_s takes the W1*gamma region, which the GEMM above was the last to read
    return backward_impl(desc, dy, x, gamma, w1, w2, h, a, rstd_saved, dx, dgamma, dw1, dw2, ws + l.dh,
                         ws + l.dn, reinterpret_cast<float *>(ws + l.part),
                         sk_partial, sk_flags, sms, s, false);
}

int mlpblk_grad_norm(const mlpblk_desc *desc, const float *dgamma, const float *dw1, const float *dw2,
                     float max_norm, float *norm_out, float *clip_scale_out, void *workspace,
                     size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (!aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (!norm_out && !clip_scale_out) return MLPBLK_EINVAL;
    if ((norm_out && (reinterpret_cast<uintptr_t>(norm_out) & 3u)) ||
        (clip_scale_out && (reinterpret_cast<uintptr_t>(clip_scale_out) & 3u)))
        return MLPBLK_EINVAL;
    if (!(max_norm > 0.0f) || !isfinite(max_norm)) return MLPBLK_EINVAL;
    const WsLayout l = ws_layout(desc, false);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    const int64_t d = desc->d_model, F = desc->ffn;
    const int64_t part_bytes = static_cast<int64_t>(kMaxParts) * d * 4;
    const int max_parts = static_cast<int>(part_bytes / 8 < 1024 ? part_bytes / 8 : 1024);
    double *partial = reinterpret_cast<double *>(static_cast<uint8_t *>(workspace) + l.part);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int parts = 0;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GRAD_NORM, s,
                  launch_grad_norm_partial(dgamma, d, dw1, F * d, dw2, F * d, partial, max_parts, &parts, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GRAD_NORM_FINAL, s,
                  launch_grad_norm_final(partial, parts, max_norm, norm_out, clip_scale_out, s));
    return MLPBLK_OK;
}

int mlpblk_clip_grads(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2, const float *clip_scale,
                      void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (!aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2)) return MLPBLK_EINVAL;
    if (!clip_scale || (reinterpret_cast<uintptr_t>(clip_scale) & 3u)) return MLPBLK_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_CLIP_GRADS, s, launch_clip_grads(dgamma, d, dw1, F * d, dw2, F * d, clip_scale, s));
    return MLPBLK_OK;
}

int mlpblk_adamw_step(const mlpblk_param *params, int count, const mlpblk_adamw *hp, int64_t step, int dtype,
                      const float *grad_scale, void *stream) {
    if (!params || count < 1 || count > 1024 || !hp || step < 1) return MLPBLK_EINVAL;
    if (dtype != MLPBLK_BF16 && dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    const float vals[5] = {hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay};
    for (float v : vals)
        if (!isfinite(v) || v < 0.0f) return MLPBLK_EINVAL;
    if (!(hp->beta1 < 1.0f) || !(hp->beta2 < 1.0f)) return MLPBLK_EINVAL;
    if (grad_scale && (reinterpret_cast<uintptr_t>(grad_scale) & 3u)) return MLPBLK_EINVAL;
    const uintptr_t walign = dtype == MLPBLK_BF16 ? 7u : 15u;
    AdamTensor t[1024];
    for (int i = 0; i < count; ++i) {
        const mlpblk_param &p = params[i];
        if (!aligned16(p.master) || !aligned16(p.grad) || !aligned16(p.m) || !aligned16(p.v)) return MLPBLK_EINVAL;
        if (p.weight && (reinterpret_cast<uintptr_t>(p.weight) & walign)) return MLPBLK_EINVAL;
        if (p.n <= 0 || p.n % 4 != 0) return MLPBLK_EINVAL;
        t[i] = AdamTensor{p.master, p.weight, p.grad, p.m, p.v, p.n, p.decay != 0};
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ADAMW, s,
                  launch_adamw(t, count, hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay, step,
                               dtype == MLPBLK_BF16, grad_scale, s));
    return MLPBLK_OK;
}

static int check_fp8_desc(const mlpblk_desc *desc) {
    MLPBLK_TRY(check_desc(desc));
    if (desc->dtype != MLPBLK_BF16) return MLPBLK_ENOTSUP;
    if (desc->d_model % 16 != 0 || desc->ffn % 16 != 0) return MLPBLK_ENOTSUP;  // 16-byte E4M3 rows
    return MLPBLK_OK;
}

size_t mlpblk_workspace_size_fp8(const mlpblk_desc *desc) {
    if (check_fp8_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(ws_layout_f8(desc).total);
}

}  // extern "C"

namespace {

// E4M3 codes of the weights, each with its scale record {amax, 448/amax, amax/448, 0}.
struct F8Weights {
    const uint8_t *w1g, *w2, *w1;  // W1*gamma [F,d], W2 [d,F], W1 [F,d]
    const float *s_w1g, *s_w2, *s_w1;
};

// A caller-owned pre-quantised weight buffer: the three code tensors, then the
// three scale records.
struct WqLayout {
    int64_t w1g, w2, w1, scales, total;
};

WqLayout wq_layout(const mlpblk_desc *d) {
    WqLayout l;
    const int64_t fd = align256(d->ffn * d->d_model);
    l.w1g = 0;
    l.w2 = fd;
    l.w1 = 2 * fd;
    l.scales = 3 * fd;
    l.total = 3 * fd + 256;
    return l;
}

// amax pass, scale record, codes of one tensor (colmul: per-column bf16 factor)
int quantize_tensor(const void *v, const void *colmul, int64_t cols, int64_t n, float *amax, float *rec,
                    uint8_t *codes, cudaStream_t s) {
    int parts = 0;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_AMAX, s, launch_amax_e4m3(v, colmul, cols, n, amax, kAmaxParts, &parts, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_SCALE, s, launch_scale_e4m3(amax, parts, rec, nullptr, 0, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_APPLY, s, launch_apply_e4m3(v, colmul, cols, n, rec, codes, s));
    return MLPBLK_OK;
}

int forward_fp8_impl(const mlpblk_desc *desc, const void *x, const F8Weights &w, void *y, void *h_saved,
                     void *a8_saved, void *n8_saved, float *rstd_saved, float *scales_saved, uint8_t *ws,
                     const WsLayoutF8 &l, int sms, cudaStream_t s) {
    const int64_t T = desc->tokens, d = desc->d_model, F = desc->ffn;
    float *amax = reinterpret_cast<float *>(ws + l.amax);
    float *sk_partial = reinterpret_cast<float *>(ws + l.sk_partial);
    int *sk_flags = reinterpret_cast<int *>(ws + l.sk_flags);
    void *a16 = ws + l.t16;
    // n' = x * rstd in E4M3 (scale 1) and rstd; clears the W1 GEMM's flags
    MLPBLK_LAUNCH(MLPBLK_KERNEL_NORM_QUANT, s,
                  launch_norm_quant(x, rstd_saved, static_cast<uint8_t *>(n8_saved), T, d, desc->eps,
                                    sk_flags + kSetFwdW1 * kSkFlagsPerSet, kSkFlagsPerSet, s));
    // h (saved, bf16) and a (bf16, scratch) = relu(h)^2, h = (n' . (W1*gamma)^T) * s_w1g
    // (the epilogue also leaves max |a| per epilogue warp in amax)
    GemmArgs g1 = {};
    g1.deq_b = w.s_w1g + 2;
    g1.sk_partial = sk_partial;
    g1.sk_flags = sk_flags + kSetFwdW1 * kSkFlagsPerSet;
    g1.amax_out = amax;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W1, s,
                  launch_gemm_tc_f8(kEpiFwdW1Pre, (int)T, (int)F, (int)d, n8_saved, w.w1g, h_saved, a16, g1, sms, s));
    // a in E4M3 (saved with its scale record; clears the W2 GEMM's flags)
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_SCALE, s,
                  launch_scale_e4m3(amax, kMaxSkSlots * kMaxEpiWarps, scales_saved, sk_flags + kSetFwdW2 * kSkFlagsPerSet,
                                    kSkFlagsPerSet, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_APPLY, s,
                  launch_apply_e4m3(a16, nullptr, F, T * F, scales_saved, static_cast<uint8_t *>(a8_saved), s));
    // y = x + (a . W2^T) * s_a * s_w2
    GemmArgs g2 = {};
    g2.aux = static_cast<const uint16_t *>(x);
    g2.ld_aux = (int)d;
    g2.deq_a = scales_saved + 2;
    g2.deq_b = w.s_w2 + 2;
    g2.sk_partial = sk_partial;
    g2.sk_flags = sk_flags + kSetFwdW2 * kSkFlagsPerSet;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W2, s,
                  launch_gemm_tc_f8(kEpiFwdW2, (int)T, (int)d, (int)F, a8_saved, w.w2, y, nullptr, g2, sms, s));
    return MLPBLK_OK;
}

int backward_fp8_impl(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma, const F8Weights &w,
                      const void *h_saved, const void *a8_saved, const void *n8_saved, const float *rstd_saved,
                      const float *scales_saved, void *dx, float *dgamma, float *dw1, float *dw2, uint8_t *ws,
                      const WsLayoutF8 &l, int sms, cudaStream_t s, bool overwrite) {
    const int64_t T = desc->tokens, d = desc->d_model, F = desc->ffn;
    float *amax = reinterpret_cast<float *>(ws + l.amax);
    float *sc = reinterpret_cast<float *>(ws + l.scales);  // records: 2 dy, 3 dh
    float *sk_partial = reinterpret_cast<float *>(ws + l.sk_partial);
    int *sk_flags = reinterpret_cast<int *>(ws + l.sk_flags);
    uint8_t *dyq = ws + l.dyq, *dh8 = ws + l.dh8;
    void *dh16 = ws + l.t16;
    float *dn_s = reinterpret_cast<float *>(ws + l.dn);
    float *part = reinterpret_cast<float *>(ws + l.part);
    int parts = 0;
    // dW2 += (dy^T . a) * s_dy * s_a; clears the dgrad-h GEMM's flags
    GemmArgs gw2 = {};
    gw2.deq_a = sc + 8 + 2;
    gw2.deq_b = scales_saved + 2;
    gw2.zero_flags = sk_flags + kSetDgradH * kSkFlagsPerSet;
    gw2.pdl = kPdlWaitFirst;  // (dW2, dh) and (dn, dW1) overlap as in the bf16 backward
    // dW1 += gamma[col] * (dh^T . n') * s_dh
    GemmArgs gw1 = {};
    gw1.colscale = static_cast<const uint16_t *>(gamma);
    gw1.deq_a = sc + 12 + 2;
    gw1.pdl = kPdlDeferWait;
    if (overwrite) {
        // = instead of +=, as in the bf16 backward: whole tiles stored, the split
        // tiles' regions (and dgamma) cleared by the call's first launch
        gw2.overwrite = 1;
        gw1.overwrite = 1;
        GemmArgs plan2 = {}, plan1 = {};
        GemmArgs q2 = gw2, q1 = gw1;
        q2.plan_out = &plan2;
        q1.plan_out = &plan1;
        MLPBLK_TRY(launch_gemm_tc_f8(kEpiAccF32, (int)d, (int)F, (int)T, dyq, a8_saved, dw2, nullptr, q2, sms, s));
        MLPBLK_TRY(launch_gemm_tc_f8(kEpiAccF32ColScale, (int)F, (int)d, (int)T, dh8, n8_saved, dw1, nullptr, q1,
                                     sms, s));
        MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s,
                      launch_zero_split_tiles(split_tiles_of(plan2, dw2, F), split_tiles_of(plan1, dw1, d), dgamma,
                                              d, s));
    }
    MLPBLK_TRY(quantize_tensor(dy, nullptr, d, T * d, amax, sc + 8, dyq, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W2, s,
                  launch_gemm_tc_f8(kEpiAccF32, (int)d, (int)F, (int)T, dyq, a8_saved, dw2, nullptr, gw2, sms, s));
    // dh = (dy . W2) * s_dy * s_w2 * 2 relu(h)   (bf16; the row scale goes to dgrad-n)
    // (the epilogue also leaves max |dh| per epilogue warp in amax)
    GemmArgs gd = {};
    gd.aux = static_cast<const uint16_t *>(h_saved);
    gd.ld_aux = (int)F;
    gd.deq_a = sc + 8 + 2;
    gd.deq_b = w.s_w2 + 2;
    gd.sk_partial = sk_partial;
    gd.sk_flags = sk_flags + kSetDgradH * kSkFlagsPerSet;
    gd.amax_out = amax;
    gd.pdl = kPdlDeferWait;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_H, s,
                  launch_gemm_tc_f8(kEpiDgradH, (int)T, (int)F, (int)d, dyq, w.w2, dh16, nullptr, gd, sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_SCALE, s,
                  launch_scale_e4m3(amax, kMaxSkSlots * kMaxEpiWarps, sc + 12, sk_flags + kSetDgradN * kSkFlagsPerSet,
                                    kSkFlagsPerSet, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_QUANT_APPLY, s, launch_apply_e4m3(dh16, nullptr, F, T * F, sc + 12, dh8, s));
    // dn_s = rstd * (dh . W1) * s_dh * s_w1   (fp32)
    GemmArgs gn = {};
    gn.rstd_in = rstd_saved;
    gn.deq_a = sc + 12 + 2;
    gn.deq_b = w.s_w1 + 2;
    gn.sk_partial = sk_partial;
    gn.sk_flags = sk_flags + kSetDgradN * kSkFlagsPerSet;
    gn.pdl = kPdlWaitFirst;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_N, s,
                  launch_gemm_tc_f8(kEpiStoreF32, (int)T, (int)d, (int)F, dh8, w.w1, dn_s, nullptr, gn, sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W1, s,
                  launch_gemm_tc_f8(kEpiAccF32ColScale, (int)F, (int)d, (int)T, dh8, n8_saved, dw1, nullptr, gw1,
                                    sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_NORM_BWD, s, launch_rmsnorm_bwd(desc->dtype, x, dn_s, 0, dy, rstd_saved, gamma, dx, part, T, d, kMaxParts, &parts, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_DGAMMA_REDUCE, s, launch_dgamma_finalize(part, parts, dgamma, d, s));
    return MLPBLK_OK;
}

}  // namespace

extern "C" {

int mlpblk_forward_fp8(const mlpblk_desc *desc, const void *x, const void *gamma, const void *w1, const void *w2,
                       void *y, void *h_saved, void *a8_saved, void *n8_saved, float *rstd_saved,
                       float *scales_saved, void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_fp8_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(w1) || !aligned16(w2) || !aligned16(y) ||
        !aligned16(h_saved) || !aligned16(a8_saved) || !aligned16(n8_saved) || !aligned16(rstd_saved) ||
        !aligned16(scales_saved) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (y == x) return MLPBLK_EINVAL;
    const WsLayoutF8 l = ws_layout_f8(desc);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *amax = reinterpret_cast<float *>(ws + l.amax);
    float *sc = reinterpret_cast<float *>(ws + l.scales);  // records: 0 W1*gamma, 1 W2
    uint8_t *w1q = ws + l.w1q, *w2q = ws + l.w2q;
    // W1 * gamma and W2 in E4M3, into the workspace
    MLPBLK_TRY(quantize_tensor(w1, gamma, d, F * d, amax, sc + 0, w1q, s));
    MLPBLK_TRY(quantize_tensor(w2, nullptr, F, d * F, amax, sc + 4, w2q, s));
    const F8Weights w = {w1q, w2q, nullptr, sc + 0, sc + 4, nullptr};
    return forward_fp8_impl(desc, x, w, y, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved, ws, l, sms, s);
}

}  // extern "C"

namespace {

// T = 0: += adds nothing; = leaves zero gradients.
int empty_backward(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2, void *stream, bool overwrite) {
    if (!overwrite) return MLPBLK_OK;
    if (!aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2)) return MLPBLK_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s, launch_grads(true, 0.0f, dgamma, d, dw1, F * d, dw2, d * F, s));
    return MLPBLK_OK;
}

int backward_fp8_entry(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma, const void *w1,
                       const void *w2, const void *h_saved, const void *a8_saved, const void *n8_saved,
                       const float *rstd_saved, const float *scales_saved, void *dx, float *dgamma, float *dw1,
                       float *dw2, void *workspace, size_t workspace_bytes, void *stream, bool overwrite) {
    MLPBLK_TRY(check_fp8_desc(desc));
    if (desc->tokens == 0) return empty_backward(desc, dgamma, dw1, dw2, stream, overwrite);
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(w1) || !aligned16(w2) ||
        !aligned16(h_saved) || !aligned16(a8_saved) || !aligned16(n8_saved) || !aligned16(rstd_saved) ||
        !aligned16(scales_saved) || !aligned16(dx) || !aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2) ||
        !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (dx == dy || dx == x) return MLPBLK_EINVAL;
    const WsLayoutF8 l = ws_layout_f8(desc);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *amax = reinterpret_cast<float *>(ws + l.amax);
    float *sc = reinterpret_cast<float *>(ws + l.scales);  // records: 0 W1, 1 W2
    uint8_t *w1q = ws + l.w1q, *w2q = ws + l.w2q;
    MLPBLK_TRY(quantize_tensor(w2, nullptr, F, d * F, amax, sc + 4, w2q, s));
    MLPBLK_TRY(quantize_tensor(w1, nullptr, d, F * d, amax, sc + 0, w1q, s));
    const F8Weights w = {nullptr, w2q, w1q, nullptr, sc + 4, sc + 0};
    return backward_fp8_impl(desc, dy, x, gamma, w, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved, dx,
                             dgamma, dw1, dw2, ws, l, sms, s, overwrite);
}

int backward_fp8_prequant_entry(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                                const void *wq, const void *h_saved, const void *a8_saved, const void *n8_saved,
                                const float *rstd_saved, const float *scales_saved, void *dx, float *dgamma,
                                float *dw1, float *dw2, void *workspace, size_t workspace_bytes, void *stream,
                                bool overwrite) {
    MLPBLK_TRY(check_fp8_desc(desc));
    if (desc->tokens == 0) return empty_backward(desc, dgamma, dw1, dw2, stream, overwrite);
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(wq) || !aligned16(h_saved) ||
        !aligned16(a8_saved) || !aligned16(n8_saved) || !aligned16(rstd_saved) || !aligned16(scales_saved) ||
        !aligned16(dx) || !aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (dx == dy || dx == x) return MLPBLK_EINVAL;
    const WsLayoutF8 l = ws_layout_f8(desc);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    const WqLayout q = wq_layout(desc);
    const uint8_t *b = static_cast<const uint8_t *>(wq);
    const float *rec = reinterpret_cast<const float *>(b + q.scales);
    const F8Weights w = {b + q.w1g, b + q.w2, b + q.w1, rec + 0, rec + 4, rec + 8};
    return backward_fp8_impl(desc, dy, x, gamma, w, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved, dx,
                             dgamma, dw1, dw2, static_cast<uint8_t *>(workspace), l, sms,
                             static_cast<cudaStream_t>(stream), overwrite);
}

}  // namespace

extern "C" {

int mlpblk_backward_fp8(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma, const void *w1,
                        const void *w2, const void *h_saved, const void *a8_saved, const void *n8_saved,
                        const float *rstd_saved, const float *scales_saved, void *dx, float *dgamma, float *dw1,
                        float *dw2, void *workspace, size_t workspace_bytes, void *stream) {
    return backward_fp8_entry(desc, dy, x, gamma, w1, w2, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved, dx,
                              dgamma, dw1, dw2, workspace, workspace_bytes, stream, false);
}

int mlpblk_backward_fp8_overwrite(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                                  const void *w1, const void *w2, const void *h_saved, const void *a8_saved,
                                  const void *n8_saved, const float *rstd_saved, const float *scales_saved,
                                  void *dx, float *dgamma, float *dw1, float *dw2, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    return backward_fp8_entry(desc, dy, x, gamma, w1, w2, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved, dx,
                              dgamma, dw1, dw2, workspace, workspace_bytes, stream, true);
}

size_t mlpblk_fp8_weights_size(const mlpblk_desc *desc) {
    if (check_fp8_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(wq_layout(desc).total);
}

int mlpblk_fp8_quantize_weights(const mlpblk_desc *desc, const void *gamma, const void *w1, const void *w2,
                                void *wq, size_t wq_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_fp8_desc(desc));
    if (!aligned16(gamma) || !aligned16(w1) || !aligned16(w2) || !aligned16(wq) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    const WqLayout q = wq_layout(desc);
    const WsLayoutF8 l = ws_layout_f8(desc);
    if (wq_bytes < static_cast<size_t>(q.total) || workspace_bytes < static_cast<size_t>(l.total))
        return MLPBLK_EWORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    uint8_t *b = static_cast<uint8_t *>(wq);
    float *rec = reinterpret_cast<float *>(b + q.scales);  // [3][4]: W1*gamma, W2, W1
    float *amax = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + l.amax);
    MLPBLK_TRY(quantize_tensor(w1, gamma, d, F * d, amax, rec + 0, b + q.w1g, s));
    MLPBLK_TRY(quantize_tensor(w2, nullptr, F, d * F, amax, rec + 4, b + q.w2, s));
    MLPBLK_TRY(quantize_tensor(w1, nullptr, d, F * d, amax, rec + 8, b + q.w1, s));
    return MLPBLK_OK;
}

int mlpblk_forward_fp8_prequant(const mlpblk_desc *desc, const void *x, const void *wq, void *y, void *h_saved,
                                void *a8_saved, void *n8_saved, float *rstd_saved, float *scales_saved,
                                void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_fp8_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(wq) || !aligned16(y) || !aligned16(h_saved) || !aligned16(a8_saved) ||
        !aligned16(n8_saved) || !aligned16(rstd_saved) || !aligned16(scales_saved) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (y == x) return MLPBLK_EINVAL;
    const WsLayoutF8 l = ws_layout_f8(desc);
    if (workspace_bytes < static_cast<size_t>(l.total)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    const WqLayout q = wq_layout(desc);
    const uint8_t *b = static_cast<const uint8_t *>(wq);
    const float *rec = reinterpret_cast<const float *>(b + q.scales);
    const F8Weights w = {b + q.w1g, b + q.w2, b + q.w1, rec + 0, rec + 4, rec + 8};
    return forward_fp8_impl(desc, x, w, y, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved,
                            static_cast<uint8_t *>(workspace), l, sms, static_cast<cudaStream_t>(stream));
}

int mlpblk_backward_fp8_prequant(const mlpblk_desc *desc, const void *dy, const void *x, const void *gamma,
                                 const void *wq, const void *h_saved, const void *a8_saved, const void *n8_saved,
                                 const float *rstd_saved, const float *scales_saved, void *dx, float *dgamma,
                                 float *dw1, float *dw2, void *workspace, size_t workspace_bytes, void *stream) {
    return backward_fp8_prequant_entry(desc, dy, x, gamma, wq, h_saved, a8_saved, n8_saved, rstd_saved,
                                       scales_saved, dx, dgamma, dw1, dw2, workspace, workspace_bytes, stream, false);
}

int mlpblk_backward_fp8_prequant_overwrite(const mlpblk_desc *desc, const void *dy, const void *x,
                                           const void *gamma, const void *wq, const void *h_saved,
                                           const void *a8_saved, const void *n8_saved, const float *rstd_saved,
                                           const float *scales_saved, void *dx, float *dgamma, float *dw1,
                                           float *dw2, void *workspace, size_t workspace_bytes, void *stream) {
    return backward_fp8_prequant_entry(desc, dy, x, gamma, wq, h_saved, a8_saved, n8_saved, rstd_saved,
                                       scales_saved, dx, dgamma, dw1, dw2, workspace, workspace_bytes, stream, true);
}

}  // extern "C"

namespace {

// Buffers of the routed-expert block.  R = the row space of the experts'
// segments: T*k assignments plus up to 255 padding rows per expert, rounded to 256.
struct MoeLayout {
    int64_t R;
    // saved
    int64_t rstd, pos, row_token, row_slot, seg, count, chunk_count, rstd_perm, x_perm, h_perm, a_perm, o_perm, saved;
    // workspace
    int64_t w1g, do_perm, dh_perm, dn_perm, part, sk_partial, sk_flags, ws;
};

int check_moe_desc(const mlpblk_moe_desc *m) {
    if (!m) return MLPBLK_EINVAL;
    MLPBLK_TRY(check_desc(&m->base));
    if (m->base.dtype != MLPBLK_BF16) return MLPBLK_ENOTSUP;
    if (m->experts < 1 || m->experts > 256 || m->top_k < 1 || m->top_k > m->experts) return MLPBLK_EINVAL;
    const int64_t lim = static_cast<int64_t>(1) << 31;
    const int64_t T = m->base.tokens, d = m->base.d_model, F = m->base.ffn, E = m->experts;
    if (T * m->top_k + E * 256 >= lim / (d > F ? d : F)) return MLPBLK_EINVAL;
    if (E * F >= lim / d) return MLPBLK_EINVAL;
    return MLPBLK_OK;
}

MoeLayout moe_layout(const mlpblk_moe_desc *m) {
    const int64_t T = m->base.tokens, d = m->base.d_model, F = m->base.ffn, E = m->experts, k = m->top_k;
    MoeLayout l;
    l.R = (T * k + E * 255 + 255) / 256 * 256;
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = off;
        off += align256(bytes);
        return at;
    };
    l.rstd = take(T * 4);
    l.pos = take(T * k * 4);
    l.row_token = take(l.R * 4);
    l.row_slot = take(l.R * 4);
    l.seg = take((E + 1) * 4);
    l.count = take(E * 4);
    l.chunk_count = take(moe_route_chunks(T * k) * E * 4);
    l.rstd_perm = take(l.R * 4);
    l.x_perm = take(l.R * d * 2);
    l.h_perm = take(l.R * F * 2);
    l.a_perm = take(l.R * F * 2);
    l.o_perm = take(l.R * d * 2);
    l.saved = off;
    // workspace: the forward's W1*gamma and the backward's buffers share it
    off = 0;
    const int64_t w1g = align256(E * F * d * 2);
    l.w1g = 0;
    l.do_perm = take(l.R * d * 2);
    l.dh_perm = take(l.R * F * 2);
    l.dn_perm = take(l.R * d * 2);
    l.part = take(static_cast<int64_t>(kMaxParts) * d * 4);
    // the M-grouped GEMMs' split schedule: partial sums and flags, apart from the
    // forward's W1*gamma (both live in the forward)
    off = off > w1g ? off : w1g;
    l.sk_partial = take(static_cast<int64_t>(kMaxSkSlots) * kSkSlotFloats * 4);
    l.sk_flags = take(static_cast<int64_t>(kSkSets) * kSkFlagsPerSet * 4);
    l.ws = off;
    return l;
}

}  // namespace

extern "C" {

size_t mlpblk_moe_saved_size(const mlpblk_moe_desc *desc) {
    if (check_moe_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(moe_layout(desc).saved);
}

size_t mlpblk_moe_workspace_size(const mlpblk_moe_desc *desc) {
    if (check_moe_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(moe_layout(desc).ws);
}

int mlpblk_moe_forward(const mlpblk_moe_desc *desc, const void *x, const void *gamma, const void *w1s,
                       const void *w2s, const int32_t *expert_idx, const float *routing_weights, void *y,
                       void *saved, size_t saved_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_moe_desc(desc));
    if (desc->base.tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(w1s) || !aligned16(w2s) || !aligned16(expert_idx) ||
        !aligned16(routing_weights) || !aligned16(y) || !aligned16(saved) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (y == x) return MLPBLK_EINVAL;
    const MoeLayout l = moe_layout(desc);
    if (saved_bytes < static_cast<size_t>(l.saved) || workspace_bytes < static_cast<size_t>(l.ws))
        return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t T = desc->base.tokens, d = desc->base.d_model, F = desc->base.ffn;
    const int E = desc->experts, k = desc->top_k;
    uint8_t *sv = static_cast<uint8_t *>(saved);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *rstd = reinterpret_cast<float *>(sv + l.rstd);
    int *pos = reinterpret_cast<int *>(sv + l.pos);
    int *row_token = reinterpret_cast<int *>(sv + l.row_token);
    int *row_slot = reinterpret_cast<int *>(sv + l.row_slot);
    int *seg = reinterpret_cast<int *>(sv + l.seg);
    int *count = reinterpret_cast<int *>(sv + l.count);
    int *chunk_count = reinterpret_cast<int *>(sv + l.chunk_count);
    float *rstd_perm = reinterpret_cast<float *>(sv + l.rstd_perm);
    void *x_perm = sv + l.x_perm, *h_perm = sv + l.h_perm, *a_perm = sv + l.a_perm, *o_perm = sv + l.o_perm;
    void *w1g = ws + l.w1g;
    float *sk_partial = reinterpret_cast<float *>(ws + l.sk_partial);
    int *sk_flags = reinterpret_cast<int *>(ws + l.sk_flags);
    // rstd and every expert's W1 * gamma (the experts' W1 as one [E*F, d] matrix);
    // clears the W1 GEMM's flags
    MLPBLK_LAUNCH(MLPBLK_KERNEL_FOLD_GAMMA, s,
                  launch_norm_prep(MLPBLK_BF16, x, rstd, T, d, desc->base.eps, w1s, gamma, w1g, E * F,
                                   sk_flags + kSetFwdW1 * kSkFlagsPerSet, kSkFlagsPerSet, s));
    for (int step = 0; step < kMoeRouteLaunches; ++step)
        MLPBLK_LAUNCH(MLPBLK_KERNEL_MOE_ROUTE, s,
                      launch_moe_route(expert_idx, T * k, k, E, chunk_count, count, seg, pos, row_token, row_slot,
                                       step, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_MOE_GATHER, s,
                  launch_moe_gather(x, rstd, row_token, seg, E, l.R, d, x_perm, rstd_perm, s));
    GemmArgs g1 = {};
    g1.rstd_in = rstd_perm;
    g1.grp_mode = kGroupM;
    g1.grp_count = E;
    g1.grp_rows = seg;
    g1.grp_b_off = static_cast<int>(F);
    g1.sk_partial = sk_partial;
    g1.sk_flags = sk_flags + kSetFwdW1 * kSkFlagsPerSet;
    g1.zero_flags = sk_flags + kSetFwdW2 * kSkFlagsPerSet;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W1, s,
                  launch_gemm_tc_fwd(kEpiFwdW1Pre, (int)l.R, (int)F, (int)d, x_perm, w1g, h_perm, a_perm, g1, sms, s));
    GemmArgs g2 = {};
    g2.grp_mode = kGroupM;
    g2.grp_count = E;
    g2.grp_rows = seg;
    g2.grp_b_off = static_cast<int>(d);
    g2.sk_partial = sk_partial;
    g2.sk_flags = sk_flags + kSetFwdW2 * kSkFlagsPerSet;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_FWD_W2, s,
                  launch_gemm_tc_fwd(kEpiStoreBf16, (int)l.R, (int)d, (int)F, a_perm, w2s, o_perm, nullptr, g2, sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_MOE_COMBINE, s, launch_moe_combine(x, o_perm, routing_weights, pos, T, k, d, y, s));
    return MLPBLK_OK;
}

}  // extern "C"

namespace {

int moe_backward_entry(const mlpblk_moe_desc *desc, const void *dy, const void *x, const void *gamma,
                       const void *w1s, const void *w2s, const float *routing_weights, const void *saved,
                       void *dx, float *d_routing_weights, float *dgamma, float *dw1s, float *dw2s,
                       void *workspace, size_t workspace_bytes, void *stream, bool overwrite) {
    MLPBLK_TRY(check_moe_desc(desc));
    if (desc->base.tokens == 0) {
        // no rows: += adds nothing; = leaves zero gradients
        if (!overwrite) return MLPBLK_OK;
        if (!aligned16(dgamma) || !aligned16(dw1s) || !aligned16(dw2s)) return MLPBLK_EINVAL;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const int64_t d = desc->base.d_model, EF = static_cast<int64_t>(desc->experts) * desc->base.ffn;
        MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s,
                      launch_grads(true, 0.0f, dgamma, d, dw1s, EF * d, dw2s, d * EF, s));
        return MLPBLK_OK;
    }
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(w1s) || !aligned16(w2s) ||
        !aligned16(routing_weights) || !aligned16(saved) || !aligned16(dx) || !aligned16(d_routing_weights) ||
        !aligned16(dgamma) || !aligned16(dw1s) || !aligned16(dw2s) || !aligned16(workspace))
        return MLPBLK_EINVAL;
    if (dx == dy || dx == x) return MLPBLK_EINVAL;
    const MoeLayout l = moe_layout(desc);
    if (workspace_bytes < static_cast<size_t>(l.ws)) return MLPBLK_EWORKSPACE;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t T = desc->base.tokens, d = desc->base.d_model, F = desc->base.ffn;
    const int E = desc->experts, k = desc->top_k;
    const uint8_t *sv = static_cast<const uint8_t *>(saved);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const float *rstd = reinterpret_cast<const float *>(sv + l.rstd);
    const int *pos = reinterpret_cast<const int *>(sv + l.pos);
    const int *seg = reinterpret_cast<const int *>(sv + l.seg);
    const int *count = reinterpret_cast<const int *>(sv + l.count);
    const float *rstd_perm = reinterpret_cast<const float *>(sv + l.rstd_perm);
    const void *x_perm = sv + l.x_perm, *h_perm = sv + l.h_perm, *a_perm = sv + l.a_perm, *o_perm = sv + l.o_perm;
    void *do_perm = ws + l.do_perm, *dh_perm = ws + l.dh_perm;
    uint16_t *dn_perm = reinterpret_cast<uint16_t *>(ws + l.dn_perm);  // bf16
    float *part = reinterpret_cast<float *>(ws + l.part);
    float *sk_partial = reinterpret_cast<float *>(ws + l.sk_partial);
    int *sk_flags = reinterpret_cast<int *>(ws + l.sk_flags);
    int parts = 0;
    // d_routing_weights and each slot's output gradient p * dy in segment order
    // (overwrite: it also clears the gradient blocks of experts no token chose,
    // which the K-grouped wgrads skip)
    MLPBLK_LAUNCH(MLPBLK_KERNEL_MOE_DP, s,
                  launch_moe_dout(dy, o_perm, routing_weights, pos, count, seg, T, k, E, d, d_routing_weights, do_perm,
                                  overwrite ? dw1s : nullptr, overwrite ? dw2s : nullptr, F, s));
    GemmArgs gw2 = {};
    gw2.grp_mode = kGroupK;
    gw2.grp_count = E;
    gw2.grp_rows = seg;
    gw2.grp_c_off = static_cast<int>(d);
    gw2.overwrite = overwrite ? 1 : 0;  // whole tiles: a store instead of an add
    gw2.zero_flags = sk_flags + kSetDgradH * kSkFlagsPerSet;
    gw2.pdl = kPdlWaitFirst;  // (dW2, dh) and (dn, dW1) overlap as in the dense backward
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W2, s,
                  launch_gemm_tc_bwd(kEpiAccF32, (int)d, (int)F, (int)l.R, do_perm, a_perm, dw2s, nullptr, gw2, sms, s));
    GemmArgs gd = {};
    gd.aux = static_cast<const uint16_t *>(h_perm);
    gd.ld_aux = (int)F;
    gd.rstd_in = rstd_perm;
    gd.grp_mode = kGroupM;
    gd.grp_count = E;
    gd.grp_rows = seg;
    gd.grp_b_off = static_cast<int>(d);
    gd.sk_partial = sk_partial;
    gd.sk_flags = sk_flags + kSetDgradH * kSkFlagsPerSet;
    gd.zero_flags = sk_flags + kSetDgradN * kSkFlagsPerSet;
    gd.pdl = kPdlDeferWait;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_H, s,
                  launch_gemm_tc_bwd(kEpiDgradH, (int)l.R, (int)F, (int)d, do_perm, w2s, dh_perm, nullptr, gd, sms, s));
    GemmArgs gn = {};
    gn.grp_mode = kGroupM;
    gn.grp_count = E;
    gn.grp_rows = seg;
    gn.grp_b_off = static_cast<int>(F);
    gn.sk_partial = sk_partial;
    gn.sk_flags = sk_flags + kSetDgradN * kSkFlagsPerSet;
    gn.pdl = kPdlWaitFirst;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_DGRAD_N, s,
                  launch_gemm_tc_bwd(kEpiStoreBf16, (int)l.R, (int)d, (int)F, dh_perm, w1s, dn_perm, nullptr, gn, sms, s));
    GemmArgs gw1 = {};
    gw1.colscale = static_cast<const uint16_t *>(gamma);
    gw1.grp_mode = kGroupK;
    gw1.grp_count = E;
    gw1.grp_rows = seg;
    gw1.grp_c_off = static_cast<int>(F);
    gw1.overwrite = overwrite ? 1 : 0;
    gw1.pdl = kPdlDeferWait;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_GEMM_WGRAD_W1, s,
                  launch_gemm_tc_bwd(kEpiAccF32ColScale, (int)F, (int)d, (int)l.R, dh_perm, x_perm, dw1s, nullptr, gw1,
                                     sms, s));
    // the slots' dn meet at n (sum rule) inside the RMSNorm backward
    MLPBLK_LAUNCH(MLPBLK_KERNEL_NORM_BWD, s,
                  launch_rmsnorm_bwd_gather(x, dn_perm, 1, pos, k, dy, rstd, gamma, dx, part, T, d, kMaxParts, &parts,
                                            s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_DGAMMA_REDUCE, s,
                  launch_dgamma_finalize(part, parts, dgamma, d, s, overwrite ? 1 : 0));
    return MLPBLK_OK;
}

}  // namespace

namespace {

// The bytes of one argument, for the check that outputs lie apart (NULL: none).
struct Span {
    uintptr_t first, end;
    Span(const void *p, int64_t n, int64_t element, int64_t more = 1) : first(reinterpret_cast<uintptr_t>(p)), end(first) {
        const unsigned __int128 top = static_cast<unsigned __int128>(first) + static_cast<unsigned __int128>(n) * element * more;
        if (p) end = top > UINTPTR_MAX ? UINTPTR_MAX : static_cast<uintptr_t>(top);
    }
    bool meets(const Span &o) const { return first < o.end && o.first < end; }
};

// No output shares a byte with an input or with another output.
bool apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (o->meets(i)) return false;
        for (const Span *p = outputs.begin(); p != o; ++p)
            if (o->meets(*p)) return false;
    }
    return true;
}

// ----------------------------------------------- tokens sorted by expert and back

// Bytes of a row's element.
int64_t element_bytes(int dtype) { return dtype == MLPBLK_BF16 ? 2 : 4; }

int check_sort_desc(const mlpblk_sort_desc *d) {
    if (!d) return MLPBLK_EINVAL;
    if (d->dtype != MLPBLK_BF16 && d->dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->tokens < 0 || d->width < 1 || d->experts < 1 || d->experts > 256 || d->top_k < 1 || d->top_k > 256 ||
        d->pad < 1 || d->pad > 1024)
        return MLPBLK_EINVAL;
    const int64_t lim = static_cast<int64_t>(1) << 31;
    if (d->width >= lim / 2 || d->tokens >= lim) return MLPBLK_EINVAL;
    if (d->tokens * d->top_k + static_cast<int64_t>(d->experts + 1) * d->pad >= lim) return MLPBLK_EINVAL;
    return MLPBLK_OK;
}

int64_t sort_rows(const mlpblk_sort_desc *d) {
    const int64_t n = d->tokens * d->top_k, used = n < d->experts ? n : d->experts;
    return (n + used * (d->pad - 1) + d->pad - 1) / d->pad * d->pad;
}

// ------------------------------------------------------------------------ MXFP4

constexpr int64_t kFp4Lim = static_cast<int64_t>(1) << 31;

int check_fp4_desc(const mlpblk_fp4_desc *d) {
    if (!d) return MLPBLK_EINVAL;
    if (d->dtype != MLPBLK_BF16 && d->dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->act != MLPBLK_FP4_ACT_NONE && d->act != MLPBLK_FP4_ACT_RELU2) return MLPBLK_ENOTSUP;
    if (d->transposed != 0 && d->transposed != 1) return MLPBLK_EINVAL;
    if (d->rows < 0 || d->cols < 0 || d->batch < 1 || d->cols >= kFp4Lim) return MLPBLK_EINVAL;
    if (d->rows >= kFp4Lim || d->rows * d->batch >= kFp4Lim) return MLPBLK_EINVAL;
    if ((d->rows + 127) / 128 * d->batch >= kFp4Lim / 4) return MLPBLK_EINVAL;  // CTAs of a launch
    const int64_t pieces = (d->cols + 255) / 256;  // of a row: warps of a launch
    if ((d->rows + 127) / 128 * d->batch * pieces >= kFp4Lim / 8 || d->rows * d->batch * pieces >= kFp4Lim) return MLPBLK_EINVAL;
    return MLPBLK_OK;
}

int check_fp4_matmul(const mlpblk_fp4_matmul_desc *d, int mode) {
    if (!d) return MLPBLK_EINVAL;
    if (d->out_dtype != MLPBLK_BF16 && d->out_dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->accumulate != 0 && d->accumulate != 1) return MLPBLK_EINVAL;
    if (d->accumulate && d->out_dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->m < 0 || d->n < 1 || d->k < (mode == kFp4GroupK ? 0 : 1)) return MLPBLK_EINVAL;
    if (d->m >= kFp4Lim || d->n >= kFp4Lim || d->k >= kFp4Lim) return MLPBLK_EINVAL;
    if (d->max_rows < 0 || (d->max_rows > 0 && mode != kFp4GroupRows)) return MLPBLK_EINVAL;
    int64_t tiles = ((d->m + 31) / 32) * ((d->n + 127) / 128);
    if (mode == kFp4Dense) {
        if (d->experts != 0 || d->pad != 0) return MLPBLK_EINVAL;
    } else {
        if (d->experts < 1 || d->experts > 256 || d->pad < 1) return MLPBLK_EINVAL;
        if (d->pad % (mode == kFp4GroupRows ? 128 : 256) != 0) return MLPBLK_ENOTSUP;
        if ((mode == kFp4GroupRows ? d->n : d->m) * d->experts >= kFp4Lim) return MLPBLK_EINVAL;
        tiles *= mode == kFp4GroupK ? d->experts : 1;
    }
    return tiles < kFp4Lim / 2 ? MLPBLK_OK : MLPBLK_EINVAL;
}

// A product's sizes and types; its buffers are the caller's to fill in.
Fp4Product fp4_product_of(const mlpblk_fp4_matmul_desc *desc, int mode) {
    Fp4Product p = {};
    p.mode = mode;
    p.m = desc->m;
    p.n = desc->n;
    p.k = desc->k;
    p.experts = desc->experts;
    p.max_rows = desc->max_rows;
    p.out_dtype = desc->out_dtype;
    p.accumulate = desc->accumulate;
    return p;
}

int fp4_product(const mlpblk_fp4_matmul_desc *desc, int mode, const void *a_codes, const void *a_scales,
                const void *b_codes, const void *b_scales, const int32_t *count, const int32_t *seg, void *c,
                void *stream) {
    MLPBLK_TRY(check_fp4_matmul(desc, mode));
    if (desc->m == 0) return MLPBLK_OK;
    if (desc->k == 0) {  // weight gradients of no rows at all
        if (!aligned16(c)) return MLPBLK_EINVAL;
        if (desc->accumulate) return MLPBLK_OK;
        const size_t bytes = static_cast<size_t>(desc->experts) * desc->m * desc->n * (desc->out_dtype == MLPBLK_BF16 ? 2 : 4);
        return cuda_status(cudaMemsetAsync(c, 0, bytes, static_cast<cudaStream_t>(stream)));
    }
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) || !aligned16(c))
        return MLPBLK_EINVAL;
    if ((mode != kFp4Dense && !aligned16(seg)) || (mode == kFp4GroupRows && !aligned16(count))) return MLPBLK_EINVAL;
    const int64_t b_mats = mode == kFp4GroupRows ? desc->experts : 1, c_mats = mode == kFp4GroupK ? desc->experts : 1;
    if (!apart({Span(c, desc->m, desc->n * element_bytes(desc->out_dtype), c_mats)},
               {Span(a_codes, desc->m, fp4_row_bytes(desc->k)), Span(a_scales, fp4_scales_bytes(desc->m, desc->k), 1),
                Span(b_codes, desc->n, fp4_row_bytes(desc->k), b_mats), Span(b_scales, fp4_scales_bytes(desc->n, desc->k), b_mats),
                Span(count, desc->experts, 4), Span(seg, desc->experts + 1, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Fp4Product p = fp4_product_of(desc, mode);
    p.a = static_cast<const uint8_t *>(a_codes);
    p.sa = static_cast<const uint8_t *>(a_scales);
    p.b = static_cast<const uint8_t *>(b_codes);
    p.sb = static_cast<const uint8_t *>(b_scales);
    p.count = count;
    p.seg = seg;
    p.c = c;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_FP4_GEMM, s, launch_fp4_matmul(p, sms, s));
    return MLPBLK_OK;
}

}  // namespace

extern "C" {

int64_t mlpblk_moe_sort_rows(const mlpblk_sort_desc *desc) {
    return check_sort_desc(desc) != MLPBLK_OK ? -1 : sort_rows(desc);
}

int mlpblk_moe_sort(const mlpblk_sort_desc *desc, const int32_t *expert_idx, int32_t *count, int32_t *seg,
                    int32_t *pos, int32_t *row_map, void *stream) {
    MLPBLK_TRY(check_sort_desc(desc));
    const int64_t n = desc->tokens * desc->top_k;
    if (!aligned16(count) || !aligned16(seg)) return MLPBLK_EINVAL;
    if (n > 0 && (!aligned16(expert_idx) || !aligned16(pos) || !aligned16(row_map))) return MLPBLK_EINVAL;
    if (!apart({Span(count, desc->experts, 4), Span(seg, desc->experts + 1, 4), Span(pos, n, 4), Span(row_map, sort_rows(desc), 4)},
               {Span(expert_idx, n, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_SORT, s,
                  launch_sort(expert_idx, n, desc->experts, desc->pad, sort_rows(desc), count, seg, pos, row_map, s));
    return MLPBLK_OK;
}

int mlpblk_moe_permute(const mlpblk_sort_desc *desc, const void *x, const int32_t *pos, const int32_t *count,
                       const int32_t *seg, void *rows, void *stream) {
    MLPBLK_TRY(check_sort_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(x) || !aligned16(pos) || !aligned16(count) || !aligned16(seg) || !aligned16(rows)) return MLPBLK_EINVAL;
    const int64_t row = desc->width * element_bytes(desc->dtype);
    if (!apart({Span(rows, sort_rows(desc), row)}, {Span(x, desc->tokens, row), Span(pos, desc->tokens * desc->top_k, 4),
                                                    Span(count, desc->experts, 4), Span(seg, desc->experts + 1, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_PERMUTE, s,
                  launch_permute(x, pos, count, seg, desc->tokens, desc->width, desc->dtype, desc->top_k, desc->experts,
                                 desc->pad, sort_rows(desc), rows, s));
    return MLPBLK_OK;
}

int mlpblk_moe_unpermute(const mlpblk_sort_desc *desc, const void *rows, const int32_t *pos, const float *weights,
                         const void *residual, void *y, void *stream) {
    MLPBLK_TRY(check_sort_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(rows) || !aligned16(pos) || !aligned16(y)) return MLPBLK_EINVAL;
    if ((weights && !aligned16(weights)) || (residual && !aligned16(residual))) return MLPBLK_EINVAL;
    const int64_t row = desc->width * element_bytes(desc->dtype), n = desc->tokens * desc->top_k;
    if (!apart({Span(y, desc->tokens, row)}, {Span(rows, sort_rows(desc), row), Span(pos, n, 4), Span(weights, n, 4),
                                              Span(residual == y ? nullptr : residual, desc->tokens, row)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_UNPERMUTE, s,
                  launch_unpermute(rows, pos, weights, residual, desc->tokens, desc->width, desc->dtype, desc->top_k,
                                   sort_rows(desc), y, s));
    return MLPBLK_OK;
}

int mlpblk_moe_permute_backward(const mlpblk_sort_desc *desc, const void *d_rows, const int32_t *pos, void *dx,
                                void *stream) {
    return mlpblk_moe_unpermute(desc, d_rows, pos, nullptr, nullptr, dx, stream);
}

int mlpblk_moe_unpermute_backward(const mlpblk_sort_desc *desc, const void *dy, const void *rows,
                                  const int32_t *pos, const int32_t *count, const int32_t *seg,
                                  const float *weights, void *d_rows, float *d_weights, void *stream) {
    MLPBLK_TRY(check_sort_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(dy) || !aligned16(pos) || !aligned16(count) || !aligned16(seg) || !aligned16(d_rows)) return MLPBLK_EINVAL;
    if ((weights && !aligned16(weights)) || (d_weights && (!aligned16(d_weights) || !aligned16(rows)))) return MLPBLK_EINVAL;
    const int64_t row = desc->width * element_bytes(desc->dtype), n = desc->tokens * desc->top_k, r = sort_rows(desc);
    if (d_rows == rows) return MLPBLK_EINVAL;
    if (!apart({Span(d_rows, r, row), Span(d_weights, n, 4)},
               {Span(dy, desc->tokens, row), Span(d_weights ? rows : nullptr, r, row), Span(pos, n, 4), Span(count, desc->experts, 4),
                Span(seg, desc->experts + 1, 4), Span(weights, n, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_UNPERMUTE_BWD, s,
                  launch_unpermute_bwd(dy, rows, pos, count, seg, weights, desc->tokens, desc->width, desc->dtype,
                                       desc->top_k, desc->experts, desc->pad, sort_rows(desc), d_rows, d_weights, s));
    return MLPBLK_OK;
}

size_t mlpblk_fp4_codes_size(const mlpblk_fp4_desc *desc) {
    if (check_fp4_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(desc->rows * fp4_row_bytes(desc->cols) * desc->batch);
}

size_t mlpblk_fp4_scales_size(const mlpblk_fp4_desc *desc) {
    if (check_fp4_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(fp4_scales_bytes(desc->rows, desc->cols) * desc->batch);
}

int mlpblk_fp4_quantize(const mlpblk_fp4_desc *desc, const void *x, const int32_t *row_map, int32_t map_div,
                        void *codes, void *scales, void *stream) {
    MLPBLK_TRY(check_fp4_desc(desc));
    if (map_div < 0 || (row_map && desc->batch != 1)) return MLPBLK_EINVAL;
    if (desc->rows == 0 || desc->cols == 0) return MLPBLK_OK;
    const int64_t source_rows = row_map && map_div > 0 ? desc->source_rows : 1;
    if (source_rows < 1 || source_rows >= kFp4Lim) return MLPBLK_EINVAL;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || (row_map && !aligned16(row_map))) return MLPBLK_EINVAL;
    // x's rows: Q's, or, transposed, its columns, or those that the map gathers from
    const int64_t mapped = desc->transposed ? desc->cols : desc->rows, width = desc->transposed ? desc->rows : desc->cols;
    const int64_t x_rows = row_map && map_div > 0 ? source_rows : mapped * desc->batch;
    if (!apart({Span(codes, desc->rows * desc->batch, fp4_row_bytes(desc->cols)),
                Span(scales, fp4_scales_bytes(desc->rows, desc->cols), desc->batch)},
               {Span(x, x_rows, width * element_bytes(desc->dtype)), Span(row_map, mapped, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_FP4_QUANT, s,
                  launch_fp4_quantize(desc->dtype, x, row_map, map_div, static_cast<int>(source_rows), desc->rows, desc->cols, desc->batch,
                                      desc->transposed != 0, desc->act == MLPBLK_FP4_ACT_RELU2,
                                      static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales), s));
    return MLPBLK_OK;
}

int mlpblk_fp4_dequantize(const mlpblk_fp4_desc *desc, const void *codes, const void *scales, void *y,
                          void *stream) {
    MLPBLK_TRY(check_fp4_desc(desc));
    if (desc->transposed != 0 || desc->act != MLPBLK_FP4_ACT_NONE) return MLPBLK_ENOTSUP;
    if (desc->rows == 0 || desc->cols == 0) return MLPBLK_OK;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(y)) return MLPBLK_EINVAL;
    if (!apart({Span(y, desc->rows * desc->batch, desc->cols * element_bytes(desc->dtype))},
               {Span(codes, desc->rows * desc->batch, fp4_row_bytes(desc->cols)),
                Span(scales, fp4_scales_bytes(desc->rows, desc->cols), desc->batch)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_FP4_DEQUANT, s,
                  launch_fp4_dequantize(desc->dtype, static_cast<const uint8_t *>(codes),
                                        static_cast<const uint8_t *>(scales), desc->rows, desc->cols, desc->batch, y, s));
    return MLPBLK_OK;
}

int mlpblk_fp4_matmul(const mlpblk_fp4_matmul_desc *desc, const void *a_codes, const void *a_scales,
                      const void *b_codes, const void *b_scales, void *c, void *stream) {
    return fp4_product(desc, kFp4Dense, a_codes, a_scales, b_codes, b_scales, nullptr, nullptr, c, stream);
}

int mlpblk_fp4_matmul_grouped(const mlpblk_fp4_matmul_desc *desc, const void *a_codes, const void *a_scales,
                              const void *b_codes, const void *b_scales, const int32_t *count,
                              const int32_t *seg, void *c, void *stream) {
    return fp4_product(desc, kFp4GroupRows, a_codes, a_scales, b_codes, b_scales, count, seg, c, stream);
}

int mlpblk_fp4_wgrad_grouped(const mlpblk_fp4_matmul_desc *desc, const void *a_codes, const void *a_scales,
                             const void *b_codes, const void *b_scales, const int32_t *seg, void *c,
                             void *stream) {
    return fp4_product(desc, kFp4GroupK, a_codes, a_scales, b_codes, b_scales, nullptr, seg, c, stream);
}

int mlpblk_fp4_product_kernel(const mlpblk_fp4_matmul_desc *desc, int form, int sms) {
    if (form < kFp4Dense || form > kFp4GroupK || sms < 1 || check_fp4_matmul(desc, form) != MLPBLK_OK) return -1;
    if (desc->m == 0 || desc->k == 0) return -1;
    const Fp4Choice c = choose_fp4_matmul(fp4_product_of(desc, form), sms);
    return c.pair ? (c.tma ? MLPBLK_FP4_KERNEL_PAIR_TMA : MLPBLK_FP4_KERNEL_PAIR) : c.split;
}

}  // extern "C"

extern "C" {

// ------------------------------------------- the router, the residual norm, Muon

namespace {

constexpr int64_t kLim31 = static_cast<int64_t>(1) << 31;

int check_route_desc(const mlpblk_route_desc *d) {
    if (!d) return MLPBLK_EINVAL;
    if (d->dtype != MLPBLK_BF16 && d->dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->score != MLPBLK_ROUTE_SOFTMAX && d->score != MLPBLK_ROUTE_SIGMOID) return MLPBLK_ENOTSUP;
    if (d->tokens < 0 || d->tokens >= kLim31 || d->experts < 1 || d->experts > 256 || d->top_k < 1 ||
        d->top_k > MLPBLK_ROUTE_MAX_TOP_K)
        return MLPBLK_EINVAL;
    if (d->groups < 1 || d->groups > 64 || d->experts % d->groups != 0 || d->top_groups < 1 || d->top_groups > d->groups)
        return MLPBLK_EINVAL;
    if (d->top_k > d->top_groups * (d->experts / d->groups)) return MLPBLK_EINVAL;
    if ((d->renorm != 0 && d->renorm != 1) || !isfinite(d->scale)) return MLPBLK_EINVAL;
    return MLPBLK_OK;
}

int check_norm_desc(const mlpblk_norm_desc *d) {
    if (!d) return MLPBLK_EINVAL;
    if (d->dtype != MLPBLK_BF16 && d->dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->tokens < 0 || d->tokens >= kLim31 || d->width < 1) return MLPBLK_EINVAL;
    if (d->width > kNormMaxWidth) return MLPBLK_ENOTSUP;
    if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return MLPBLK_EINVAL;
    if (d->block != 0 && d->block != 128) return MLPBLK_ENOTSUP;
    return MLPBLK_OK;
}

int check_ortho_desc(const mlpblk_ortho_desc *d) {
    if (!d) return MLPBLK_EINVAL;
    if (d->dtype != MLPBLK_BF16 && d->dtype != MLPBLK_FP32) return MLPBLK_ENOTSUP;
    if (d->rows < 1 || d->cols < 1 || d->rows > 131072 || d->cols > 131072 || d->batch < 1 || d->batch > 65535) return MLPBLK_EINVAL;
    if (d->rows * d->cols * d->batch >= static_cast<int64_t>(1) << 40) return MLPBLK_EINVAL;
    if (d->steps < 1 || d->steps > MLPBLK_ORTHO_MAX_STEPS || !(d->eps >= 0.0f) || !isfinite(d->eps)) return MLPBLK_EINVAL;
    for (int i = 0; i < d->steps; ++i)
        for (int j = 0; j < 3; ++j)
            if (!isfinite(d->coefficients[i][j])) return MLPBLK_EINVAL;
    return MLPBLK_OK;
}

// Workspace of an orthogonalisation: X twice (a step reads one and writes the other), its
// low parts, four square matrices of the short side, the remainders of three diagonals, the
// norm's partial sums.
struct OrthoLayout {
    int64_t x[2], lo, g[4], diag[3], partial, total;
};
OrthoLayout ortho_layout(const mlpblk_ortho_desc *d) {
    OrthoLayout l = {};
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = off;
        off += align256(bytes);
        return at;
    };
    const int64_t m = d->rows < d->cols ? d->rows : d->cols;
    const int64_t x = d->rows * ortho_pitch(d->cols) * d->batch * 2, g = m * ortho_pitch(m) * d->batch * 2;
    l.x[0] = take(x);
    l.x[1] = take(x);
    l.lo = take(x);
    for (int64_t &at : l.g) at = take(g);
    for (int64_t &at : l.diag) at = take(ortho_pitch(m) * d->batch * 4);
    l.partial = take((d->batch > kOrthoNormParts ? d->batch : kOrthoNormParts) * static_cast<int64_t>(8));
    l.total = off;
    return l;
}

// The steps on `u`; the last X goes to o as bf16, or stays in the workspace (*x_out, times
// *sx_out) where o is NULL.
int orthogonalize_impl(const mlpblk_ortho_desc *d, const OrthoSource &u, void *o, void *workspace, const __half **x_out,
                       float *sx_out, int sms, cudaStream_t s) {
    const OrthoLayout l = ortho_layout(d);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    __half *x[2] = {reinterpret_cast<__half *>(ws + l.x[0]), reinterpret_cast<__half *>(ws + l.x[1])};
    __half *lo = reinterpret_cast<__half *>(ws + l.lo), *g[4];
    float *diag[3];
    for (int i = 0; i < 4; ++i) g[i] = reinterpret_cast<__half *>(ws + l.g[i]);
    for (int i = 0; i < 3; ++i) diag[i] = reinterpret_cast<float *>(ws + l.diag[i]);
    double *partial = reinterpret_cast<double *>(ws + l.partial);
    const bool tall = d->rows > d->cols;
    const int64_t n = tall ? d->rows : d->cols;
    // X is kept times a power of two near sqrt(n): an orthogonal matrix's entries are near 1 then
    const float sx = exp2f(roundf(0.5f * log2f(static_cast<float>(n))));
    int parts = 0;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ORTHO_NORM, s, launch_ortho_norm(u, d->rows * d->cols, d->batch, partial, &parts, sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ORTHO_SCALE, s,
                  launch_ortho_scale(u, d->rows, d->cols, d->batch, partial, parts, d->eps, sx, x[0], d->steps > 1 ? lo : nullptr, sms, s));
    if (ns_fused_fits(d->rows, d->cols, d->batch, sms)) {
        NsFusedProblem q = {};
        q.rows = d->rows;
        q.cols = d->cols;
        q.batch = d->batch;
        q.steps = d->steps;
        q.x[0] = x[0];
        q.x[1] = x[1];
        q.lo = lo;
        q.g = g[0];
        q.p = g[1];
        q.diag = diag[0];
        q.o = o;
        q.sx = sx;
        q.coefficients = d->coefficients;
        MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_STEPS, s, launch_ns_fused(q, s));
        *x_out = x[d->steps & 1];
        *sx_out = sx;
        return MLPBLK_OK;
    }
    // Two steps at a time (csrc/gemm_ns.cu) save 3 m^2 (n - m) operations a matrix for one launch
    // more: worth it from some 6 us of the tensor cores on, or where G has few tiles and a long K
    // (640 x 5000: 135 -> 121 us).  Never the last step: its X is kept in one fp16 value, and G's errors would reach
    // the result.  Nor a short side below 512: the joined polynomial's diagonal meets X's low part and its other entries do
    // not, which a dense strong direction of few rows feels (three directions in 64 x 4000: off by 6.0e-3, one step at a
    // time 1.1e-3; in 256 x 4000 2.3e-3 and 1.1e-3, in 512 x 4000 1.6e-3 and 1.1e-3).
    const int64_t m = tall ? d->cols : d->rows;
    const bool two = m >= 512 && ((n >= 2 * m && 3.0 * d->batch * m * m * (n - m) >= 8e9) || n >= 2048 + 4 * m);
    int at = 0;   // which of x holds X
    for (int i = 0; i < d->steps;) {
        const bool pair = two && i + 2 < d->steps;
        const float *c1 = d->coefficients[i], *c2 = d->coefficients[i + (pair ? 1 : 0)];
        const int after = i + (pair ? 2 : 1);
        const bool last = after == d->steps;
        NsProduct q = {};
        q.tall = tall;
        q.rows = d->rows;
        q.cols = d->cols;
        q.batch = d->batch;
        q.op = kNsGram;
        q.x = x[at];
        q.out = g[0];
        q.alpha = 1.0f / (sx * sx);
        MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_GRAM, s, launch_ns_product(q, sms, s));
        auto square = [&](const float *c, __half *to, float *rest) {
            NsProduct r = q;
            r.op = kNsSquare;
            r.y = g[0];
            r.b = c[1];
            r.c = c[2];
            r.out = to;
            r.diag_out = rest;
            return launch_ns_product(r, sms, s);
        };
        auto apply = [&](const __half *y, __half *to) {
            NsProduct r = q;
            r.op = kNsApply;
            r.y = y;
            r.p = g[1];
            r.diag = diag[0];
            r.a = c1[0];
            r.out = to;
            return launch_ns_product(r, sms, s);
        };
        MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_SQUARE, s, square(c1, g[1], diag[0]));
        if (pair) {
            MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_APPLY, s, apply(g[0], g[2]));
            MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_APPLY, s, apply(g[2], g[0]));
            MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_SQUARE, s, square(c2, g[3], diag[1]));
            NsProduct r = q;
            r.op = kNsJoin;
            r.y = g[1];
            r.p = g[3];
            r.diag = diag[1];
            r.diag2 = diag[0];
            r.a = c2[0];
            r.b = c1[0];
            r.out = g[2];
            r.diag_out = diag[2];
            MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_JOIN, s, launch_ns_product(r, sms, s));
        }
        q.op = kNsUpdate;
        q.p = g[pair ? 2 : 1];
        q.diag = diag[pair ? 2 : 0];
        q.a = pair ? c1[0] * c2[0] : c1[0];
        q.x_lo = !last ? lo : nullptr;
        q.out = x[at ^ 1];
        q.out_lo = after + 1 < d->steps ? lo : nullptr;
        q.o = last ? o : nullptr;
        q.alpha = 1.0f / sx;
        MLPBLK_LAUNCH(MLPBLK_KERNEL_NS_UPDATE, s, launch_ns_product(q, sms, s));
        i = after;
        at ^= 1;
    }
    *x_out = x[at];
    *sx_out = sx;
    return MLPBLK_OK;
}

}  // namespace

int mlpblk_moe_route(const mlpblk_route_desc *desc, const void *logits, const float *bias, int32_t *expert_idx,
                     float *routing_weights, void *stream) {
    MLPBLK_TRY(check_route_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(logits) || !aligned16(expert_idx) || !aligned16(routing_weights) || (bias && !aligned16(bias))) return MLPBLK_EINVAL;
    const int64_t n = desc->tokens * desc->top_k, row = desc->experts * element_bytes(desc->dtype);
    if (!apart({Span(expert_idx, n, 4), Span(routing_weights, n, 4)}, {Span(logits, desc->tokens, row), Span(bias, desc->experts, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ROUTE, s, launch_route(*desc, logits, bias, expert_idx, routing_weights, sms, s));
    return MLPBLK_OK;
}

int mlpblk_moe_route_backward(const mlpblk_route_desc *desc, const void *logits, const int32_t *expert_idx,
                              const float *d_routing_weights, void *d_logits, void *stream) {
    MLPBLK_TRY(check_route_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if (!aligned16(logits) || !aligned16(expert_idx) || !aligned16(d_routing_weights) || !aligned16(d_logits)) return MLPBLK_EINVAL;
    const int64_t n = desc->tokens * desc->top_k, row = desc->experts * element_bytes(desc->dtype);
    if (!apart({Span(d_logits, desc->tokens, row)},
               {Span(logits, desc->tokens, row), Span(expert_idx, n, 4), Span(d_routing_weights, n, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ROUTE_BWD, s, launch_route_bwd(*desc, logits, expert_idx, d_routing_weights, d_logits, sms, s));
    return MLPBLK_OK;
}

int mlpblk_add_rmsnorm(const mlpblk_norm_desc *desc, const void *x, const void *residual, const void *gamma,
                       void *sum, void *n, void *codes, float *scales, float *rstd, void *stream) {
    MLPBLK_TRY(check_norm_desc(desc));
    if (desc->tokens == 0) return MLPBLK_OK;
    if ((residual == nullptr) != (sum == nullptr) || (codes == nullptr) != (scales == nullptr) || (!n && !codes)) return MLPBLK_EINVAL;
    if (!aligned16(x) || !aligned16(gamma)) return MLPBLK_EINVAL;
    for (const void *p : {residual, static_cast<const void *>(sum), static_cast<const void *>(n), static_cast<const void *>(codes),
                          static_cast<const void *>(scales), static_cast<const void *>(rstd)})
        if (p && !aligned16(p)) return MLPBLK_EINVAL;
    const int64_t T = desc->tokens, e = element_bytes(desc->dtype), row = desc->width * e;
    const int64_t per = desc->block ? (desc->width + 127) / 128 : 1;
    if (!apart({Span(sum, T, row), Span(n, T, row), Span(codes, T, desc->width), Span(scales, T * per, 4), Span(rstd, T, 4)},
               {Span(x == sum ? nullptr : x, T, row), Span(residual == sum ? nullptr : residual, T, row), Span(gamma, desc->width, e)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ADD_NORM, s,
                  launch_add_rmsnorm(*desc, x, residual, gamma, sum, n, static_cast<uint8_t *>(codes), scales, rstd, sms, s));
    return MLPBLK_OK;
}

size_t mlpblk_add_rmsnorm_workspace_size(const mlpblk_norm_desc *desc) {
    if (check_norm_desc(desc) != MLPBLK_OK) return 0;
    int64_t parts = desc->tokens < kNormMaxParts ? desc->tokens : kNormMaxParts;
    if (parts < 1) parts = 1;
    return static_cast<size_t>(parts * norm_part_pitch(desc->width) * 4);
}

int mlpblk_add_rmsnorm_backward(const mlpblk_norm_desc *desc, const void *dn, const void *d_sum, const void *sum,
                                const float *rstd, const void *gamma, void *dx, float *dgamma, int32_t overwrite,
                                void *workspace, size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_norm_desc(desc));
    if ((overwrite != 0 && overwrite != 1) || !aligned16(dgamma)) return MLPBLK_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    if (desc->tokens == 0) {
        if (!overwrite) return MLPBLK_OK;
        MLPBLK_TRY(device_sms(&sms));
        MLPBLK_LAUNCH(MLPBLK_KERNEL_ADD_NORM_DG, s, launch_norm_dgamma(nullptr, 0, desc->width, dgamma, 1, s));
        return MLPBLK_OK;
    }
    if (!aligned16(dn) || !aligned16(sum) || !aligned16(rstd) || !aligned16(gamma) || !aligned16(dx) || !aligned16(workspace) ||
        (d_sum && !aligned16(d_sum)))
        return MLPBLK_EINVAL;
    const size_t need = mlpblk_add_rmsnorm_workspace_size(desc);
    if (workspace_bytes < need) return MLPBLK_EWORKSPACE;
    const int64_t T = desc->tokens, e = element_bytes(desc->dtype), row = desc->width * e;
    if (!apart({Span(dx, T, row), Span(dgamma, desc->width, 4), Span(workspace, static_cast<int64_t>(need), 1)},
               {Span(dn == dx ? nullptr : dn, T, row), Span(d_sum == dx ? nullptr : d_sum, T, row), Span(sum, T, row), Span(rstd, T, 4),
                Span(gamma, desc->width, e)}))
        return MLPBLK_EINVAL;
    MLPBLK_TRY(device_sms(&sms));
    float *part = static_cast<float *>(workspace);
    int parts = 0;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ADD_NORM_BWD, s, launch_add_rmsnorm_bwd(*desc, dn, d_sum, sum, rstd, gamma, dx, part, &parts, sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ADD_NORM_DG, s, launch_norm_dgamma(part, parts, desc->width, dgamma, overwrite, s));
    return MLPBLK_OK;
}

size_t mlpblk_orthogonalize_workspace_size(const mlpblk_ortho_desc *desc) {
    if (check_ortho_desc(desc) != MLPBLK_OK) return 0;
    return static_cast<size_t>(ortho_layout(desc).total);
}

int mlpblk_orthogonalize(const mlpblk_ortho_desc *desc, const void *u, void *o, void *workspace,
                         size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_ortho_desc(desc));
    if (!aligned16(u) || !aligned16(o) || !aligned16(workspace)) return MLPBLK_EINVAL;
    const int64_t need = ortho_layout(desc).total, n = desc->rows * desc->cols * desc->batch;
    if (workspace_bytes < static_cast<size_t>(need)) return MLPBLK_EWORKSPACE;
    if (!apart({Span(o, n, 2), Span(workspace, need, 1)}, {Span(u, n, element_bytes(desc->dtype))})) return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    OrthoSource src = {};
    src.u = u;
    src.dtype = desc->dtype;
    const __half *x;
    float sx;
    return orthogonalize_impl(desc, src, o, workspace, &x, &sx, sms, static_cast<cudaStream_t>(stream));
}

int mlpblk_muon_step(const mlpblk_ortho_desc *desc, const mlpblk_muon *hp, float *master, void *weight,
                     const float *grad, float *momentum, const float *grad_scale, void *workspace,
                     size_t workspace_bytes, void *stream) {
    MLPBLK_TRY(check_ortho_desc(desc));
    if (!hp || !isfinite(hp->lr) || !isfinite(hp->weight_decay) || !isfinite(hp->scale) || !(hp->lr >= 0.0f) ||
        !(hp->weight_decay >= 0.0f) || !(hp->momentum >= 0.0f && hp->momentum < 1.0f) || (hp->nesterov != 0 && hp->nesterov != 1))
        return MLPBLK_EINVAL;
    if (!aligned16(master) || !aligned16(grad) || !aligned16(momentum) || !aligned16(workspace) || (weight && !aligned16(weight)) ||
        (grad_scale && (reinterpret_cast<uintptr_t>(grad_scale) & 3u)))
        return MLPBLK_EINVAL;
    const int64_t need = ortho_layout(desc).total, n = desc->rows * desc->cols * desc->batch;
    if (workspace_bytes < static_cast<size_t>(need)) return MLPBLK_EWORKSPACE;
    if (!apart({Span(master, n, 4), Span(momentum, n, 4), Span(weight, n, element_bytes(desc->dtype)), Span(workspace, need, 1)},
               {Span(grad, n, 4), Span(grad_scale, 1, 4)}))
        return MLPBLK_EINVAL;
    int sms = 0;
    MLPBLK_TRY(device_sms(&sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    OrthoSource src = {};
    src.momentum = momentum;
    src.grad = grad;
    src.grad_scale = grad_scale;
    src.beta = hp->momentum;
    src.nesterov = hp->nesterov;
    const __half *x;
    float sx;
    MLPBLK_TRY(orthogonalize_impl(desc, src, nullptr, workspace, &x, &sx, sms, s));
    MLPBLK_LAUNCH(MLPBLK_KERNEL_MUON_APPLY, s,
                  launch_muon_apply(x, desc->rows, desc->cols, desc->batch, 1.0f - hp->lr * hp->weight_decay, hp->lr * hp->scale / sx,
                                    master, weight, desc->dtype, sms, s));
    return MLPBLK_OK;
}

int mlpblk_moe_backward(const mlpblk_moe_desc *desc, const void *dy, const void *x, const void *gamma,
                        const void *w1s, const void *w2s, const float *routing_weights, const void *saved, void *dx,
                        float *d_routing_weights, float *dgamma, float *dw1s, float *dw2s, void *workspace,
                        size_t workspace_bytes, void *stream) {
    return moe_backward_entry(desc, dy, x, gamma, w1s, w2s, routing_weights, saved, dx, d_routing_weights, dgamma,
                              dw1s, dw2s, workspace, workspace_bytes, stream, false);
}

int mlpblk_moe_backward_overwrite(const mlpblk_moe_desc *desc, const void *dy, const void *x, const void *gamma,
                                  const void *w1s, const void *w2s, const float *routing_weights, const void *saved,
                                  void *dx, float *d_routing_weights, float *dgamma, float *dw1s, float *dw2s,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    return moe_backward_entry(desc, dy, x, gamma, w1s, w2s, routing_weights, saved, dx, d_routing_weights, dgamma,
                              dw1s, dw2s, workspace, workspace_bytes, stream, true);
}

int mlpblk_zero_grads(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2, void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (!aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2)) return MLPBLK_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_ZERO_GRADS, s,
                  launch_grads(true, 0.0f, dgamma, d, dw1, F * d, dw2, F * d, s));
    return MLPBLK_OK;
}

int mlpblk_scale_grads(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2, float sc,
                       void *stream) {
    MLPBLK_TRY(check_desc(desc));
    if (!aligned16(dgamma) || !aligned16(dw1) || !aligned16(dw2)) return MLPBLK_EINVAL;
    if (!isfinite(sc)) return MLPBLK_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t d = desc->d_model, F = desc->ffn;
    MLPBLK_LAUNCH(MLPBLK_KERNEL_SCALE_GRADS, s,
                  launch_grads(false, sc, dgamma, d, dw1, F * d, dw2, F * d, s));
    return MLPBLK_OK;
}

int mlpblk_set_rmsnorm_mode(int mode) {
    if (mode != MLPBLK_RMSNORM_STATS_PASS && mode != MLPBLK_RMSNORM_IN_W1_PROLOGUE) return MLPBLK_EINVAL;
    g_rms_mode = mode;
    return MLPBLK_OK;
}

int mlpblk_set_test_fault(int fault) {
    if (fault != MLPBLK_TEST_FAULT_NONE && fault != MLPBLK_TEST_FAULT_SKIP_LOADS) return MLPBLK_EINVAL;
    g_test_fault = fault;
    return MLPBLK_OK;
}

int mlpblk_trace_begin(void **events, int *kinds, int capacity) {
    if (!events || !kinds || capacity < 1) return MLPBLK_EINVAL;
    g_trace.events = reinterpret_cast<cudaEvent_t *>(events);
    g_trace.kinds = kinds;
    g_trace.capacity = capacity;
    g_trace.count = 0;
    g_trace.on = true;
    return MLPBLK_OK;
}

int mlpblk_trace_end(void) {
    g_trace.on = false;
    return g_trace.count;
}

const char *mlpblk_cuda_error_string(void) {
    if (g_last_cuda_error == 0) return "no CUDA error recorded";
    return cudaGetErrorString(static_cast<cudaError_t>(g_last_cuda_error));
}

int mlpblk_last_error(void) {
    if (cuda_status(cudaDeviceSynchronize()) != MLPBLK_OK) return MLPBLK_ECUDA;
    const int a = take_device_error_gemm_fwd();
    const int b = take_device_error_gemm_bwd();
    const int c = take_device_error_gemm_f8();
    const int f = take_device_error_gemm_f4();
    const int n = take_device_error_gemm_ns();
    const int r = take_device_error_rowops();
    if (n != MLPBLK_OK && a == MLPBLK_OK && b == MLPBLK_OK && c == MLPBLK_OK && f == MLPBLK_OK) return n;
    return a != MLPBLK_OK ? a : (b != MLPBLK_OK ? b : (c != MLPBLK_OK ? c : (f != MLPBLK_OK ? f : r)));
}

}  // extern "C"
