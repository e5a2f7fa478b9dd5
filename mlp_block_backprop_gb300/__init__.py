"""Python binding of libmlpblk.so, the GB300 forward/backward of the pre-norm
residual ReLU² MLP block (C ABI in include/mlpblk.h).

Argument marshalling only: every step of the block runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (device memory and streams are the
only things torch provides); the functions keep the C names and raise
``MlpBlkError`` on a non-zero status.  Importing this package fails loudly when
the library has not been built: there is no fallback.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmlpblk.so")
# csrc/pycalls.c as built for this interpreter: the name carries its ABI tag
CALLS_PATH = os.path.join(_HERE, "_mlpblk_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])

MLPBLK_OK = 0
MLPBLK_EINVAL = 1
MLPBLK_ENOTSUP = 2
MLPBLK_EWORKSPACE = 3
MLPBLK_ECUDA = 4
MLPBLK_ETIMEOUT = 5
MLPBLK_ENODEV = 6
MLPBLK_BF16 = 1
MLPBLK_FP32 = 2

EXPORTED = ("mlpblk_workspace_size", "mlpblk_forward", "mlpblk_backward", "mlpblk_zero_grads",
            "mlpblk_scale_grads", "mlpblk_last_error", "mlpblk_strerror", "mlpblk_version",
            "mlpblk_trace_begin", "mlpblk_trace_end", "mlpblk_cuda_error_string",
            "mlpblk_rmsnorm_backward_noalloc", "mlpblk_set_test_fault",
            "mlpblk_workspace_size_recompute", "mlpblk_forward_recompute", "mlpblk_backward_recompute",
            "mlpblk_grad_norm", "mlpblk_clip_grads", "mlpblk_adamw_step", "mlpblk_set_rmsnorm_mode",
            "mlpblk_workspace_size_fp8", "mlpblk_forward_fp8", "mlpblk_backward_fp8",
            "mlpblk_fp8_weights_size", "mlpblk_fp8_quantize_weights", "mlpblk_forward_fp8_prequant",
            "mlpblk_backward_fp8_prequant",
            "mlpblk_moe_saved_size", "mlpblk_moe_workspace_size", "mlpblk_moe_forward", "mlpblk_moe_backward",
            "mlpblk_fold_weights", "mlpblk_forward_prefolded", "mlpblk_backward_overwrite",
            "mlpblk_moe_backward_overwrite", "mlpblk_backward_fp8_overwrite",
            "mlpblk_backward_fp8_prequant_overwrite",
            "mlpblk_moe_sort_rows", "mlpblk_moe_sort", "mlpblk_moe_permute", "mlpblk_moe_permute_backward",
            "mlpblk_moe_unpermute", "mlpblk_moe_unpermute_backward",
            "mlpblk_fp4_codes_size", "mlpblk_fp4_scales_size", "mlpblk_fp4_quantize", "mlpblk_fp4_dequantize",
            "mlpblk_fp4_matmul", "mlpblk_fp4_matmul_grouped", "mlpblk_fp4_wgrad_grouped",
            "mlpblk_fp4_product_kernel",
            "mlpblk_moe_route", "mlpblk_moe_route_backward",
            "mlpblk_add_rmsnorm", "mlpblk_add_rmsnorm_workspace_size", "mlpblk_add_rmsnorm_backward",
            "mlpblk_orthogonalize_workspace_size", "mlpblk_orthogonalize", "mlpblk_muon_step")
MLPBLK_ROUTE_SOFTMAX = 0
MLPBLK_ROUTE_SIGMOID = 1
MLPBLK_ROUTE_MAX_TOP_K = 16
MLPBLK_ORTHO_MAX_STEPS = 16
MLPBLK_FP4_KERNEL_PAIR_TMA = 256
MLPBLK_FP4_KERNEL_PAIR = 257
MLPBLK_FP4_ACT_NONE = 0
MLPBLK_FP4_ACT_RELU2 = 1
MLPBLK_RMSNORM_STATS_PASS = 0
MLPBLK_RMSNORM_IN_W1_PROLOGUE = 1
MLPBLK_TEST_FAULT_NONE = 0
MLPBLK_TEST_FAULT_SKIP_LOADS = 1

KERNEL_NAMES = {1: "fold_gamma", 2: "gemm_fwd_w1", 3: "gemm_fwd_w2", 4: "gemm_dgrad_h",
                5: "gemm_wgrad_w2", 6: "gemm_dgrad_n", 7: "gemm_wgrad_w1", 8: "norm_bwd",
                9: "dgamma_reduce", 10: "zero_grads", 11: "scale_grads", 12: "rstd",
                13: "grad_norm", 14: "clip_grads", 15: "adamw", 16: "grad_norm_final",
                17: "quant_amax", 18: "quant_scale", 19: "quant_apply", 20: "norm_quant",
                21: "moe_route", 22: "moe_gather", 23: "moe_combine", 24: "moe_dp", 25: "moe_scatter",
                26: "sort", 27: "permute", 28: "unpermute", 29: "unpermute_bwd",
                30: "fp4_quant", 31: "fp4_dequant", 32: "fp4_gemm", 33: "route", 34: "route_bwd",
                35: "add_norm", 36: "add_norm_bwd", 37: "add_norm_dgamma", 38: "ortho_norm", 39: "ortho_scale",
                40: "ns_gram", 41: "ns_square", 42: "ns_update", 43: "muon_apply",
                44: "ns_apply", 45: "ns_join", 46: "ns_steps"}


class MlpBlkError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        extra = ""
        if code == MLPBLK_ECUDA:
            extra = "; CUDA: " + lib.mlpblk_cuda_error_string().decode()
        super().__init__(f"{where}: status {code} ({strerror(code)}{extra})")


class Desc(ctypes.Structure):
    """mlpblk_desc: shape of one microbatch through one block."""
    _fields_ = [("tokens", ctypes.c_int64), ("d_model", ctypes.c_int64), ("ffn", ctypes.c_int64),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class MoeDesc(ctypes.Structure):
    """mlpblk_moe_desc: the dense descriptor plus the expert count and top-k."""
    _fields_ = [("base", Desc), ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32)]


class SortDesc(ctypes.Structure):
    """mlpblk_sort_desc: tokens sorted by expert."""
    _fields_ = [("tokens", ctypes.c_int64), ("width", ctypes.c_int64), ("experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("pad", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Fp4Desc(ctypes.Structure):
    """mlpblk_fp4_desc: an MXFP4 matrix (a batch of them) and what it is made from."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("transposed", ctypes.c_int32), ("act", ctypes.c_int32),
                ("source_rows", ctypes.c_int64)]


class Fp4MatmulDesc(ctypes.Structure):
    """mlpblk_fp4_matmul_desc: a product of MXFP4 matrices."""
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("out_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("pad", ctypes.c_int32), ("max_rows", ctypes.c_int64)]


class RouteDesc(ctypes.Structure):
    """mlpblk_route_desc: the router of routed experts."""
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    """mlpblk_norm_desc: the residual sum with RMSNorm."""
    _fields_ = [("tokens", ctypes.c_int64), ("width", ctypes.c_int64), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("block", ctypes.c_int32)]


class OrthoDesc(ctypes.Structure):
    """mlpblk_ortho_desc: an orthogonalised update."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("steps", ctypes.c_int32), ("eps", ctypes.c_float),
                ("coefficients", ctypes.c_float * 3 * MLPBLK_ORTHO_MAX_STEPS)]


class Muon(ctypes.Structure):
    """mlpblk_muon: Muon's hyper-parameters."""
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale", ctypes.c_float), ("nesterov", ctypes.c_int32)]


class Param(ctypes.Structure):
    """mlpblk_param: one tensor of an AdamW update."""
    _fields_ = [("master", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n", ctypes.c_int64), ("decay", ctypes.c_int32)]


class AdamW(ctypes.Structure):
    """mlpblk_adamw: AdamW hyper-parameters."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run mlp_block_backprop_gb300.build.build_library() "
                          "(or __graft_entry__.build()) first; there is no non-CUDA fallback")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    pd = ctypes.POINTER(Desc)
    lib.mlpblk_workspace_size.argtypes = [pd]
    lib.mlpblk_workspace_size.restype = sz
    lib.mlpblk_forward.argtypes = [pd] + [vp] * 9 + [sz, vp]
    lib.mlpblk_forward.restype = i32
    lib.mlpblk_backward.argtypes = [pd] + [vp] * 13 + [sz, vp]
    lib.mlpblk_fold_weights.argtypes = [pd, vp, vp, vp, vp]
    lib.mlpblk_fold_weights.restype = i32
    lib.mlpblk_forward_prefolded.argtypes = [pd] + [vp] * 8 + [sz, vp]
    lib.mlpblk_forward_prefolded.restype = i32
    lib.mlpblk_backward.restype = i32
    lib.mlpblk_backward_overwrite.argtypes = lib.mlpblk_backward.argtypes
    lib.mlpblk_backward_overwrite.restype = i32
    lib.mlpblk_workspace_size_recompute.argtypes = [pd]
    lib.mlpblk_workspace_size_recompute.restype = sz
    lib.mlpblk_forward_recompute.argtypes = [pd] + [vp] * 7 + [sz, vp]
    lib.mlpblk_forward_recompute.restype = i32
    lib.mlpblk_backward_recompute.argtypes = [pd] + [vp] * 11 + [sz, vp]
    lib.mlpblk_backward_recompute.restype = i32
    lib.mlpblk_grad_norm.argtypes = [pd, vp, vp, vp, f32, vp, vp, vp, sz, vp]
    lib.mlpblk_grad_norm.restype = i32
    lib.mlpblk_clip_grads.argtypes = [pd, vp, vp, vp, vp, vp]
    lib.mlpblk_clip_grads.restype = i32
    lib.mlpblk_adamw_step.argtypes = [ctypes.POINTER(Param), i32, ctypes.POINTER(AdamW), ctypes.c_int64, i32, vp, vp]
    lib.mlpblk_adamw_step.restype = i32
    lib.mlpblk_workspace_size_fp8.argtypes = [pd]
    lib.mlpblk_workspace_size_fp8.restype = sz
    lib.mlpblk_forward_fp8.argtypes = [pd] + [vp] * 11 + [sz, vp]
    lib.mlpblk_forward_fp8.restype = i32
    lib.mlpblk_backward_fp8.argtypes = [pd] + [vp] * 15 + [sz, vp]
    lib.mlpblk_backward_fp8.restype = i32
    lib.mlpblk_fp8_weights_size.argtypes = [pd]
    lib.mlpblk_fp8_weights_size.restype = sz
    lib.mlpblk_fp8_quantize_weights.argtypes = [pd, vp, vp, vp, vp, sz, vp, sz, vp]
    lib.mlpblk_fp8_quantize_weights.restype = i32
    lib.mlpblk_forward_fp8_prequant.argtypes = [pd] + [vp] * 9 + [sz, vp]
    lib.mlpblk_forward_fp8_prequant.restype = i32
    lib.mlpblk_backward_fp8_prequant.argtypes = [pd] + [vp] * 14 + [sz, vp]
    lib.mlpblk_backward_fp8_prequant.restype = i32
    lib.mlpblk_backward_fp8_overwrite.argtypes = lib.mlpblk_backward_fp8.argtypes
    lib.mlpblk_backward_fp8_overwrite.restype = i32
    lib.mlpblk_backward_fp8_prequant_overwrite.argtypes = lib.mlpblk_backward_fp8_prequant.argtypes
    lib.mlpblk_backward_fp8_prequant_overwrite.restype = i32
    pm = ctypes.POINTER(MoeDesc)
    lib.mlpblk_moe_saved_size.argtypes = [pm]
    lib.mlpblk_moe_saved_size.restype = sz
    lib.mlpblk_moe_workspace_size.argtypes = [pm]
    lib.mlpblk_moe_workspace_size.restype = sz
    lib.mlpblk_moe_forward.argtypes = [pm] + [vp] * 8 + [sz, vp, sz, vp]
    lib.mlpblk_moe_forward.restype = i32
    lib.mlpblk_moe_backward.argtypes = [pm] + [vp] * 13 + [sz, vp]
    lib.mlpblk_moe_backward.restype = i32
    lib.mlpblk_moe_backward_overwrite.argtypes = lib.mlpblk_moe_backward.argtypes
    lib.mlpblk_moe_backward_overwrite.restype = i32
    ps, pf, pp, i64 = ctypes.POINTER(SortDesc), ctypes.POINTER(Fp4Desc), ctypes.POINTER(Fp4MatmulDesc), ctypes.c_int64
    lib.mlpblk_moe_sort_rows.argtypes = [ps]
    lib.mlpblk_moe_sort_rows.restype = i64
    lib.mlpblk_moe_sort.argtypes = [ps] + [vp] * 6
    lib.mlpblk_moe_sort.restype = i32
    lib.mlpblk_moe_permute.argtypes = [ps] + [vp] * 6
    lib.mlpblk_moe_permute.restype = i32
    lib.mlpblk_moe_permute_backward.argtypes = [ps] + [vp] * 4
    lib.mlpblk_moe_permute_backward.restype = i32
    lib.mlpblk_moe_unpermute.argtypes = [ps] + [vp] * 6
    lib.mlpblk_moe_unpermute.restype = i32
    lib.mlpblk_moe_unpermute_backward.argtypes = [ps] + [vp] * 9
    lib.mlpblk_moe_unpermute_backward.restype = i32
    lib.mlpblk_fp4_codes_size.argtypes = [pf]
    lib.mlpblk_fp4_codes_size.restype = sz
    lib.mlpblk_fp4_scales_size.argtypes = [pf]
    lib.mlpblk_fp4_scales_size.restype = sz
    lib.mlpblk_fp4_quantize.argtypes = [pf, vp, vp, i32, vp, vp, vp]
    lib.mlpblk_fp4_quantize.restype = i32
    lib.mlpblk_fp4_dequantize.argtypes = [pf] + [vp] * 4
    lib.mlpblk_fp4_dequantize.restype = i32
    lib.mlpblk_fp4_matmul.argtypes = [pp] + [vp] * 6
    lib.mlpblk_fp4_matmul.restype = i32
    lib.mlpblk_fp4_matmul_grouped.argtypes = [pp] + [vp] * 8
    lib.mlpblk_fp4_matmul_grouped.restype = i32
    lib.mlpblk_fp4_wgrad_grouped.argtypes = [pp] + [vp] * 7
    lib.mlpblk_fp4_wgrad_grouped.restype = i32
    lib.mlpblk_fp4_product_kernel.argtypes = [pp, i32, i32]
    lib.mlpblk_fp4_product_kernel.restype = i32
    pr, pn, po = ctypes.POINTER(RouteDesc), ctypes.POINTER(NormDesc), ctypes.POINTER(OrthoDesc)
    lib.mlpblk_moe_route.argtypes = [pr] + [vp] * 5
    lib.mlpblk_moe_route.restype = i32
    lib.mlpblk_moe_route_backward.argtypes = [pr] + [vp] * 5
    lib.mlpblk_moe_route_backward.restype = i32
    lib.mlpblk_add_rmsnorm.argtypes = [pn] + [vp] * 9
    lib.mlpblk_add_rmsnorm.restype = i32
    lib.mlpblk_add_rmsnorm_workspace_size.argtypes = [pn]
    lib.mlpblk_add_rmsnorm_workspace_size.restype = sz
    lib.mlpblk_add_rmsnorm_backward.argtypes = [pn] + [vp] * 7 + [i32, vp, sz, vp]
    lib.mlpblk_add_rmsnorm_backward.restype = i32
    lib.mlpblk_orthogonalize_workspace_size.argtypes = [po]
    lib.mlpblk_orthogonalize_workspace_size.restype = sz
    lib.mlpblk_orthogonalize.argtypes = [po, vp, vp, vp, sz, vp]
    lib.mlpblk_orthogonalize.restype = i32
    lib.mlpblk_muon_step.argtypes = [po, ctypes.POINTER(Muon)] + [vp] * 6 + [sz, vp]
    lib.mlpblk_muon_step.restype = i32
    lib.mlpblk_zero_grads.argtypes = [pd, vp, vp, vp, vp]
    lib.mlpblk_zero_grads.restype = i32
    lib.mlpblk_scale_grads.argtypes = [pd, vp, vp, vp, f32, vp]
    lib.mlpblk_scale_grads.restype = i32
    lib.mlpblk_last_error.argtypes = []
    lib.mlpblk_last_error.restype = i32
    lib.mlpblk_strerror.argtypes = [i32]
    lib.mlpblk_strerror.restype = ctypes.c_char_p
    lib.mlpblk_version.argtypes = []
    lib.mlpblk_version.restype = i32
    lib.mlpblk_trace_begin.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int), i32]
    lib.mlpblk_trace_begin.restype = i32
    lib.mlpblk_rmsnorm_backward_noalloc.argtypes = [pd] + [vp] * 8
    lib.mlpblk_rmsnorm_backward_noalloc.restype = i32
    lib.mlpblk_set_rmsnorm_mode.argtypes = [i32]
    lib.mlpblk_set_rmsnorm_mode.restype = i32
    lib.mlpblk_set_test_fault.argtypes = [i32]
    lib.mlpblk_set_test_fault.restype = i32
    lib.mlpblk_cuda_error_string.argtypes = []
    lib.mlpblk_cuda_error_string.restype = ctypes.c_char_p
    lib.mlpblk_trace_end.argtypes = []
    lib.mlpblk_trace_end.restype = i32
    return lib


lib = _load()


class _Calls:
    """The latency-bound entry points for the classes below, descriptors and tensors by
    address: csrc/pycalls.c where it was built for this interpreter (it needs Python's
    headers), else the same functions through ctypes."""

    def __init__(self):
        native = self._native()
        for name in ("moe_sort", "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
                     "fp4_quantize", "fp4_dequantize", "fp4_matmul", "fp4_matmul_grouped", "fp4_wgrad_grouped",
                     "moe_route", "moe_route_backward", "add_rmsnorm", "add_rmsnorm_backward", "orthogonalize"):
            setattr(self, name, getattr(native, "mlpblk_" + name) if native else self._ctypes("mlpblk_" + name))
        self.native = native is not None

    @staticmethod
    def _native():
        """The module at CALLS_PATH, or None.  By its path: an import would also take a
        file without an ABI tag, whichever interpreter it was built for."""
        if not os.path.exists(CALLS_PATH):
            return None
        spec = importlib.util.spec_from_file_location(__name__ + "._mlpblk_calls", CALLS_PATH)
        try:
            native = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(native)
        except ImportError:
            return None
        return native

    @staticmethod
    def _ctypes(name):
        f = getattr(lib, name)
        desc = f.argtypes[0]
        return lambda d, *a: f(ctypes.cast(d, desc), *a)


_calls = _Calls()


def strerror(code: int) -> str:
    return lib.mlpblk_strerror(int(code)).decode()


def make_desc(tokens: int, d_model: int, ffn: int, eps: float = 1e-6, dtype: int = MLPBLK_BF16) -> Desc:
    return Desc(int(tokens), int(d_model), int(ffn), float(eps), int(dtype))


class _Torch:
    """What the calls need of torch, looked up once (torch is imported with the first
    call, not with this package)."""
    _one = None

    @staticmethod
    def get():
        if _Torch._one is None:
            import torch
            o = _Torch()
            o.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            # the handle of a device's current stream; without the raw getter, through
            # the Stream object (3 us a call instead of 0.2 on a Grace core)
            o.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                   lambda dev: torch.cuda.current_stream(dev).cuda_stream)
            o.int32, o.uint8, o.float32, o.bfloat16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16
            o.row = {MLPBLK_BF16: torch.bfloat16, MLPBLK_FP32: torch.float32}
            o.code = {torch.bfloat16: MLPBLK_BF16, torch.float32: MLPBLK_FP32, "bf16": MLPBLK_BF16, "f32": MLPBLK_FP32}
            _Torch._one = o
        return _Torch._one


def _ptr(t):
    """Device address of a tensor, an int address, or None (NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        t = _Torch.get()
        return t.raw_stream(t.device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc, where):
    if rc != MLPBLK_OK:
        raise MlpBlkError(rc, where)


def mlpblk_workspace_size(desc: Desc) -> int:
    return int(lib.mlpblk_workspace_size(ctypes.byref(desc)))


def mlpblk_forward(desc, x, gamma, w1, w2, y, h_saved, a_saved, rstd_saved, workspace,
                   workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    rc = lib.mlpblk_forward(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(w1), _ptr(w2), _ptr(y),
                            _ptr(h_saved), _ptr(a_saved), _ptr(rstd_saved), _ptr(workspace),
                            nbytes, _stream(stream))
    _check(rc, "mlpblk_forward")


def mlpblk_fold_weights(desc, gamma, w1, w1g, stream=None):
    _check(lib.mlpblk_fold_weights(ctypes.byref(desc), _ptr(gamma), _ptr(w1), _ptr(w1g), _stream(stream)),
           "mlpblk_fold_weights")


def mlpblk_forward_prefolded(desc, x, w1g, w2, y, h_saved, a_saved, rstd_saved, workspace,
                             workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    rc = lib.mlpblk_forward_prefolded(ctypes.byref(desc), _ptr(x), _ptr(w1g), _ptr(w2), _ptr(y),
                                      _ptr(h_saved), _ptr(a_saved), _ptr(rstd_saved), _ptr(workspace),
                                      nbytes, _stream(stream))
    _check(rc, "mlpblk_forward_prefolded")


def mlpblk_backward(desc, dy, x, gamma, w1, w2, h_saved, a_saved, rstd_saved, dx, dgamma, dw1, dw2,
                    workspace, workspace_bytes=None, stream=None, overwrite=False):
    """overwrite=True calls mlpblk_backward_overwrite (gradients written, not added into)."""
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    fn = lib.mlpblk_backward_overwrite if overwrite else lib.mlpblk_backward
    rc = fn(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(w1), _ptr(w2),
            _ptr(h_saved), _ptr(a_saved), _ptr(rstd_saved), _ptr(dx), _ptr(dgamma),
            _ptr(dw1), _ptr(dw2), _ptr(workspace), nbytes, _stream(stream))
    _check(rc, "mlpblk_backward_overwrite" if overwrite else "mlpblk_backward")


def mlpblk_workspace_size_recompute(desc: Desc) -> int:
    return int(lib.mlpblk_workspace_size_recompute(ctypes.byref(desc)))


def mlpblk_forward_recompute(desc, x, gamma, w1, w2, y, rstd_saved, workspace, workspace_bytes=None,
                             stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    rc = lib.mlpblk_forward_recompute(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(w1), _ptr(w2),
                                      _ptr(y), _ptr(rstd_saved), _ptr(workspace), nbytes, _stream(stream))
    _check(rc, "mlpblk_forward_recompute")


def mlpblk_backward_recompute(desc, dy, x, gamma, w1, w2, rstd_saved, dx, dgamma, dw1, dw2, workspace,
                              workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    rc = lib.mlpblk_backward_recompute(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(w1),
                                       _ptr(w2), _ptr(rstd_saved), _ptr(dx), _ptr(dgamma), _ptr(dw1),
                                       _ptr(dw2), _ptr(workspace), nbytes, _stream(stream))
    _check(rc, "mlpblk_backward_recompute")


def mlpblk_grad_norm(desc, dgamma, dw1, dw2, max_norm, norm_out, clip_scale_out, workspace,
                     workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    rc = lib.mlpblk_grad_norm(ctypes.byref(desc), _ptr(dgamma), _ptr(dw1), _ptr(dw2), float(max_norm),
                              _ptr(norm_out), _ptr(clip_scale_out), _ptr(workspace), nbytes, _stream(stream))
    _check(rc, "mlpblk_grad_norm")


def mlpblk_clip_grads(desc, dgamma, dw1, dw2, clip_scale, stream=None):
    rc = lib.mlpblk_clip_grads(ctypes.byref(desc), _ptr(dgamma), _ptr(dw1), _ptr(dw2), _ptr(clip_scale),
                               _stream(stream))
    _check(rc, "mlpblk_clip_grads")


def mlpblk_adamw_step(params, hp, step, dtype, grad_scale=None, stream=None):
    """params: sequence of (master, weight, grad, m, v, decay) tensors/flags; hp: AdamW."""
    arr = (Param * len(params))()
    for i, (master, weight, grad, m, v, decay) in enumerate(params):
        arr[i] = Param(_ptr(master), _ptr(weight), _ptr(grad), _ptr(m), _ptr(v), master.numel(), int(decay))
    rc = lib.mlpblk_adamw_step(arr, len(params), ctypes.byref(hp), int(step), int(dtype), _ptr(grad_scale),
                               _stream(stream))
    _check(rc, "mlpblk_adamw_step")


def mlpblk_workspace_size_fp8(desc: Desc) -> int:
    return int(lib.mlpblk_workspace_size_fp8(ctypes.byref(desc)))


def mlpblk_forward_fp8(desc, x, gamma, w1, w2, y, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved,
                       workspace, workspace_bytes=None, stream=None):
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    rc = lib.mlpblk_forward_fp8(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(w1), _ptr(w2), _ptr(y),
                                _ptr(h_saved), _ptr(a8_saved), _ptr(n8_saved), _ptr(rstd_saved),
                                _ptr(scales_saved), _ptr(workspace), nbytes, _stream(stream))
    _check(rc, "mlpblk_forward_fp8")


def mlpblk_backward_fp8(desc, dy, x, gamma, w1, w2, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved,
                        dx, dgamma, dw1, dw2, workspace, workspace_bytes=None, stream=None, overwrite=False):
    """overwrite=True calls mlpblk_backward_fp8_overwrite (gradients set, not added into)."""
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    fn = lib.mlpblk_backward_fp8_overwrite if overwrite else lib.mlpblk_backward_fp8
    rc = fn(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(w1), _ptr(w2),
            _ptr(h_saved), _ptr(a8_saved), _ptr(n8_saved), _ptr(rstd_saved),
            _ptr(scales_saved), _ptr(dx), _ptr(dgamma), _ptr(dw1), _ptr(dw2),
            _ptr(workspace), nbytes, _stream(stream))
    _check(rc, "mlpblk_backward_fp8_overwrite" if overwrite else "mlpblk_backward_fp8")


def mlpblk_fp8_weights_size(desc: Desc) -> int:
    return int(lib.mlpblk_fp8_weights_size(ctypes.byref(desc)))


def mlpblk_fp8_quantize_weights(desc, gamma, w1, w2, wq, workspace, stream=None):
    rc = lib.mlpblk_fp8_quantize_weights(ctypes.byref(desc), _ptr(gamma), _ptr(w1), _ptr(w2), _ptr(wq),
                                         wq.numel() * wq.element_size(), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "mlpblk_fp8_quantize_weights")


def mlpblk_forward_fp8_prequant(desc, x, wq, y, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved,
                                workspace, stream=None):
    rc = lib.mlpblk_forward_fp8_prequant(ctypes.byref(desc), _ptr(x), _ptr(wq), _ptr(y), _ptr(h_saved),
                                         _ptr(a8_saved), _ptr(n8_saved), _ptr(rstd_saved), _ptr(scales_saved),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream))
    _check(rc, "mlpblk_forward_fp8_prequant")


def mlpblk_backward_fp8_prequant(desc, dy, x, gamma, wq, h_saved, a8_saved, n8_saved, rstd_saved, scales_saved,
                                 dx, dgamma, dw1, dw2, workspace, stream=None, overwrite=False):
    """overwrite=True calls mlpblk_backward_fp8_prequant_overwrite (gradients set, not added into)."""
    fn = lib.mlpblk_backward_fp8_prequant_overwrite if overwrite else lib.mlpblk_backward_fp8_prequant
    rc = fn(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(wq),
            _ptr(h_saved), _ptr(a8_saved), _ptr(n8_saved), _ptr(rstd_saved),
            _ptr(scales_saved), _ptr(dx), _ptr(dgamma), _ptr(dw1), _ptr(dw2),
            _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream))
    _check(rc, "mlpblk_backward_fp8_prequant_overwrite" if overwrite else "mlpblk_backward_fp8_prequant")


def make_moe_desc(tokens, d_model, ffn, experts, top_k, eps=1e-6) -> MoeDesc:
    return MoeDesc(make_desc(tokens, d_model, ffn, eps, MLPBLK_BF16), int(experts), int(top_k))


def mlpblk_moe_saved_size(desc: MoeDesc) -> int:
    return int(lib.mlpblk_moe_saved_size(ctypes.byref(desc)))


def mlpblk_moe_workspace_size(desc: MoeDesc) -> int:
    return int(lib.mlpblk_moe_workspace_size(ctypes.byref(desc)))


def mlpblk_moe_forward(desc, x, gamma, w1s, w2s, expert_idx, routing_weights, y, saved, workspace, stream=None):
    rc = lib.mlpblk_moe_forward(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(w1s), _ptr(w2s), _ptr(expert_idx),
                                _ptr(routing_weights), _ptr(y), _ptr(saved), saved.numel(), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _check(rc, "mlpblk_moe_forward")


def mlpblk_moe_backward(desc, dy, x, gamma, w1s, w2s, routing_weights, saved, dx, d_routing_weights, dgamma,
                        dw1s, dw2s, workspace, stream=None, overwrite=False):
    """overwrite=True calls mlpblk_moe_backward_overwrite (gradients written, not added into)."""
    fn = lib.mlpblk_moe_backward_overwrite if overwrite else lib.mlpblk_moe_backward
    rc = fn(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(w1s), _ptr(w2s),
            _ptr(routing_weights), _ptr(saved), _ptr(dx), _ptr(d_routing_weights),
            _ptr(dgamma), _ptr(dw1s), _ptr(dw2s), _ptr(workspace), workspace.numel(),
            _stream(stream))
    _check(rc, "mlpblk_moe_backward_overwrite" if overwrite else "mlpblk_moe_backward")


class MoeBuffers:
    """Device buffers of one routed-expert block (bf16 tensors, fp32 routing weights
    and gradients, int32 expert ids)."""

    def __init__(self, tokens, d_model, ffn, experts, top_k, eps=1e-6, device="cuda"):
        import torch
        self.desc = make_moe_desc(tokens, d_model, ffn, experts, top_k, eps)
        T, d, F, E, k = tokens, d_model, ffn, experts, top_k
        e = dict(device=device)
        bf = torch.bfloat16
        self.gamma = torch.empty(d, dtype=bf, **e)
        self.w1s = torch.empty(E, F, d, dtype=bf, **e)
        self.w2s = torch.empty(E, d, F, dtype=bf, **e)
        self.x = torch.empty(T, d, dtype=bf, **e)
        self.dy = torch.empty(T, d, dtype=bf, **e)
        self.y = torch.empty(T, d, dtype=bf, **e)
        self.dx = torch.empty(T, d, dtype=bf, **e)
        self.idx = torch.empty(T, k, dtype=torch.int32, **e)
        self.p = torch.empty(T, k, dtype=torch.float32, **e)
        self.dp = torch.empty(T, k, dtype=torch.float32, **e)
        self.dgamma = torch.zeros(d, dtype=torch.float32, **e)
        self.dw1s = torch.zeros(E, F, d, dtype=torch.float32, **e)
        self.dw2s = torch.zeros(E, d, F, dtype=torch.float32, **e)
        sv, ws = mlpblk_moe_saved_size(self.desc), mlpblk_moe_workspace_size(self.desc)
        if sv == 0 or ws == 0:
            raise MlpBlkError(MLPBLK_EINVAL, "mlpblk_moe_saved_size")
        self.saved = torch.empty(sv, dtype=torch.uint8, **e)
        self.ws = torch.empty(ws, dtype=torch.uint8, **e)

    def forward(self, stream=None):
        mlpblk_moe_forward(self.desc, self.x, self.gamma, self.w1s, self.w2s, self.idx, self.p, self.y, self.saved,
                           self.ws, stream=stream)

    def backward(self, stream=None, overwrite=False):
        mlpblk_moe_backward(self.desc, self.dy, self.x, self.gamma, self.w1s, self.w2s, self.p, self.saved,
                            self.dx, self.dp, self.dgamma, self.dw1s, self.dw2s, self.ws, stream=stream,
                            overwrite=overwrite)

    def zero_grads(self, stream=None):
        # the experts' gradients as one block's of ffn E*F (same element counts)
        d = self.desc
        flat = make_desc(0, d.base.d_model, d.base.ffn * d.experts)
        mlpblk_zero_grads(flat, self.dgamma, self.dw1s, self.dw2s, stream=stream)


def _operand(t, where, name, dtype, numel, dev):
    """Device address of tensor argument `name` of `where`, checked: a contiguous CUDA
    tensor of `dtype` with at least `numel` elements, on the current device `dev` (a
    call goes to the current device's stream, so a tensor of another one is
    refused).  Integers (raw addresses) and None pass unchecked: the library checks
    what it can of those."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() == dev and t.dtype is dtype and t.numel() >= numel and t.is_contiguous():
        return t.data_ptr()
    raise MlpBlkError(MLPBLK_EINVAL, f"{where}: {name} must be a contiguous {dtype} tensor of at least {numel} "
                      f"elements on cuda:{dev}, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _dtype_code(dtype):
    """MLPBLK_BF16 / MLPBLK_FP32 of "bf16", "f32", a torch dtype or the code itself."""
    code = dtype if isinstance(dtype, int) else _Torch.get().code.get(dtype)
    if code is None:
        raise MlpBlkError(MLPBLK_ENOTSUP, f"element type {dtype}")
    return code


def make_sort_desc(tokens, width, experts, top_k, pad=128, dtype=MLPBLK_BF16) -> SortDesc:
    return SortDesc(int(tokens), int(width), int(experts), int(top_k), int(pad), _dtype_code(dtype))


def mlpblk_moe_sort_rows(desc: SortDesc) -> int:
    return int(lib.mlpblk_moe_sort_rows(ctypes.byref(desc)))


def mlpblk_moe_sort(desc, expert_idx, count, seg, pos, row_map, stream=None):
    where = "mlpblk_moe_sort"
    t = _Torch.get()
    dev, i32 = t.device(), t.int32
    n = desc.tokens * desc.top_k
    rc = lib.mlpblk_moe_sort(
        ctypes.byref(desc), _operand(expert_idx, where, "expert_idx", i32, n, dev),
        _operand(count, where, "count", i32, desc.experts, dev), _operand(seg, where, "seg", i32, desc.experts + 1, dev),
        _operand(pos, where, "pos", i32, n, dev),
        _operand(row_map, where, "row_map", i32, mlpblk_moe_sort_rows(desc), dev), _stream(stream))
    _check(rc, where)


def mlpblk_moe_permute(desc, x, pos, count, seg, rows, stream=None):
    where = "mlpblk_moe_permute"
    t = _Torch.get()
    dev, i32 = t.device(), t.int32
    dt = t.row.get(desc.dtype)
    rc = lib.mlpblk_moe_permute(
        ctypes.byref(desc), _operand(x, where, "x", dt, desc.tokens * desc.width, dev),
        _operand(pos, where, "pos", i32, desc.tokens * desc.top_k, dev),
        _operand(count, where, "count", i32, desc.experts, dev), _operand(seg, where, "seg", i32, desc.experts + 1, dev),
        _operand(rows, where, "rows", dt, mlpblk_moe_sort_rows(desc) * desc.width, dev), _stream(stream))
    _check(rc, where)


def mlpblk_moe_permute_backward(desc, d_rows, pos, dx, stream=None):
    where = "mlpblk_moe_permute_backward"
    t = _Torch.get()
    dev, i32 = t.device(), t.int32
    dt = t.row.get(desc.dtype)
    rc = lib.mlpblk_moe_permute_backward(
        ctypes.byref(desc), _operand(d_rows, where, "d_rows", dt, mlpblk_moe_sort_rows(desc) * desc.width, dev),
        _operand(pos, where, "pos", i32, desc.tokens * desc.top_k, dev),
        _operand(dx, where, "dx", dt, desc.tokens * desc.width, dev), _stream(stream))
    _check(rc, where)


def mlpblk_moe_unpermute(desc, rows, pos, weights, residual, y, stream=None):
    where = "mlpblk_moe_unpermute"
    t = _Torch.get()
    dev, i32, f32 = t.device(), t.int32, t.float32
    dt = t.row.get(desc.dtype)
    n = desc.tokens * desc.width
    rc = lib.mlpblk_moe_unpermute(
        ctypes.byref(desc), _operand(rows, where, "rows", dt, mlpblk_moe_sort_rows(desc) * desc.width, dev),
        _operand(pos, where, "pos", i32, desc.tokens * desc.top_k, dev),
        _operand(weights, where, "weights", f32, desc.tokens * desc.top_k, dev),
        _operand(residual, where, "residual", dt, n, dev), _operand(y, where, "y", dt, n, dev), _stream(stream))
    _check(rc, where)


def mlpblk_moe_unpermute_backward(desc, dy, rows, pos, count, seg, weights, d_rows, d_weights, stream=None):
    where = "mlpblk_moe_unpermute_backward"
    t = _Torch.get()
    dev, i32, f32 = t.device(), t.int32, t.float32
    dt = t.row.get(desc.dtype)
    n, r = desc.tokens * desc.top_k, mlpblk_moe_sort_rows(desc) * desc.width
    rc = lib.mlpblk_moe_unpermute_backward(
        ctypes.byref(desc), _operand(dy, where, "dy", dt, desc.tokens * desc.width, dev),
        _operand(rows, where, "rows", dt, r, dev), _operand(pos, where, "pos", i32, n, dev),
        _operand(count, where, "count", i32, desc.experts, dev), _operand(seg, where, "seg", i32, desc.experts + 1, dev),
        _operand(weights, where, "weights", f32, n, dev), _operand(d_rows, where, "d_rows", dt, r, dev),
        _operand(d_weights, where, "d_weights", f32, n, dev), _stream(stream))
    _check(rc, where)


class _Kept:
    """Base of the classes that keep device buffers of their own: the buffers cannot
    be replaced, so their addresses are taken once and a call checks only what it is
    given.  A call of these classes costs 2.4 to 3.9 us of host time on a Grace core, 1.5 of
    them the runtime's launch: the checks of the common case stand in the
    methods themselves, _operand only words the refusal."""

    def _where(self, dev, where):
        """Refuses a call whose device is not the buffers' own."""
        if dev != self._dev:
            raise MlpBlkError(MLPBLK_EINVAL, f"{where}: the buffers are on cuda:{self._dev}, the call on cuda:{dev}")


class MoeSort(_Kept):
    """The plan of one batch's routing and its buffers: `sort` fills count, seg, pos
    and row_map from the expert ids, the other methods move rows by it (the
    mlpblk_moe_* calls of the same names).  `rows` is R, the row count of the sorted
    buffers.  Before the first `sort` the plan is that of ids that select nothing."""

    def __init__(self, tokens, width, experts, top_k, pad=128, dtype="bf16", device="cuda"):
        import torch
        self.desc = make_sort_desc(tokens, width, experts, top_k, pad, dtype)
        self.rows = mlpblk_moe_sort_rows(self.desc)
        if self.rows < 0:
            raise MlpBlkError(MLPBLK_EINVAL, "mlpblk_moe_sort_rows")
        e = dict(dtype=torch.int32, device=device)
        self._count = torch.zeros(experts, **e)
        self._seg = torch.zeros(experts + 1, **e)
        self._pos = torch.full((tokens, top_k), -1, **e)   # a plan of no entry until `sort` makes one
        self._row_map = torch.full((self.rows,), -1, **e)
        self._dev = self._count.get_device()
        self._d = ctypes.addressof(self.desc)
        self._at = tuple(t.data_ptr() for t in (self._count, self._seg, self._pos, self._row_map))
        self._entries, self._x_n, self._r_n = tokens * top_k, tokens * width, self.rows * width
        self._t = _Torch.get()
        self._type = self._t.row[self.desc.dtype]

    count = property(lambda self: self._count)
    seg = property(lambda self: self._seg)
    pos = property(lambda self: self._pos)
    row_map = property(lambda self: self._row_map)

    def _at_of(self, x, where, name, dtype, numel, dev):
        """The address of a tensor, or a refusal; None is None."""
        if x is None:
            return None
        if x.dtype is dtype and x.numel() >= numel and x.get_device() == dev and x.is_contiguous():
            return x.data_ptr()
        return _operand(x, where, name, dtype, numel, dev)

    def sort(self, expert_idx, stream=None):
        where = "MoeSort.sort"
        t = self._t
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        if (expert_idx.dtype is not t.int32 or expert_idx.numel() < self._entries or expert_idx.get_device() != dev
                or not expert_idx.is_contiguous()):
            _operand(expert_idx, where, "expert_idx", t.int32, self._entries, dev)
        count, seg, pos, row_map = self._at
        rc = _calls.moe_sort(self._d, expert_idx.data_ptr(), count, seg, pos, row_map,
                             t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def permute(self, x, rows, stream=None):
        where = "MoeSort.permute"
        t, dt = self._t, self._type
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        if x.dtype is not dt or x.numel() < self._x_n or x.get_device() != dev or not x.is_contiguous():
            _operand(x, where, "x", dt, self._x_n, dev)
        if rows.dtype is not dt or rows.numel() < self._r_n or rows.get_device() != dev or not rows.is_contiguous():
            _operand(rows, where, "rows", dt, self._r_n, dev)
        count, seg, pos, _ = self._at
        rc = _calls.moe_permute(self._d, x.data_ptr(), pos, count, seg, rows.data_ptr(),
                                t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def permute_backward(self, d_rows, dx, stream=None):
        where = "MoeSort.permute_backward"
        t, dt = self._t, self._type
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        if d_rows.dtype is not dt or d_rows.numel() < self._r_n or d_rows.get_device() != dev or not d_rows.is_contiguous():
            _operand(d_rows, where, "d_rows", dt, self._r_n, dev)
        if dx.dtype is not dt or dx.numel() < self._x_n or dx.get_device() != dev or not dx.is_contiguous():
            _operand(dx, where, "dx", dt, self._x_n, dev)
        rc = _calls.moe_permute_backward(self._d, d_rows.data_ptr(), self._at[2], dx.data_ptr(),
                                         t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def unpermute(self, rows, y, weights=None, residual=None, stream=None):
        where = "MoeSort.unpermute"
        t, dt, at = self._t, self._type, self._at_of
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        rc = _calls.moe_unpermute(self._d, at(rows, where, "rows", dt, self._r_n, dev), self._at[2],
                                  at(weights, where, "weights", t.float32, self._entries, dev),
                                  at(residual, where, "residual", dt, self._x_n, dev), at(y, where, "y", dt, self._x_n, dev),
                                  t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def unpermute_backward(self, dy, rows, weights, d_rows, d_weights, stream=None):
        where = "MoeSort.unpermute_backward"
        t, dt, at = self._t, self._type, self._at_of
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        count, seg, pos, _ = self._at
        rc = _calls.moe_unpermute_backward(
            self._d, at(dy, where, "dy", dt, self._x_n, dev), at(rows, where, "rows", dt, self._r_n, dev), pos, count, seg,
            at(weights, where, "weights", t.float32, self._entries, dev), at(d_rows, where, "d_rows", dt, self._r_n, dev),
            at(d_weights, where, "d_weights", t.float32, self._entries, dev),
            t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)


def make_fp4_desc(rows, cols, batch=1, dtype=MLPBLK_BF16, transposed=False, act=MLPBLK_FP4_ACT_NONE,
                  source_rows=0) -> Fp4Desc:
    return Fp4Desc(int(rows), int(cols), int(batch), _dtype_code(dtype), int(bool(transposed)), int(act), int(source_rows))


def mlpblk_fp4_codes_size(desc: Fp4Desc) -> int:
    return int(lib.mlpblk_fp4_codes_size(ctypes.byref(desc)))


def mlpblk_fp4_scales_size(desc: Fp4Desc) -> int:
    return int(lib.mlpblk_fp4_scales_size(ctypes.byref(desc)))


def mlpblk_fp4_quantize(desc, x, codes, scales, row_map=None, map_div=0, stream=None):
    """x holds the whole source; where a row_map gathers its rows (map_div > 0), that is
    desc.source_rows of them, or, where the descriptor leaves that 0, the rows that the
    tensor x has."""
    where = "mlpblk_fp4_quantize"
    t = _Torch.get()
    dev, i32, u8 = t.device(), t.int32, t.uint8
    mapped, width = (desc.cols, desc.rows) if desc.transposed else (desc.rows, desc.cols)  # the source's
    n = desc.rows * desc.cols * desc.batch
    if row_map is not None and map_div > 0:
        if desc.source_rows == 0 and not isinstance(x, int) and x is not None and width > 0:
            desc = Fp4Desc(desc.rows, desc.cols, desc.batch, desc.dtype, desc.transposed, desc.act,
                           min(x.numel() // width, 2 ** 31 - 1))
        n = desc.source_rows * width
    rc = lib.mlpblk_fp4_quantize(
        ctypes.byref(desc), _operand(x, where, "x", t.row.get(desc.dtype), n, dev),
        _operand(row_map, where, "row_map", i32, mapped, dev), int(map_div),
        _operand(codes, where, "codes", u8, mlpblk_fp4_codes_size(desc), dev),
        _operand(scales, where, "scales", u8, mlpblk_fp4_scales_size(desc), dev), _stream(stream))
    _check(rc, where)


def mlpblk_fp4_dequantize(desc, codes, scales, y, stream=None):
    where = "mlpblk_fp4_dequantize"
    t = _Torch.get()
    dev, u8 = t.device(), t.uint8
    rc = lib.mlpblk_fp4_dequantize(
        ctypes.byref(desc), _operand(codes, where, "codes", u8, mlpblk_fp4_codes_size(desc), dev),
        _operand(scales, where, "scales", u8, mlpblk_fp4_scales_size(desc), dev),
        _operand(y, where, "y", t.row.get(desc.dtype), desc.rows * desc.cols * desc.batch, dev), _stream(stream))
    _check(rc, where)


def make_fp4_matmul_desc(m, n, k, out_dtype=MLPBLK_BF16, accumulate=False, experts=0, pad=0,
                         max_rows=0) -> Fp4MatmulDesc:
    return Fp4MatmulDesc(int(m), int(n), int(k), _dtype_code(out_dtype), int(bool(accumulate)), int(experts), int(pad),
                         int(max_rows))


def _fp4_operands(where, a, a_rows, b, b_rows, b_batch, k, dev, u8):
    """Addresses of (codes, scales) of A and B, sizes checked."""
    out = []
    for name, (codes, scales), rows, batch in (("a", a, a_rows, 1), ("b", b, b_rows, b_batch)):
        d = Fp4Desc(rows, k, batch, MLPBLK_BF16, 0, 0)
        out.append(_operand(codes, where, name + "_codes", u8, mlpblk_fp4_codes_size(d), dev))
        out.append(_operand(scales, where, name + "_scales", u8, mlpblk_fp4_scales_size(d), dev))
    return out


def mlpblk_fp4_matmul(desc, a_codes, a_scales, b_codes, b_scales, c, stream=None):
    where = "mlpblk_fp4_matmul"
    t = _Torch.get()
    dev, u8 = t.device(), t.uint8
    ops = _fp4_operands(where, (a_codes, a_scales), desc.m, (b_codes, b_scales), desc.n, 1, desc.k, dev, u8)
    rc = lib.mlpblk_fp4_matmul(ctypes.byref(desc), *ops,
                               _operand(c, where, "c", t.row.get(desc.out_dtype), desc.m * desc.n, dev), _stream(stream))
    _check(rc, where)


def mlpblk_fp4_matmul_grouped(desc, a_codes, a_scales, b_codes, b_scales, count, seg, c, stream=None):
    where = "mlpblk_fp4_matmul_grouped"
    t = _Torch.get()
    dev, i32, u8 = t.device(), t.int32, t.uint8
    ops = _fp4_operands(where, (a_codes, a_scales), desc.m, (b_codes, b_scales), desc.n, max(desc.experts, 1), desc.k,
                        dev, u8)
    rc = lib.mlpblk_fp4_matmul_grouped(
        ctypes.byref(desc), *ops, _operand(count, where, "count", i32, desc.experts, dev),
        _operand(seg, where, "seg", i32, desc.experts + 1, dev),
        _operand(c, where, "c", t.row.get(desc.out_dtype), desc.m * desc.n, dev), _stream(stream))
    _check(rc, where)


def mlpblk_fp4_wgrad_grouped(desc, a_codes, a_scales, b_codes, b_scales, seg, c, stream=None):
    where = "mlpblk_fp4_wgrad_grouped"
    t = _Torch.get()
    dev, i32, u8 = t.device(), t.int32, t.uint8
    ops = _fp4_operands(where, (a_codes, a_scales), desc.m, (b_codes, b_scales), desc.n, 1, desc.k, dev, u8)
    rc = lib.mlpblk_fp4_wgrad_grouped(
        ctypes.byref(desc), *ops, _operand(seg, where, "seg", i32, desc.experts + 1, dev),
        _operand(c, where, "c", t.row.get(desc.out_dtype), desc.experts * desc.m * desc.n, dev), _stream(stream))
    _check(rc, where)


def mlpblk_fp4_product_kernel(desc, form: int, sms: int) -> int:
    return int(lib.mlpblk_fp4_product_kernel(ctypes.byref(desc), int(form), int(sms)))


class Fp4Matrix(_Kept):
    """An MXFP4 matrix [rows, cols] (or a batch of them): its codes and scales, and
    the products that take it as A.  `codes` and `scales` given: buffers that hold a
    quantised matrix already (uint8)."""
    _ACTS = {"none": MLPBLK_FP4_ACT_NONE, "relu2": MLPBLK_FP4_ACT_RELU2}

    def __init__(self, rows, cols, batch=1, codes=None, scales=None, device="cuda"):
        import torch
        self.rows, self.cols, self.batch = int(rows), int(cols), int(batch)
        d = make_fp4_desc(rows, cols, batch)
        nc, ns = mlpblk_fp4_codes_size(d), mlpblk_fp4_scales_size(d)
        if (nc == 0 or ns == 0) and rows != 0 and cols != 0:
            raise MlpBlkError(MLPBLK_EINVAL, "mlpblk_fp4_codes_size")
        u8 = dict(dtype=torch.uint8, device=device)
        self._codes = torch.empty(nc, **u8) if codes is None else codes
        self._scales = torch.empty(ns, **u8) if scales is None else scales
        for t, n in ((self._codes, nc), (self._scales, ns)):
            if t.dtype is not torch.uint8 or t.numel() != n or not t.is_contiguous() or t.device != self._codes.device:
                raise MlpBlkError(MLPBLK_EINVAL, f"Fp4Matrix: {nc} bytes of codes and {ns} of scales, contiguous uint8 "
                                  "tensors of one device")
        self._dev = self._codes.get_device()
        self._at = (self._codes.data_ptr(), self._scales.data_ptr())
        self._n = self.rows * self.cols * self.batch
        self._t = _Torch.get()
        self._descs, self._kept = {}, []   # addresses of descriptors, and the descriptors

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)

    def _desc(self, dtype, transposed, act, source_rows=0):
        """Address of the descriptor for these options, made once."""
        key = (dtype, transposed, act, source_rows)
        at = self._descs.get(key)
        if at is None:
            if act not in self._ACTS:
                raise MlpBlkError(MLPBLK_ENOTSUP, f"Fp4Matrix.quantize: act {act!r}")
            d = make_fp4_desc(self.rows, self.cols, self.batch, dtype, transposed, self._ACTS[act], source_rows)
            self._kept.append(d)
            # another thread may make the same one: the first stays, each lives in _kept
            at = self._descs.setdefault(key, ctypes.addressof(d))
        return at

    def quantize(self, x, transposed=False, act="none", sort=None, gather=False, stream=None):
        """From x (bf16 or float32; stored [cols, rows] when transposed).  sort: a
        MoeSort whose row_map says which source rows are live; gather=True reads
        them from x's tokens, otherwise x is already in sorted order."""
        where = "Fp4Matrix.quantize"
        t = self._t
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        n, row_map, div, source_rows = self._n, None, 0, 0
        if sort is not None:
            width, mapped = (self.rows, self.cols) if transposed else (self.cols, self.rows)
            if mapped != sort.rows or (gather and width != sort.desc.width):
                raise MlpBlkError(MLPBLK_EINVAL, f"{where}: [{self.rows}, {self.cols}] is not made of the sort's "
                                  f"{sort.rows} rows of {sort.desc.width}")
            sort._where(dev, where)
            row_map = sort._at[3]
            if gather:
                n, div, source_rows = sort._x_n, sort.desc.top_k, sort.desc.tokens
        elif gather:
            raise MlpBlkError(MLPBLK_EINVAL, f"{where}: gather needs a sort")
        if x.numel() < n or x.get_device() != dev or not x.is_contiguous():
            _operand(x, where, "x", x.dtype, n, dev)
        key = (x.dtype, transposed, act, source_rows)
        d = self._descs.get(key) or self._desc(*key)
        codes, scales = self._at
        rc = _calls.fp4_quantize(d, x.data_ptr(), row_map, div, codes, scales,
                                     t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def dequantize(self, y, stream=None):
        where = "Fp4Matrix.dequantize"
        t = self._t
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        d = self._descs.get((y.dtype, False, "none", 0)) or self._desc(y.dtype, False, "none")
        if y.numel() < self._n or y.get_device() != dev or not y.is_contiguous():
            _operand(y, where, "y", y.dtype, self._n, dev)
        codes, scales = self._at
        rc = _calls.fp4_dequantize(d, codes, scales, y.data_ptr(), t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def _product(self, where, b, c, accumulate, key, make):
        """Address of the product's descriptor (made once for each key), C's address and
        the current stream."""
        t = self._t
        dev = t.device()
        if dev != self._dev or dev != b._dev:
            self._where(dev, where)
            b._where(dev, where)
        if self.batch != 1 or b.cols != self.cols:
            raise MlpBlkError(MLPBLK_EINVAL, f"{where}: A [{self.rows}, {self.cols}] x {self.batch}, B [{b.rows}, {b.cols}]")
        key = (where, c.dtype, accumulate, b.rows, key)
        e = self._descs.get(key)
        if e is None:
            d, n = make(_dtype_code(c.dtype))
            self._kept.append(d)
            e = self._descs[key] = (ctypes.addressof(d), n)
        if c.numel() < e[1] or c.get_device() != dev or not c.is_contiguous():
            _operand(c, where, "c", c.dtype, e[1], dev)
        return e[0], c.data_ptr(), t.raw_stream(dev)

    def matmul(self, b, c, accumulate=False, stream=None):
        """c[rows, b.rows] = self . b^T (or += with accumulate, float32)."""
        where = "Fp4Matrix.matmul"
        if b.batch != 1:
            raise MlpBlkError(MLPBLK_EINVAL, f"{where}: b is a batch")
        d, at, st = self._product(where, b, c, accumulate, None, lambda dt: (
            make_fp4_matmul_desc(self.rows, b.rows, self.cols, dt, accumulate), self.rows * b.rows))
        rc = _calls.fp4_matmul(d, *self._at, *b._at, at, st if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def matmul_grouped(self, b, sort, c, accumulate=False, stream=None):
        """c[R, b.rows]: expert e's rows of self times the batch's matrix e."""
        where = "Fp4Matrix.matmul_grouped"
        if b.batch != sort.desc.experts or self.rows != sort.rows:
            raise MlpBlkError(MLPBLK_EINVAL, f"{where}: b is not the experts' batch or self not the sorted rows")
        d, at, st = self._product(where, b, c, accumulate, (b.batch, sort.desc.pad, sort._entries), lambda dt: (
            make_fp4_matmul_desc(self.rows, b.rows, self.cols, dt, accumulate, b.batch, sort.desc.pad, sort._entries),
            self.rows * b.rows))
        sort._where(self._dev, where)
        rc = _calls.fp4_matmul_grouped(d, *self._at, *b._at, sort._at[0], sort._at[1], at,
                                           st if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def wgrad_grouped(self, b, sort, c, accumulate=False, stream=None):
        """c[experts, rows, b.rows]: self . b^T over each expert's segment."""
        where = "Fp4Matrix.wgrad_grouped"
        if b.batch != 1 or self.cols != sort.rows:
            raise MlpBlkError(MLPBLK_EINVAL, f"{where}: the columns are not the sorted rows")
        E = sort.desc.experts
        d, at, st = self._product(where, b, c, accumulate, (E, sort.desc.pad), lambda dt: (
            make_fp4_matmul_desc(self.rows, b.rows, self.cols, dt, accumulate, E, sort.desc.pad),
            E * self.rows * b.rows))
        sort._where(self._dev, where)
        rc = _calls.fp4_wgrad_grouped(d, *self._at, *b._at, sort._at[1], at, st if stream is None else _stream(stream))
        if rc:
            _check(rc, where)


_SCORES = {"softmax": MLPBLK_ROUTE_SOFTMAX, "sigmoid": MLPBLK_ROUTE_SIGMOID}


def make_route_desc(tokens, experts, top_k, score="softmax", groups=1, top_groups=None, renorm=True, scale=1.0,
                    dtype=MLPBLK_BF16) -> RouteDesc:
    code = score if isinstance(score, int) else _SCORES.get(score)
    if code is None:
        raise MlpBlkError(MLPBLK_ENOTSUP, f"score {score!r}")
    return RouteDesc(int(tokens), int(experts), int(top_k), code, int(groups), int(groups if top_groups is None else top_groups),
                     int(bool(renorm)), float(scale), _dtype_code(dtype))


def mlpblk_moe_route(desc, logits, bias, expert_idx, routing_weights, stream=None):
    where = "mlpblk_moe_route"
    t = _Torch.get()
    dev, n = t.device(), desc.tokens * desc.top_k
    rc = lib.mlpblk_moe_route(
        ctypes.byref(desc), _operand(logits, where, "logits", t.row.get(desc.dtype), desc.tokens * desc.experts, dev),
        _operand(bias, where, "bias", t.float32, desc.experts, dev),
        _operand(expert_idx, where, "expert_idx", t.int32, n, dev),
        _operand(routing_weights, where, "routing_weights", t.float32, n, dev), _stream(stream))
    _check(rc, where)


def mlpblk_moe_route_backward(desc, logits, expert_idx, d_routing_weights, d_logits, stream=None):
    where = "mlpblk_moe_route_backward"
    t = _Torch.get()
    dev, n = t.device(), desc.tokens * desc.top_k
    dt, e = t.row.get(desc.dtype), desc.tokens * desc.experts
    rc = lib.mlpblk_moe_route_backward(
        ctypes.byref(desc), _operand(logits, where, "logits", dt, e, dev),
        _operand(expert_idx, where, "expert_idx", t.int32, n, dev),
        _operand(d_routing_weights, where, "d_routing_weights", t.float32, n, dev),
        _operand(d_logits, where, "d_logits", dt, e, dev), _stream(stream))
    _check(rc, where)


class MoeRouter:
    """The router of one batch: `route` turns logits into expert ids and weights (those that
    MoeSort.sort and MoeSort.unpermute take), `route_backward` the weights' gradient into
    the logits'.  It keeps no buffers: every tensor is the caller's."""

    def __init__(self, tokens, experts, top_k, score="softmax", groups=1, top_groups=None, renorm=True, scale=1.0,
                 dtype="bf16"):
        self.desc = make_route_desc(tokens, experts, top_k, score, groups, top_groups, renorm, scale, dtype)
        rc = lib.mlpblk_moe_route(ctypes.byref(make_route_desc(0, experts, top_k, score, groups, top_groups, renorm, scale, dtype)),
                                  None, None, None, None, None)   # no tokens: checks the descriptor alone
        if rc or self.desc.tokens < 0 or self.desc.tokens >= 2 ** 31:
            raise MlpBlkError(rc or MLPBLK_EINVAL, "MoeRouter")
        self._d = ctypes.addressof(self.desc)
        self._n, self._l, self._e = self.desc.tokens * self.desc.top_k, self.desc.tokens * self.desc.experts, self.desc.experts
        self._t = _Torch.get()
        self._type = self._t.row[self.desc.dtype]

    def route(self, logits, expert_idx, routing_weights, bias=None, stream=None):
        """expert_idx [tokens, top_k] int32 and routing_weights [tokens, top_k] float32 of
        logits [tokens, experts]; bias [experts] float32 or None."""
        where = "MoeRouter.route"
        t, dt, n = self._t, self._type, self._n
        dev = t.device()
        if logits.dtype is not dt or logits.numel() < self._l or logits.get_device() != dev or not logits.is_contiguous():
            _operand(logits, where, "logits", dt, self._l, dev)
        if (expert_idx.dtype is not t.int32 or expert_idx.numel() < n or expert_idx.get_device() != dev
                or not expert_idx.is_contiguous()):
            _operand(expert_idx, where, "expert_idx", t.int32, n, dev)
        if (routing_weights.dtype is not t.float32 or routing_weights.numel() < n or routing_weights.get_device() != dev
                or not routing_weights.is_contiguous()):
            _operand(routing_weights, where, "routing_weights", t.float32, n, dev)
        if bias is not None:
            if bias.dtype is not t.float32 or bias.numel() < self._e or bias.get_device() != dev or not bias.is_contiguous():
                _operand(bias, where, "bias", t.float32, self._e, dev)
            bias = bias.data_ptr()
        rc = _calls.moe_route(self._d, logits.data_ptr(), bias, expert_idx.data_ptr(), routing_weights.data_ptr(),
                              t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def route_backward(self, logits, expert_idx, d_routing_weights, d_logits, stream=None):
        """d_logits [tokens, experts] (written) of the same logits and the ids `route` gave."""
        where = "MoeRouter.route_backward"
        t, dt, n = self._t, self._type, self._n
        dev = t.device()
        for x, name, want, least in ((logits, "logits", dt, self._l), (expert_idx, "expert_idx", t.int32, n),
                                     (d_routing_weights, "d_routing_weights", t.float32, n), (d_logits, "d_logits", dt, self._l)):
            if x.dtype is not want or x.numel() < least or x.get_device() != dev or not x.is_contiguous():
                _operand(x, where, name, want, least, dev)
        rc = _calls.moe_route_backward(self._d, logits.data_ptr(), expert_idx.data_ptr(), d_routing_weights.data_ptr(),
                                       d_logits.data_ptr(), t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)


def make_norm_desc(tokens, width, eps=1e-6, dtype=MLPBLK_BF16, block=0) -> NormDesc:
    return NormDesc(int(tokens), int(width), float(eps), _dtype_code(dtype), int(block))


def _norm_scales(desc):
    """Scales of one row."""
    return (desc.width + 127) // 128 if desc.block else 1


def _codes(t, where, numel, dev):
    """Address of a tensor of codes: torch.float8_e4m3fn or uint8."""
    if t is None or isinstance(t, int):
        return t
    import torch
    return _operand(t, where, "codes", t.dtype if t.dtype in (torch.float8_e4m3fn, torch.uint8) else torch.float8_e4m3fn, numel, dev)


def mlpblk_add_rmsnorm(desc, x, residual, gamma, sum, n, codes, scales, rstd, stream=None):
    where = "mlpblk_add_rmsnorm"
    t = _Torch.get()
    dev, dt, e = t.device(), t.row.get(desc.dtype), desc.tokens * desc.width
    rc = lib.mlpblk_add_rmsnorm(
        ctypes.byref(desc), _operand(x, where, "x", dt, e, dev), _operand(residual, where, "residual", dt, e, dev),
        _operand(gamma, where, "gamma", dt, desc.width, dev), _operand(sum, where, "sum", dt, e, dev),
        _operand(n, where, "n", dt, e, dev), _codes(codes, where, e, dev),
        _operand(scales, where, "scales", t.float32, desc.tokens * _norm_scales(desc), dev),
        _operand(rstd, where, "rstd", t.float32, desc.tokens, dev), _stream(stream))
    _check(rc, where)


def mlpblk_add_rmsnorm_workspace_size(desc: NormDesc) -> int:
    return int(lib.mlpblk_add_rmsnorm_workspace_size(ctypes.byref(desc)))


def mlpblk_add_rmsnorm_backward(desc, dn, d_sum, sum, rstd, gamma, dx, dgamma, workspace, overwrite=False, stream=None):
    where = "mlpblk_add_rmsnorm_backward"
    t = _Torch.get()
    dev, dt, e = t.device(), t.row.get(desc.dtype), desc.tokens * desc.width
    rc = lib.mlpblk_add_rmsnorm_backward(
        ctypes.byref(desc), _operand(dn, where, "dn", dt, e, dev), _operand(d_sum, where, "d_sum", dt, e, dev),
        _operand(sum, where, "sum", dt, e, dev), _operand(rstd, where, "rstd", t.float32, desc.tokens, dev),
        _operand(gamma, where, "gamma", dt, desc.width, dev), _operand(dx, where, "dx", dt, e, dev),
        _operand(dgamma, where, "dgamma", t.float32, desc.width, dev), int(bool(overwrite)),
        _operand(workspace, where, "workspace", t.uint8, 0, dev), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check(rc, where)


class AddRmsNorm(_Kept):
    """The residual sum and RMSNorm of one batch, with E4M3 codes and their scales: `forward`
    and `backward`.  It keeps rstd (written by `forward`, read by `backward`) and the
    backward's scratch; a forward whose backward is to come keeps both until then."""

    def __init__(self, tokens, width, eps=1e-6, dtype="bf16", block=0, device="cuda"):
        import torch
        self.desc = make_norm_desc(tokens, width, eps, dtype, block)
        size = mlpblk_add_rmsnorm_workspace_size(self.desc)
        if size == 0:   # (a call without tensors tells why)
            raise MlpBlkError(lib.mlpblk_add_rmsnorm(ctypes.byref(self.desc), *[None] * 9) or MLPBLK_EINVAL, "AddRmsNorm")
        self._rstd = torch.zeros(tokens, dtype=torch.float32, device=device)
        self._ws = torch.empty(size, dtype=torch.uint8, device=device)
        self._dev = self._ws.get_device()
        self._d = ctypes.addressof(self.desc)
        self._at = (self._rstd.data_ptr(), self._ws.data_ptr(), size)
        self._n, self._s = tokens * width, tokens * _norm_scales(self.desc)
        self._t = _Torch.get()
        self._type = self._t.row[self.desc.dtype]
        self._code_types = (torch.float8_e4m3fn, torch.uint8)

    rstd = property(lambda self: self._rstd)

    def forward(self, x, gamma, codes=None, scales=None, n=None, residual=None, sum=None, stream=None):
        """codes [tokens, width] (torch.float8_e4m3fn, or uint8) with scales [tokens] or
        [tokens, ceil(width / 128)] float32, and / or n; with residual, sum = x + residual
        (x or residual itself, or another tensor)."""
        where = "AddRmsNorm.forward"
        t, dt, e = self._t, self._type, self._n
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        if x.dtype is not dt or x.numel() < e or x.get_device() != dev or not x.is_contiguous():
            _operand(x, where, "x", dt, e, dev)
        if gamma.dtype is not dt or gamma.numel() < self.desc.width or gamma.get_device() != dev or not gamma.is_contiguous():
            _operand(gamma, where, "gamma", dt, self.desc.width, dev)
        if codes is not None:
            if codes.dtype not in self._code_types or codes.numel() < e or codes.get_device() != dev or not codes.is_contiguous():
                _codes(codes, where, e, dev)
            codes = codes.data_ptr()
        if scales is not None:
            if scales.dtype is not t.float32 or scales.numel() < self._s or scales.get_device() != dev or not scales.is_contiguous():
                _operand(scales, where, "scales", t.float32, self._s, dev)
            scales = scales.data_ptr()
        if n is not None:
            if n.dtype is not dt or n.numel() < e or n.get_device() != dev or not n.is_contiguous():
                _operand(n, where, "n", dt, e, dev)
            n = n.data_ptr()
        if residual is not None:
            if residual.dtype is not dt or residual.numel() < e or residual.get_device() != dev or not residual.is_contiguous():
                _operand(residual, where, "residual", dt, e, dev)
            residual = residual.data_ptr()
        if sum is not None:
            if sum.dtype is not dt or sum.numel() < e or sum.get_device() != dev or not sum.is_contiguous():
                _operand(sum, where, "sum", dt, e, dev)
            sum = sum.data_ptr()
        rc = _calls.add_rmsnorm(self._d, x.data_ptr(), residual, gamma.data_ptr(), sum, n, codes, scales, self._at[0],
                                t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def backward(self, dn, sum, gamma, dx, dgamma, d_sum=None, overwrite=False, stream=None):
        """dx and dgamma (added to, or set with overwrite) from dn and d_sum; sum is the
        forward's (x where it had no residual)."""
        where = "AddRmsNorm.backward"
        t, dt, e = self._t, self._type, self._n
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        rstd, ws, size = self._at
        rc = _calls.add_rmsnorm_backward(
            self._d, _operand(dn, where, "dn", dt, e, dev), _operand(d_sum, where, "d_sum", dt, e, dev),
            _operand(sum, where, "sum", dt, e, dev), rstd, _operand(gamma, where, "gamma", dt, self.desc.width, dev),
            _operand(dx, where, "dx", dt, e, dev), _operand(dgamma, where, "dgamma", t.float32, self.desc.width, dev),
            1 if overwrite else 0, ws, size, t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)


MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # K. Jordan et al., 2024


def make_ortho_desc(rows, cols, batch=1, steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7, dtype=MLPBLK_FP32) -> OrthoDesc:
    """coefficients: (a, b, c) of every step, or one such triple for each step."""
    d = OrthoDesc(int(rows), int(cols), int(batch), _dtype_code(dtype), int(steps), float(eps))
    each = list(coefficients)
    if each and not hasattr(each[0], "__len__"):
        each = [tuple(each)] * max(d.steps, 0)
    if len(each) != d.steps or d.steps > MLPBLK_ORTHO_MAX_STEPS or any(len(e) != 3 for e in each):
        raise MlpBlkError(MLPBLK_EINVAL, f"{len(each)} triples of coefficients for {steps} steps (at most {MLPBLK_ORTHO_MAX_STEPS})")
    for i, e in enumerate(each):
        for j in range(3):
            d.coefficients[i][j] = float(e[j])
    return d


def mlpblk_orthogonalize_workspace_size(desc: OrthoDesc) -> int:
    return int(lib.mlpblk_orthogonalize_workspace_size(ctypes.byref(desc)))


def mlpblk_orthogonalize(desc, u, o, workspace, stream=None):
    where = "mlpblk_orthogonalize"
    t = _Torch.get()
    dev, n = t.device(), desc.rows * desc.cols * desc.batch
    rc = lib.mlpblk_orthogonalize(
        ctypes.byref(desc), _operand(u, where, "u", t.row.get(desc.dtype), n, dev), _operand(o, where, "o", t.bfloat16, n, dev),
        _operand(workspace, where, "workspace", t.uint8, 0, dev), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check(rc, where)


def mlpblk_muon_step(desc, hp, master, weight, grad, momentum, workspace, grad_scale=None, stream=None):
    where = "mlpblk_muon_step"
    t = _Torch.get()
    dev, n, f32 = t.device(), desc.rows * desc.cols * desc.batch, t.float32
    rc = lib.mlpblk_muon_step(
        ctypes.byref(desc), ctypes.byref(hp), _operand(master, where, "master", f32, n, dev),
        _operand(weight, where, "weight", t.row.get(desc.dtype), n, dev), _operand(grad, where, "grad", f32, n, dev),
        _operand(momentum, where, "momentum", f32, n, dev), _operand(grad_scale, where, "grad_scale", f32, 1, dev),
        _operand(workspace, where, "workspace", t.uint8, 0, dev), 0 if workspace is None else workspace.numel(), _stream(stream))
    _check(rc, where)


class Orthogonalizer(_Kept):
    """Orthogonalised updates of `batch` matrices [rows, cols], and the scratch they need:
    `orthogonalize` gives the update itself, `muon_step` takes the whole optimizer step on
    float32 masters.  One workspace serves every weight of a shape in turn."""

    def __init__(self, rows, cols, batch=1, steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7, dtype="f32", device="cuda"):
        import torch
        self.desc = make_ortho_desc(rows, cols, batch, steps, coefficients, eps, dtype)
        size = mlpblk_orthogonalize_workspace_size(self.desc)
        if size == 0:   # (a call without tensors tells why)
            raise MlpBlkError(lib.mlpblk_orthogonalize(ctypes.byref(self.desc), None, None, None, 0, None) or MLPBLK_EINVAL, "Orthogonalizer")
        self._ws = torch.empty(size, dtype=torch.uint8, device=device)
        self._dev = self._ws.get_device()
        self._d = ctypes.addressof(self.desc)
        self._at = (self._ws.data_ptr(), size)
        self._n = rows * cols * batch
        self._t = _Torch.get()

    def orthogonalize(self, u, o, stream=None):
        """o (bfloat16) from u, in the descriptor's dtype; both [batch, rows, cols]."""
        where = "Orthogonalizer.orthogonalize"
        t = self._t
        dev = t.device()
        if dev != self._dev:
            self._where(dev, where)
        ws, size = self._at
        rc = _calls.orthogonalize(self._d, _operand(u, where, "u", t.row[self.desc.dtype], self._n, dev),
                                  _operand(o, where, "o", t.bfloat16, self._n, dev), ws, size,
                                  t.raw_stream(dev) if stream is None else _stream(stream))
        if rc:
            _check(rc, where)

    def muon_step(self, master, grad, momentum, lr, beta=0.95, weight_decay=0.0, scale=1.0, nesterov=True, weight=None,
                  grad_scale=None, stream=None):
        """One update of master and momentum (float32); weight: a working copy in the
        descriptor's dtype; grad_scale: a device scalar."""
        dev = self._t.device()
        if dev != self._dev:
            self._where(dev, "Orthogonalizer.muon_step")
        mlpblk_muon_step(self.desc, Muon(lr, beta, weight_decay, scale, int(bool(nesterov))), master, weight, grad, momentum,
                         self._ws, grad_scale, stream)


def mlpblk_zero_grads(desc, dgamma, dw1, dw2, stream=None):
    _check(lib.mlpblk_zero_grads(ctypes.byref(desc), _ptr(dgamma), _ptr(dw1), _ptr(dw2),
                                 _stream(stream)), "mlpblk_zero_grads")


def mlpblk_scale_grads(desc, dgamma, dw1, dw2, s, stream=None):
    _check(lib.mlpblk_scale_grads(ctypes.byref(desc), _ptr(dgamma), _ptr(dw1), _ptr(dw2), float(s),
                                  _stream(stream)), "mlpblk_scale_grads")


def mlpblk_rmsnorm_backward_noalloc(desc, x, dn, dy, gamma, rstd, dx, dgamma, stream=None):
    """RMSNorm backward + residual gradient with no workspace argument, for
    callers that cannot allocate device scratch (see include/mlpblk.h)."""
    _check(lib.mlpblk_rmsnorm_backward_noalloc(ctypes.byref(desc), _ptr(x), _ptr(dn), _ptr(dy),
                                               _ptr(gamma), _ptr(rstd), _ptr(dx), _ptr(dgamma),
                                               _stream(stream)), "mlpblk_rmsnorm_backward_noalloc")


def mlpblk_set_rmsnorm_mode(mode: int) -> None:
    _check(lib.mlpblk_set_rmsnorm_mode(int(mode)), "mlpblk_set_rmsnorm_mode")


def mlpblk_set_test_fault(fault: int) -> None:
    _check(lib.mlpblk_set_test_fault(int(fault)), "mlpblk_set_test_fault")


def mlpblk_last_error() -> int:
    return int(lib.mlpblk_last_error())


def mlpblk_version() -> int:
    return int(lib.mlpblk_version())


class KernelTrace:
    """Records CUDA events around every kernel the library launches while active
    (mlpblk_trace_begin/end); durations() then gives (kind name, ms) per launch."""

    def __init__(self, capacity):
        import torch
        self.capacity = capacity
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * capacity)]
        for e in self.events:  # torch creates the CUDA event on its first record
            e.record()
        torch.cuda.synchronize()
        if any(not e.cuda_event for e in self.events):
            raise RuntimeError("torch did not create the CUDA events for the kernel trace")
        self._handles = (ctypes.c_void_p * (2 * capacity))(*[e.cuda_event for e in self.events])
        self._kinds = (ctypes.c_int * capacity)()
        self.count = 0

    def __enter__(self):
        _check(lib.mlpblk_trace_begin(self._handles, self._kinds, self.capacity), "mlpblk_trace_begin")
        return self

    def __exit__(self, *exc):
        self.count = int(lib.mlpblk_trace_end())
        return False

    def durations(self):
        """[(kind name, milliseconds)] of the recorded launches (call after a sync)."""
        n = min(self.count, self.capacity)
        return [(KERNEL_NAMES.get(self._kinds[i], str(self._kinds[i])),
                 self.events[2 * i].elapsed_time(self.events[2 * i + 1])) for i in range(n)]


class BlockBuffers:
    """Device buffers of one block for microbatches of up to `tokens` rows:
    parameters, saved tensors, outputs, fp32 gradient buffers and workspace.
    recompute=True uses the recompute variant (no h and a buffers; a larger
    workspace holds them during each call)."""

    def __init__(self, tokens, d_model, ffn, dtype="bf16", eps=1e-6, device="cuda", recompute=False,
                 fp8=False):
        import torch
        self.torch = torch
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.code = MLPBLK_BF16 if dtype == "bf16" else MLPBLK_FP32
        self.T, self.d, self.F, self.eps = tokens, d_model, ffn, eps
        self.desc = make_desc(tokens, d_model, ffn, eps, self.code)
        e = dict(device=device)
        T, d, F = tokens, d_model, ffn
        self.gamma = torch.empty(d, dtype=self.dt, **e)
        self.w1 = torch.empty(F, d, dtype=self.dt, **e)
        self.w2 = torch.empty(d, F, dtype=self.dt, **e)
        self.x = torch.empty(T, d, dtype=self.dt, **e)
        self.dy = torch.empty(T, d, dtype=self.dt, **e)
        self.y = torch.empty(T, d, dtype=self.dt, **e)
        self.recompute = recompute
        self.fp8 = fp8
        self.h = None if recompute else torch.empty(T, F, dtype=self.dt, **e)
        self.a = None if (recompute or fp8) else torch.empty(T, F, dtype=self.dt, **e)
        if fp8:  # E4M3 codes of a and n' and a's scale record, saved for the backward
            self.a8 = torch.empty(T, F, dtype=torch.uint8, **e)
            self.n8 = torch.empty(T, d, dtype=torch.uint8, **e)
            self.scales = torch.empty(4, dtype=torch.float32, **e)
            # the weights' E4M3 codes, for the pre-quantised calls
            self.wq = torch.empty(mlpblk_fp8_weights_size(self.desc), dtype=torch.uint8, **e)
        self.rstd = torch.empty(T, dtype=torch.float32, **e)
        self.dx = torch.empty(T, d, dtype=self.dt, **e)
        self.dgamma = torch.zeros(d, dtype=torch.float32, **e)
        self.dw1 = torch.zeros(F, d, dtype=torch.float32, **e)
        self.dw2 = torch.zeros(d, F, dtype=torch.float32, **e)
        ws = (mlpblk_workspace_size_fp8 if fp8 else
              mlpblk_workspace_size_recompute if recompute else mlpblk_workspace_size)(self.desc)
        if ws == 0:
            raise MlpBlkError(MLPBLK_EINVAL, "mlpblk_workspace_size")
        self.ws = torch.empty(ws, dtype=torch.uint8, **e)

    def forward(self, stream=None):
        if self.fp8:
            mlpblk_forward_fp8(self.desc, self.x, self.gamma, self.w1, self.w2, self.y, self.h, self.a8, self.n8,
                               self.rstd, self.scales, self.ws, stream=stream)
            return
        if self.recompute:
            mlpblk_forward_recompute(self.desc, self.x, self.gamma, self.w1, self.w2, self.y, self.rstd,
                                     self.ws, stream=stream)
            return
        mlpblk_forward(self.desc, self.x, self.gamma, self.w1, self.w2, self.y, self.h, self.a,
                       self.rstd, self.ws, stream=stream)

    def fold_weights(self, stream=None):
        """W1 * gamma into self.w1g (allocated on first use), for forward_prefolded."""
        if getattr(self, "w1g", None) is None:
            self.w1g = self.torch.empty_like(self.w1)
        mlpblk_fold_weights(self.desc, self.gamma, self.w1, self.w1g, stream=stream)

    def forward_prefolded(self, stream=None):
        mlpblk_forward_prefolded(self.desc, self.x, self.w1g, self.w2, self.y, self.h, self.a, self.rstd,
                                 self.ws, stream=stream)

    def backward(self, stream=None, overwrite=False):
        """overwrite: set the gradients instead of adding into them (the saving
        and FP8 variants; the recompute variant only adds)."""
        if overwrite and self.recompute:
            raise MlpBlkError(MLPBLK_EINVAL, "overwrite is not offered by the recompute variant")
        if self.fp8:
            mlpblk_backward_fp8(self.desc, self.dy, self.x, self.gamma, self.w1, self.w2, self.h, self.a8,
                                self.n8, self.rstd, self.scales, self.dx, self.dgamma, self.dw1, self.dw2, self.ws,
                                stream=stream, overwrite=overwrite)
            return
        if self.recompute:
            mlpblk_backward_recompute(self.desc, self.dy, self.x, self.gamma, self.w1, self.w2, self.rstd,
                                      self.dx, self.dgamma, self.dw1, self.dw2, self.ws, stream=stream)
            return
        mlpblk_backward(self.desc, self.dy, self.x, self.gamma, self.w1, self.w2, self.h, self.a,
                        self.rstd, self.dx, self.dgamma, self.dw1, self.dw2, self.ws, stream=stream,
                        overwrite=overwrite)

    def zero_grads(self, stream=None):
        mlpblk_zero_grads(self.desc, self.dgamma, self.dw1, self.dw2, stream=stream)

    def scale_grads(self, s, stream=None):
        mlpblk_scale_grads(self.desc, self.dgamma, self.dw1, self.dw2, s, stream=stream)
