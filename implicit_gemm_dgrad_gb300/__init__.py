"""GB300 (sm_103a) Conv2d backward-data engine: Python binding of libcdg.so.

Argument marshalling only: every step of dgrad runs in the library's CUDA
kernels.  Tensors may be torch CUDA tensors or raw device addresses (ints);
streams may be torch streams, raw ``cudaStream_t`` values (ints) or None (the
current torch stream when torch is loaded, else the legacy default stream).

The operation (apache/tvm PR #10110, "[CUTLASS] Conv2d dgrad"):
    dX[n,h,w,c] = sum_{k,r,s} dY[n,p,q,k] * W[k,r,s,c]
over every (p, q) with h = p*stride - pad + r*dil, w = q*stride - pad + s*dil.
NHWC dX/dY, KRSC W, fp16/bf16 inputs, fp32 accumulation.

There is no CPU fallback: if the library is missing, importing the functions
that need it raises.
"""
from __future__ import annotations

import ctypes
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcdg.so")

OK = 0
STATUS_NAMES = {0: "CDG_OK", 1: "CDG_ERR_INVALID_ARG", 2: "CDG_ERR_UNSUPPORTED", 3: "CDG_ERR_ALIGNMENT",
                4: "CDG_ERR_ALIAS", 5: "CDG_ERR_CUDA", 6: "CDG_ERR_TIMEOUT", 7: "CDG_ERR_NO_DEVICE",
                8: "CDG_ERR_SCRATCH_TOO_SMALL"}
ERR_INVALID_ARG = 1
ERR_SCRATCH_TOO_SMALL = 8
NOALLOC_MAX_WEIGHT_BYTES = 8 << 20
F16, BF16, F32 = 0, 1, 2
EPI_RELU_BWD, EPI_OUT_F32, EPI_RELU_BWD_BITS, EPI_SUM, EPI_SUM_X = 1, 2, 4, 8, 16
EPI_GELU_BWD, EPI_SILU_BWD = 32, 64
FUSED_WRITE_G = 256
ACT_FLAGS = {"relu": EPI_RELU_BWD, "gelu": EPI_GELU_BWD, "silu": EPI_SILU_BWD}
DTYPES = {"f16": F16, "bf16": BF16}
ANY_DTYPES = {"f16": F16, "bf16": BF16, "f32": F32}  # the token operators and the weight update
MAX_TOP = 32
MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)

EXPORTS = ("cdg_plan", "cdg_plan_host", "cdg_destroy", "cdg_get_output_dims", "cdg_packed_weight_bytes",
           "cdg_plan_get_info", "cdg_prepack_weights", "cdg_dgrad", "cdg_device_status", "cdg_status_string",
           "cdg_dgrad_noalloc", "cdg_dgrad_noalloc_status", "cdg_autotune", "cdg_plan_set_wait_limit",
           "cdg_plan_withhold_load_for_test", "cdg_dgrad_sums", "cdg_sums_workspace_bytes",
           "cdg_fused_plan", "cdg_fused_plan_host", "cdg_fused_destroy", "cdg_fused_packed_weight_bytes",
           "cdg_fused_prepack_weights", "cdg_dgrad_fused", "cdg_fused_get_info", "cdg_fused_device_status", "cdg_pack_relu_mask", "cdg_relu_mask_bytes",
           "cdg_wgrad_plan", "cdg_wgrad_plan_host", "cdg_wgrad_destroy", "cdg_wgrad_workspace_bytes",
           "cdg_wgrad_get_info", "cdg_wgrad", "cdg_wgrad_device_status",
           "cdg_token_logprobs", "cdg_token_logprobs_grad", "cdg_embed", "cdg_embed_grad",
           "cdg_embed_grad_workspace_bytes", "cdg_muon_plan", "cdg_muon_plan_host", "cdg_muon_destroy",
           "cdg_muon_workspace_bytes", "cdg_muon_get_info", "cdg_muon_orthogonalize", "cdg_muon_step",
           "cdg_muon_device_status", "cdg_attention_plan", "cdg_attention_plan_host", "cdg_attention_destroy",
           "cdg_attention_workspace_bytes", "cdg_attention_grad_workspace_bytes", "cdg_attention", "cdg_attention_grad",
           "cdg_attention_device_status", "cdg_qk_rope", "cdg_qk_rope_grad", "cdg_qk_rope_grad_workspace_bytes",
           "cdg_rope_frequencies")


class CdgError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class PlanInfo(ctypes.Structure):
    _fields_ = [("P", ctypes.c_int), ("Q", ctypes.c_int), ("num_phases", ctypes.c_int),
                ("phase_taps", ctypes.c_int * 16), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("tile_k", ctypes.c_int), ("a_mode", ctypes.c_int), ("box_w", ctypes.c_int),
                ("box_h", ctypes.c_int), ("box_n", ctypes.c_int), ("stages", ctypes.c_int),
                ("work_items", ctypes.c_int), ("grid", ctypes.c_int), ("smem_bytes", ctypes.c_int),
                ("tmem_cols", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("mma_warps", ctypes.c_int), ("tuned", ctypes.c_int)]

    def as_dict(self) -> dict:
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["phase_taps"] = list(self.phase_taps)[: self.num_phases]
        return d


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libcdg.so (building it first if the sources are newer)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB_PATH
    if path == LIB_PATH:
        from . import build as _build
        if not _build.up_to_date():
            _build.build()
    if not os.path.exists(path):
        raise ImportError(f"libcdg.so not found at {path}; run `python -m implicit_gemm_dgrad_gb300.build`")
    lib = ctypes.CDLL(path)
    i, vp, hp = ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p
    lib.cdg_plan.argtypes = [i] * 12 + [ctypes.POINTER(hp)]
    lib.cdg_plan.restype = i
    lib.cdg_plan_host.argtypes = [i] * 13 + [ctypes.POINTER(hp)]
    lib.cdg_plan_host.restype = i
    lib.cdg_destroy.argtypes = [hp]
    lib.cdg_destroy.restype = None
    lib.cdg_get_output_dims.argtypes = [hp, ctypes.POINTER(i), ctypes.POINTER(i)]
    lib.cdg_get_output_dims.restype = i
    lib.cdg_packed_weight_bytes.argtypes = [hp]
    lib.cdg_packed_weight_bytes.restype = ctypes.c_size_t
    lib.cdg_plan_get_info.argtypes = [hp, ctypes.POINTER(PlanInfo)]
    lib.cdg_plan_get_info.restype = i
    lib.cdg_prepack_weights.argtypes = [hp, vp, vp, vp]
    lib.cdg_prepack_weights.restype = i
    lib.cdg_dgrad.argtypes = [hp, vp, vp, vp, vp, vp]
    lib.cdg_dgrad.restype = i
    lib.cdg_device_status.argtypes = [hp, vp]
    lib.cdg_device_status.restype = i
    lib.cdg_status_string.argtypes = [i]
    lib.cdg_status_string.restype = ctypes.c_char_p
    lib.cdg_dgrad_noalloc.argtypes = [hp, vp, vp, vp, vp, vp]
    lib.cdg_dgrad_noalloc.restype = i
    lib.cdg_dgrad_noalloc_status.argtypes = [vp]
    lib.cdg_dgrad_sums.argtypes = [hp, vp, vp, vp, vp, vp, vp, vp]
    lib.cdg_dgrad_sums.restype = i
    lib.cdg_sums_workspace_bytes.argtypes = [hp]
    lib.cdg_sums_workspace_bytes.restype = ctypes.c_size_t
    lib.cdg_fused_plan.argtypes = [i] * 12 + [ctypes.POINTER(hp)]
    lib.cdg_fused_plan.restype = i
    lib.cdg_fused_plan_host.argtypes = [i] * 13 + [ctypes.POINTER(hp)]
    lib.cdg_fused_plan_host.restype = i
    lib.cdg_fused_destroy.argtypes = [hp]
    lib.cdg_fused_destroy.restype = None
    lib.cdg_fused_packed_weight_bytes.argtypes = [hp, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
    lib.cdg_fused_packed_weight_bytes.restype = i
    lib.cdg_fused_prepack_weights.argtypes = [hp, vp, vp, vp, vp, vp]
    lib.cdg_fused_prepack_weights.restype = i
    lib.cdg_dgrad_fused.argtypes = [hp, vp, vp, vp, vp, vp, vp, vp]
    lib.cdg_dgrad_fused.restype = i
    lib.cdg_fused_get_info.argtypes = [hp, ctypes.POINTER(PlanInfo)]
    lib.cdg_fused_get_info.restype = i
    lib.cdg_fused_device_status.argtypes = [hp, vp]
    lib.cdg_fused_device_status.restype = i
    lib.cdg_plan_set_wait_limit.argtypes = [hp, ctypes.c_ulonglong]
    lib.cdg_plan_set_wait_limit.restype = i
    lib.cdg_plan_withhold_load_for_test.argtypes = [hp, i]
    lib.cdg_plan_withhold_load_for_test.restype = i
    lib.cdg_dgrad_noalloc_status.restype = i
    lib.cdg_autotune.argtypes = [hp, vp, vp, vp, vp, vp, i, ctypes.POINTER(ctypes.c_float)]
    lib.cdg_autotune.restype = i
    lib.cdg_pack_relu_mask.argtypes = [vp, vp, ctypes.c_longlong, i, i, vp]
    lib.cdg_pack_relu_mask.restype = i
    lib.cdg_relu_mask_bytes.argtypes = [ctypes.c_longlong, i]
    lib.cdg_relu_mask_bytes.restype = ctypes.c_longlong
    lib.cdg_wgrad_plan.argtypes = [i] * 13 + [ctypes.POINTER(hp)]
    lib.cdg_wgrad_plan.restype = i
    lib.cdg_wgrad_plan_host.argtypes = [i] * 14 + [ctypes.POINTER(hp)]
    lib.cdg_wgrad_plan_host.restype = i
    lib.cdg_wgrad_destroy.argtypes = [hp]
    lib.cdg_wgrad_destroy.restype = None
    lib.cdg_wgrad_workspace_bytes.argtypes = [hp]
    lib.cdg_wgrad_workspace_bytes.restype = ctypes.c_size_t
    lib.cdg_wgrad_get_info.argtypes = [hp, ctypes.POINTER(WgradInfo)]
    lib.cdg_wgrad_get_info.restype = i
    lib.cdg_wgrad.argtypes = [hp, vp, vp, vp, vp, vp]
    lib.cdg_wgrad.restype = i
    lib.cdg_wgrad_device_status.argtypes = [hp, vp]
    lib.cdg_wgrad_device_status.restype = i
    ll, f, sz = ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    lib.cdg_token_logprobs.argtypes = [vp, ll, vp, i, ll, i, i, f, i, vp, vp, vp, vp, vp, vp]
    lib.cdg_token_logprobs.restype = i
    lib.cdg_token_logprobs_grad.argtypes = [vp, ll, vp, i, ll, i, i, f, vp, vp, vp, vp, vp, ll, vp]
    lib.cdg_token_logprobs_grad.restype = i
    lib.cdg_embed.argtypes = [vp, ll, vp, i, ll, i, i, i, f, vp, ll, vp]
    lib.cdg_embed.restype = i
    lib.cdg_embed_grad.argtypes = [vp, ll, vp, i, ll, i, i, i, f, vp, ll, i, i, vp, vp]
    lib.cdg_embed_grad.restype = i
    lib.cdg_embed_grad_workspace_bytes.argtypes = [ll, i, i]
    lib.cdg_embed_grad_workspace_bytes.restype = sz
    lib.cdg_muon_plan.argtypes = [i] * 5 + [f] * 4 + [ctypes.POINTER(hp)]
    lib.cdg_muon_plan.restype = i
    lib.cdg_muon_plan_host.argtypes = [i] * 5 + [f] * 4 + [i, ctypes.POINTER(hp)]
    lib.cdg_muon_plan_host.restype = i
    lib.cdg_muon_destroy.argtypes = [hp]
    lib.cdg_muon_destroy.restype = None
    lib.cdg_muon_workspace_bytes.argtypes = [hp]
    lib.cdg_muon_workspace_bytes.restype = sz
    lib.cdg_muon_get_info.argtypes = [hp, ctypes.POINTER(MuonInfo)]
    lib.cdg_muon_get_info.restype = i
    lib.cdg_muon_orthogonalize.argtypes = [hp, vp, vp, vp, vp]
    lib.cdg_muon_orthogonalize.restype = i
    lib.cdg_muon_step.argtypes = [hp, vp, vp, vp, vp, vp, f, f, f, f, i, vp, vp]
    lib.cdg_muon_step.restype = i
    lib.cdg_muon_device_status.argtypes = [hp, vp]
    lib.cdg_muon_device_status.restype = i
    lib.cdg_attention_plan.argtypes = [i] * 6 + [f, ctypes.POINTER(hp)]
    lib.cdg_attention_plan.restype = i
    lib.cdg_attention_plan_host.argtypes = [i] * 6 + [f, ctypes.POINTER(hp)]
    lib.cdg_attention_plan_host.restype = i
    lib.cdg_attention_destroy.argtypes = [hp]
    lib.cdg_attention_destroy.restype = None
    lib.cdg_attention_workspace_bytes.argtypes = [hp, ll, ll, i]
    lib.cdg_attention_workspace_bytes.restype = sz
    lib.cdg_attention_grad_workspace_bytes.argtypes = [hp, ll, ll, i]
    lib.cdg_attention_grad_workspace_bytes.restype = sz
    lib.cdg_attention.argtypes = [hp] + [vp, ll] * 3 + [ll, ll, vp, vp, i, i, vp, ll, vp, vp, vp]
    lib.cdg_attention.restype = i
    lib.cdg_attention_grad.argtypes = [hp] + [vp, ll] * 4 + [vp, vp, ll, ll, ll, vp, vp, i, i] + [vp, ll] * 3 + [vp, vp]
    lib.cdg_attention_grad.restype = i
    lib.cdg_attention_device_status.argtypes = [hp, vp]
    lib.cdg_attention_device_status.restype = i
    rope = [vp, ll, vp, ll, vp, i, ll, i, i, i, i, vp, i, i, f, i, f, vp, vp]
    lib.cdg_qk_rope.argtypes = rope + [vp, ll, vp, ll, vp]
    lib.cdg_qk_rope.restype = i
    lib.cdg_qk_rope_grad.argtypes = rope + [vp, ll] * 4 + [vp, vp, vp, vp]
    lib.cdg_qk_rope_grad.restype = i
    lib.cdg_qk_rope_grad_workspace_bytes.argtypes = [ll, i, i, i]
    lib.cdg_qk_rope_grad_workspace_bytes.restype = sz
    d = ctypes.c_double
    lib.cdg_rope_frequencies.argtypes = [i, d, d, ll, d, d, ctypes.POINTER(f)]
    lib.cdg_rope_frequencies.restype = i
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().cdg_status_string(status).decode()
    except Exception:  # noqa: BLE001 - message formatting must not raise
        return "?"


def _addr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _current_device() -> int:
    import torch
    return torch.cuda.current_device()


def _check_buffer(t, nbytes: int, what: str) -> None:
    """A tensor argument must be a contiguous CUDA tensor of at least nbytes
    (the kernels read and write exactly the planned extents, which the C ABI
    cannot check).  Raw integer pointers are passed through unchecked."""
    if t is None or isinstance(t, int):
        return
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{what} must be a CUDA tensor (or a device pointer)")
    idx = getattr(getattr(t, "device", None), "index", None)
    if idx is not None:
        cur = _current_device()
        if idx != cur:
            # the library launches on the current device; a pointer into
            # another GPU's memory would be read by this one's kernels
            raise ValueError(f"{what} is on cuda:{idx}, but the current device is cuda:{cur}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{what} holds {have} bytes; the plan needs {nbytes}")


_raw_stream = None  # how the current torch stream's handle is found, once torch is initialised


def _current_stream() -> int | None:
    """The current torch stream, or None without an initialised torch.  torch's
    own query builds a stream object (3.7 us on the Grace host against 0.1 us
    for the handle alone), so the handle is asked for where torch offers it."""
    global _raw_stream
    if _raw_stream is None:
        try:
            import torch
        except ImportError:
            return None
        if not (torch.cuda.is_available() and torch.cuda.is_initialized()):
            return None
        raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
        _raw_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream(s) -> int | None:
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


class Plan:
    """One planned dgrad shape (a ``cdg_handle_t``)."""

    def __init__(self, N, H, W, C, K, R, S, stride=1, pad=0, dil=1, dtype="bf16", relu=False,
                 out_f32=False, host_sms: int | None = None, relu_bits=False, sums: int = 0, act: str = "relu"):
        self.lib = load_library()
        self.shape = dict(N=N, H=H, W=W, C=C, K=K, R=R, S=S, stride=stride, pad=pad, dil=dil)
        self.dtype = dtype
        self.relu = relu          # the gate reads a saved tensor of dX's shape (ReLU's x, or act's input)
        self.relu_bits = relu_bits
        self.out_f32 = out_f32
        self.sums = int(sums)
        gate = ACT_FLAGS[act] if relu else 0
        epi = gate | (EPI_OUT_F32 if out_f32 else 0) | (EPI_RELU_BWD_BITS if relu_bits else 0)
        epi |= {0: 0, 1: EPI_SUM, 2: EPI_SUM | EPI_SUM_X}[self.sums]
        h = ctypes.c_void_p()
        dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        if host_sms is None:
            rc = self.lib.cdg_plan(N, H, W, C, K, R, S, stride, pad, dil, dt, epi, ctypes.byref(h))
        else:
            rc = self.lib.cdg_plan_host(N, H, W, C, K, R, S, stride, pad, dil, dt, epi, host_sms, ctypes.byref(h))
        if rc != OK:
            raise CdgError(rc, "cdg_plan")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.lib.cdg_destroy(self.handle)
        self.handle = None

    def __del__(self):
        self.close()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def output_dims(self) -> tuple[int, int]:
        P, Q = ctypes.c_int(), ctypes.c_int()
        rc = self.lib.cdg_get_output_dims(self.handle, ctypes.byref(P), ctypes.byref(Q))
        if rc != OK:
            raise CdgError(rc, "cdg_get_output_dims")
        return P.value, Q.value

    @property
    def packed_weight_bytes(self) -> int:
        return int(self.lib.cdg_packed_weight_bytes(self.handle))

    def info(self) -> dict:
        inf = PlanInfo()
        rc = self.lib.cdg_plan_get_info(self.handle, ctypes.byref(inf))
        if rc != OK:
            raise CdgError(rc, "cdg_plan_get_info")
        return inf.as_dict()

    def _sizes(self) -> dict:
        """Bytes of each tensor of this plan's dgrad."""
        d = self.shape
        P, Q = self.output_dims
        pixels = d["N"] * d["H"] * d["W"]
        mask = 0
        if self.relu_bits:
            mask = relu_mask_bytes(pixels, d["C"])
        elif self.relu:
            mask = 2 * pixels * d["C"]
        return {"dY": 2 * d["N"] * P * Q * d["K"], "W": 2 * d["K"] * d["R"] * d["S"] * d["C"],
                "dX": (4 if self.out_f32 else 2) * pixels * d["C"], "mask": mask}

    def _check(self, dY=None, W=None, W_packed=None, dX=None, relu_mask=None) -> None:
        z = self._sizes()
        _check_buffer(dY, z["dY"], "dY")
        _check_buffer(W, z["W"], "W")
        _check_buffer(W_packed, z["W"], "W_packed")
        _check_buffer(dX, z["dX"], "dX")
        _check_buffer(relu_mask, z["mask"], "relu_mask")

    def prepack_weights(self, W_krsc, W_packed, stream=None) -> None:
        self._check(W=W_krsc, W_packed=W_packed)
        rc = self.lib.cdg_prepack_weights(self.handle, _addr(W_krsc), _addr(W_packed), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_prepack_weights")

    def dgrad(self, dY, W_packed, dX, relu_mask=None, stream=None) -> None:
        self._check(dY=dY, W_packed=W_packed, dX=dX, relu_mask=relu_mask)
        rc = self.lib.cdg_dgrad(self.handle, _addr(dY), _addr(W_packed), _addr(dX), _addr(relu_mask),
                                _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_dgrad")

    @property
    def sums_workspace_bytes(self) -> int:
        return int(self.lib.cdg_sums_workspace_bytes(self.handle))

    def dgrad_sums(self, dY, W_packed, dX, sums, workspace, relu_mask=None, stream=None) -> None:
        """dgrad plus the per-channel sums of its output (cdg_dgrad_sums):
        sums (fp32, C values, or 2*C for sums=2) receives sum(out) per channel
        and, for sums=2, sum(out * x) where the gate passes."""
        self._check(dY=dY, W_packed=W_packed, dX=dX, relu_mask=relu_mask)
        _check_buffer(sums, 4 * self.sums * self.shape["C"], "sums")
        _check_buffer(workspace, self.sums_workspace_bytes, "workspace")
        rc = self.lib.cdg_dgrad_sums(self.handle, _addr(dY), _addr(W_packed), _addr(dX), _addr(relu_mask),
                                     _addr(sums), _addr(workspace), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_dgrad_sums")

    def dgrad_noalloc(self, dY, W_krsc, dX, relu_mask=None, stream=None) -> None:
        """dgrad from the unpacked KRSC filter without any device allocation
        (the packed weights live in the library's own scratch array; see
        cdg_dgrad_noalloc in cdg.h for the size limit and the sharing rules)."""
        self._check(dY=dY, W=W_krsc, dX=dX, relu_mask=relu_mask)
        rc = self.lib.cdg_dgrad_noalloc(self.handle, _addr(dY), _addr(W_krsc), _addr(dX), _addr(relu_mask),
                                        _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_dgrad_noalloc")

    @staticmethod
    def noalloc_status(stream=None) -> int:
        """Read and clear the status word of cdg_dgrad_noalloc launches on the
        current device (cdg_dgrad_noalloc_status): 0, or the CDG_ERR_TIMEOUT
        code of a launch that gave up a bounded wait."""
        return int(load_library().cdg_dgrad_noalloc_status(_stream(stream)))

    def autotune(self, dY, W_packed, dX, relu_mask=None, stream=None, reps: int = 3) -> float:
        """Time every configuration the planner can produce for this shape on
        these tensors and keep the fastest (cdg_autotune); returns its mean
        launch time in ms.  dX receives the correct result."""
        self._check(dY=dY, W_packed=W_packed, dX=dX, relu_mask=relu_mask)
        best = ctypes.c_float()
        rc = self.lib.cdg_autotune(self.handle, _addr(dY), _addr(W_packed), _addr(dX), _addr(relu_mask),
                                   _stream(stream), int(reps), ctypes.byref(best))
        if rc != OK:
            raise CdgError(rc, "cdg_autotune")
        return float(best.value)

    def device_status(self, stream=None) -> int:
        return int(self.lib.cdg_device_status(self.handle, _stream(stream)))

    def set_wait_limit(self, ns: int) -> None:
        """Longest time any single pipeline wait of this plan's kernel may
        take before the launch aborts with CDG_ERR_TIMEOUT (cdg_plan_set_wait_limit)."""
        rc = self.lib.cdg_plan_set_wait_limit(self.handle, int(ns))
        if rc != OK:
            raise CdgError(rc, "cdg_plan_set_wait_limit")

    def withhold_load_for_test(self, stage: int) -> None:
        """Test only: make launches withhold the operand load of pipeline stage
        `stage` in every CTA, so they take the bounded-wait timeout path
        (cdg_plan_withhold_load_for_test); -1 restores normal launches."""
        rc = self.lib.cdg_plan_withhold_load_for_test(self.handle, int(stage))
        if rc != OK:
            raise CdgError(rc, "cdg_plan_withhold_load_for_test")


class FusedPlan:
    """Back-to-back dgrads in one kernel (a ``cdg_fused_t``):
    g = act_bwd(dgrad(dY2, W2), x2) for a stride-1 R2 x S2 layer with C2 = 64
    channels, then dX1 = dgrad_1x1(g, W1) with C1 channels; g stays on chip
    and is written only with write_g=True."""

    def __init__(self, N, H, W, C1, C2, K2, R2, S2, pad2=1, dil2=1, dtype="bf16", act: str | None = "relu",
                 write_g=False, host_sms: int | None = None):
        self.lib = load_library()
        self.shape = dict(N=N, H=H, W=W, C1=C1, C2=C2, K2=K2, R2=R2, S2=S2, pad2=pad2, dil2=dil2)
        self.act = act
        self.write_g = bool(write_g)
        flags = (ACT_FLAGS[act] if act else 0) | (FUSED_WRITE_G if write_g else 0)
        dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        h = ctypes.c_void_p()
        args = (N, H, W, C1, C2, K2, R2, S2, pad2, dil2, dt, flags)
        if host_sms is None:
            rc = self.lib.cdg_fused_plan(*args, ctypes.byref(h))
        else:
            rc = self.lib.cdg_fused_plan_host(*args, host_sms, ctypes.byref(h))
        if rc != OK:
            raise CdgError(rc, "cdg_fused_plan")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.lib.cdg_fused_destroy(self.handle)
        self.handle = None

    def __del__(self):
        self.close()

    @property
    def packed_weight_bytes(self) -> tuple[int, int]:
        b2, b1 = ctypes.c_size_t(), ctypes.c_size_t()
        rc = self.lib.cdg_fused_packed_weight_bytes(self.handle, ctypes.byref(b2), ctypes.byref(b1))
        if rc != OK:
            raise CdgError(rc, "cdg_fused_packed_weight_bytes")
        return int(b2.value), int(b1.value)

    def info(self) -> dict:
        inf = PlanInfo()
        rc = self.lib.cdg_fused_get_info(self.handle, ctypes.byref(inf))
        if rc != OK:
            raise CdgError(rc, "cdg_fused_get_info")
        return inf.as_dict()

    def prepack_weights(self, W2, W1, W2p, W1p, stream=None) -> None:
        b2, b1 = self.packed_weight_bytes
        for t, n, what in ((W2, b2, "W2"), (W1, b1, "W1"), (W2p, b2, "W2p"), (W1p, b1, "W1p")):
            _check_buffer(t, n, what)
        rc = self.lib.cdg_fused_prepack_weights(self.handle, _addr(W2), _addr(W1), _addr(W2p), _addr(W1p),
                                                _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_fused_prepack_weights")

    def dgrad(self, dY2, W2p, x2, W1p, dX1, g=None, stream=None) -> None:
        d = self.shape
        P = d["H"] + 2 * d["pad2"] - d["dil2"] * (d["R2"] - 1)
        Q = d["W"] + 2 * d["pad2"] - d["dil2"] * (d["S2"] - 1)
        px = d["N"] * d["H"] * d["W"]
        b2, b1 = self.packed_weight_bytes
        _check_buffer(dY2, 2 * d["N"] * P * Q * d["K2"], "dY2")
        _check_buffer(W2p, b2, "W2p")
        _check_buffer(W1p, b1, "W1p")
        _check_buffer(x2, 2 * px * d["C2"], "x2")
        _check_buffer(dX1, 2 * px * d["C1"], "dX1")
        _check_buffer(g, 2 * px * d["C2"], "g")
        rc = self.lib.cdg_dgrad_fused(self.handle, _addr(dY2), _addr(W2p), _addr(x2), _addr(W1p), _addr(g),
                                      _addr(dX1), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_dgrad_fused")

    def device_status(self, stream=None) -> int:
        return int(self.lib.cdg_fused_device_status(self.handle, _stream(stream)))


class WgradInfo(ctypes.Structure):
    _fields_ = [("P", ctypes.c_int), ("Q", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("taps_per_item", ctypes.c_int), ("splits", ctypes.c_int), ("pos_box", ctypes.c_int * 3), ("blocks", ctypes.c_int),
                ("stages", ctypes.c_int), ("work_items", ctypes.c_int), ("grid", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("tmem_cols", ctypes.c_int), ("x_major", ctypes.c_int)]

    def as_dict(self) -> dict:
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["pos_box"] = list(self.pos_box)
        return d


class WgradPlan:
    """One planned wgrad shape (a ``cdg_wgrad_t``): dW = wgrad(dY, x)."""

    def __init__(self, N, H, W, C, K, R, S, stride=1, pad=0, dil=1, dtype="bf16", out_f32=False, splits=0,
                 host_sms: int | None = None):
        self.lib = load_library()
        self.shape = dict(N=N, H=H, W=W, C=C, K=K, R=R, S=S, stride=stride, pad=pad, dil=dil)
        self.out_f32 = bool(out_f32)
        h = ctypes.c_void_p()
        dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
        args = (N, H, W, C, K, R, S, stride, pad, dil, dt, int(bool(out_f32)), int(splits))
        if host_sms is None:
            rc = self.lib.cdg_wgrad_plan(*args, ctypes.byref(h))
        else:
            rc = self.lib.cdg_wgrad_plan_host(*args, host_sms, ctypes.byref(h))
        if rc != OK:
            raise CdgError(rc, "cdg_wgrad_plan")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.lib.cdg_wgrad_destroy(self.handle)
        self.handle = None

    def __del__(self):
        self.close()

    @property
    def workspace_bytes(self) -> int:
        return int(self.lib.cdg_wgrad_workspace_bytes(self.handle))

    def info(self) -> dict:
        inf = WgradInfo()
        rc = self.lib.cdg_wgrad_get_info(self.handle, ctypes.byref(inf))
        if rc != OK:
            raise CdgError(rc, "cdg_wgrad_get_info")
        return inf.as_dict()

    def wgrad(self, dY, x, dW, workspace, stream=None) -> None:
        d = self.shape
        inf = self.info()
        _check_buffer(dY, 2 * d["N"] * inf["P"] * inf["Q"] * d["K"], "dY")
        _check_buffer(x, 2 * d["N"] * d["H"] * d["W"] * d["C"], "x")
        _check_buffer(dW, (4 if self.out_f32 else 2) * d["K"] * d["R"] * d["S"] * d["C"], "dW")
        _check_buffer(workspace, self.workspace_bytes, "workspace")
        rc = self.lib.cdg_wgrad(self.handle, _addr(dY), _addr(x), _addr(dW), _addr(workspace), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_wgrad")

    def device_status(self, stream=None) -> int:
        return int(self.lib.cdg_wgrad_device_status(self.handle, _stream(stream)))


def wgrad_plan(N, H, W, C, K, R, S, stride=1, pad=0, dil=1, dtype="bf16", out_f32=False, splits=0) -> WgradPlan:
    return WgradPlan(N, H, W, C, K, R, S, stride, pad, dil, dtype, out_f32, splits)


def wgrad_plan_host(N, H, W, C, K, R, S, stride=1, pad=0, dil=1, dtype="bf16", out_f32=False, splits=0,
                    num_sms=148) -> WgradPlan:
    return WgradPlan(N, H, W, C, K, R, S, stride, pad, dil, dtype, out_f32, splits, host_sms=num_sms)


def plan(N, H, W, C, K, R, S, stride=1, pad=0, dil=1, dtype="bf16", relu=False, out_f32=False,
         relu_bits=False, sums: int = 0, act: str = "relu") -> Plan:
    """relu=True: the epilogue applies the backward of activation `act`
    ("relu" gate, "gelu", "silu") with the saved tensor passed to dgrad."""
    return Plan(N, H, W, C, K, R, S, stride, pad, dil, dtype, relu, out_f32, relu_bits=relu_bits, sums=sums,
                act=act)


def relu_mask_bytes(pixels: int, C: int) -> int:
    """Bytes of the packed ReLU mask of `pixels` pixels of C channels (cdg_relu_mask_bytes)."""
    n = load_library().cdg_relu_mask_bytes(int(pixels), int(C))
    if n < 0:
        raise CdgError(ERR_INVALID_ARG, "cdg_relu_mask_bytes")
    return n


def pack_relu_mask(x, bits, pixels: int, C: int, dtype="bf16", stream=None) -> None:
    """bits (relu_mask_bytes(pixels, C) bytes) = the packed mask (x > 0) of the
    NHWC activation x, one bit per element in 16-byte units per pixel
    (cdg_pack_relu_mask), for plans made with relu_bits=True."""
    lib = load_library()
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    if int(pixels) >= 0 and int(C) > 0 and int(C) % 8 == 0:
        _check_buffer(x, 2 * int(pixels) * int(C), "x")
        _check_buffer(bits, relu_mask_bytes(pixels, C), "bits")
    rc = lib.cdg_pack_relu_mask(_addr(x), _addr(bits), int(pixels), int(C), dt, _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_pack_relu_mask")


def plan_host(N, H, W, C, K, R, S, stride=1, pad=0, dil=1, dtype="bf16", relu=False, out_f32=False,
              num_sms=148, relu_bits=False, sums: int = 0, act: str = "relu") -> Plan:
    return Plan(N, H, W, C, K, R, S, stride, pad, dil, dtype, relu, out_f32, host_sms=num_sms, relu_bits=relu_bits,
                sums=sums, act=act)


# ---- token operators: log probabilities, embedding, and their gradients


def _dtype(dtype) -> int:
    return ANY_DTYPES[dtype] if isinstance(dtype, str) else int(dtype)


# Element types of the tensor arguments, by torch's names (numpy's are the same), and their bytes
# (the element type is None for a dtype that the library refuses).
_TYPES = {F16: "float16", BF16: "bfloat16", F32: "float32", "f16": "float16", "bf16": "bfloat16", "f32": "float32"}
_SIZES = {"float16": 2, "bfloat16": 2, "float32": 4, "int32": 4, "int64": 8, None: 2}

_type_names: dict = {}  # by dtype object, as they are met


def _type_name(t) -> str | None:
    """The name of a tensor's element type; None for an object that does not say."""
    dt = getattr(t, "dtype", None)
    if dt is None:
        return None
    name = _type_names.get(dt)
    if name is None:
        name = _type_names[dt] = sys.intern(str(dt).rpartition(".")[2])
    return name


_tensor = _cuda_device = None  # torch.Tensor and the current device's number, once a torch tensor has been seen


def _bytes_of(t, n: int, kind: str | None, what: str) -> int:
    """Address of a dense CUDA tensor of at least n elements of type kind."""
    esize = _SIZES[kind]
    if type(t) is _tensor and _type_names.get(t.dtype) == kind and t.nbytes >= n * esize and t.is_contiguous() and \
            t.get_device() == _cuda_device():
        return t.data_ptr()  # what the checks below find, without their cost
    if t.element_size() != esize:
        raise ValueError(f"{what} has elements of {t.element_size()} bytes; {esize} are needed")
    name = _type_name(t)
    if name is not None and kind is not None and name != kind:
        raise ValueError(f"{what} has elements of type {name}; {kind} is needed")
    _check_buffer(t, n * esize, what)
    if _tensor is None and type(t).__module__ == "torch":
        import torch
        globals().update(_tensor=torch.Tensor, _cuda_device=getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))
        _torch_types.update({n: getattr(torch, n) for n in ("float16", "bfloat16", "float32")})
    return t.data_ptr()


def _dense(t, n: int, kind: str | None, what: str) -> int | None:
    """Address of a dense argument of n elements of type kind (None stays None)."""
    if t is None or isinstance(t, int):
        return t
    return _bytes_of(t, n, kind, what)


def _row_stride(t, rows: int, cols: int, what: str) -> int:
    """Row stride of a contiguous tensor as rows of cols elements: dense where
    trailing dimensions hold just a row, or where the tensor has one dimension
    or just rows * cols elements; the last dimension where that is wider than a
    row (a padded vocabulary), which then holds at least rows of them."""
    shape = getattr(t, "shape", None)
    if shape is None or len(shape) < 2 or shape[-1] == cols or t.numel() == rows * cols:
        return cols
    last = row = shape[-1]
    for s in reversed(shape[:-1]):
        if row >= cols:
            break
        row *= s
    if row == cols:
        return cols
    if last < cols or t.numel() < rows * last:
        raise ValueError(f"{what} is {tuple(shape)}; the call needs {(rows, cols)}")
    return last


def _matrix(t, rows: int, cols: int, kind: str | None, ld: int | None, what: str) -> tuple[int | None, int]:
    """Address and row stride of a rows x cols argument.  A contiguous tensor's
    rows may be wider than cols, and more than rows; another 2-D tensor of shape
    (rows, cols) may have any row stride with unit column stride (a slice of a
    wider one); a raw address has row stride ld, or cols."""
    if t is None or isinstance(t, int):
        return t, int(ld if ld is not None else cols)
    if type(t) is _tensor and _type_names.get(t.dtype) == kind and t.nbytes == rows * cols * _SIZES[kind] and ld is None and \
            t.is_contiguous() and t.get_device() == _cuda_device():
        return t.data_ptr(), cols  # as in _bytes_of
    if type(t) is _tensor and _type_names.get(t.dtype) == kind and rows > 1 and ld is None and t.get_device() == _cuda_device():
        shape = t.shape
        if len(shape) == 2 and shape[0] == rows and shape[1] == cols:
            own, step = t.stride()
            if step == 1 and own >= cols:
                return t.data_ptr(), own  # as below
    own = cols
    if t.is_contiguous() or t.dim() != 2:
        own = _row_stride(t, rows, cols, what)
        at = _bytes_of(t, (rows - 1) * own + cols if rows > 0 else 0, kind, what)
    else:
        if tuple(t.shape) != (rows, cols):
            raise ValueError(f"{what} is {tuple(t.shape)}; the call needs {(rows, cols)}")
        if cols > 1 and t.stride(1) != 1:
            raise ValueError(f"{what} must have unit column stride")
        if rows > 1 and t.stride(0) < cols:
            raise ValueError(f"{what} has overlapping rows (row stride {t.stride(0)} for {cols} columns)")
        if rows > 1:
            own = t.stride(0)
        at = _bytes_of(t[0, :], cols, kind, what) if rows else t.data_ptr()
    if ld is not None and int(ld) != own and rows > 1:
        raise ValueError(f"{what} has row stride {own}, not {ld}")
    return at, int(own)


_torch_types: dict = {}  # torch's element types by name, once a torch tensor has been seen


def _matrices(kind: str | None, *specs) -> list:
    """Addresses and row strides of several _matrix arguments of one element
    type, one after the other: the same answers, with the checks of a dense
    tensor and of a slice of wider rows in line."""
    out: list = []
    want = _torch_types.get(kind)
    here = _cuda_device() if want is not None else -1
    for t, rows, cols, ld, what in specs:
        if type(t) is _tensor and t.dtype is want and ld is None and t.get_device() == here:
            if t.nbytes == rows * cols * _SIZES[kind] and t.is_contiguous():
                out += (t.data_ptr(), cols)
                continue
            shape = t.shape
            if rows > 1 and len(shape) == 2 and shape[0] == rows and shape[1] == cols:  # a slice of wider rows
                own, step = t.stride()
                if step == 1 and own >= cols:
                    out += (t.data_ptr(), own)
                    continue
        if t is None:
            out += (None, cols if ld is None else int(ld))
        else:
            out += _matrix(t, rows, cols, kind, ld, what)
    return out


def _vectors(n: int, *specs) -> list:
    """Addresses of several dense fp32 arguments of n elements (None stays None)."""
    out: list = []
    want = _torch_types.get("float32")
    here = _cuda_device() if want is not None else -1
    for t, what in specs:
        if t is None:
            out.append(None)
        elif type(t) is _tensor and t.dtype is want and t.get_device() == here and t.nbytes >= 4 * n and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            out.append(_dense(t, n, "float32", what))
    return out


def _dense_matrix(t, rows: int, cols: int, kind: str, what: str) -> int | None:
    """Address of a rows x cols argument whose rows lie one after the other."""
    at, own = _matrix(t, rows, cols, kind, None, what)
    if own != cols and rows > 1 and cols > 0:
        raise ValueError(f"{what} must have dense rows of {cols}; it has row stride {own}")
    return at


def _tokens(t, n: int, what: str) -> tuple[int | None, int]:
    """Address and bytes per number of a token list (int32 or int64; a raw address is int64)."""
    if t is None or isinstance(t, int):
        return t, 8
    if type(t) is _tensor and _type_names.get(t.dtype) == "int64":
        return _bytes_of(t, n, "int64", what), 8
    size = t.element_size()
    if size not in (4, 8) or t.is_floating_point() or _type_name(t) not in ("int32", "int64", None):
        raise ValueError(f"{what} must hold int32 or int64 token numbers")
    return _bytes_of(t, n, "int64" if size == 8 else "int32", what), size


def token_logprobs(logits, targets, logp, lse, rows: int, vocab: int, dtype="bf16", scale: float = 1.0,
                   entropy=None, top: int = 0, top_ids=None, top_logp=None, ld: int | None = None,
                   stream=None) -> None:
    """Log probabilities of given tokens under softmax(scale * logits)
    (cdg_token_logprobs): logp[i] of targets[i] (0 where a target names no
    token), lse[i], and on request the row's entropy and its `top` largest
    entries with their log probabilities.  Outputs fp32 (top_ids int32); a
    target list or output that is not wanted is None."""
    rows, vocab, top = int(rows), int(vocab), int(top)
    lg, ld = _matrix(logits, rows, vocab, _TYPES.get(dtype), ld, "logits")
    tg, ib = _tokens(targets, rows, "targets")
    rc = load_library().cdg_token_logprobs(
        lg, ld, tg, ib, rows, vocab, _dtype(dtype), float(scale), top, _dense(logp, rows, "float32", "logp"),
        _dense(lse, rows, "float32", "lse"), _dense(entropy, rows, "float32", "entropy"),
        _dense_matrix(top_ids, rows, top, "int32", "top_ids"),
        _dense_matrix(top_logp, rows, top, "float32", "top_logp"), _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_token_logprobs")


def token_logprobs_grad(logits, targets, lse, entropy, g_logp, g_entropy, dlogits, rows: int, vocab: int,
                        dtype="bf16", scale: float = 1.0, ld: int | None = None, ld_d: int | None = None,
                        stream=None) -> None:
    """The gradient of token_logprobs (cdg_token_logprobs_grad) for the row
    gradients g_logp and g_entropy (None: no entropy term) into dlogits, which
    may be the logits themselves."""
    rows, vocab = int(rows), int(vocab)
    lg, ld = _matrix(logits, rows, vocab, _TYPES.get(dtype), ld, "logits")
    dl, ld_d = _matrix(dlogits, rows, vocab, _TYPES.get(dtype), ld_d, "dlogits")
    tg, ib = _tokens(targets, rows, "targets")
    rc = load_library().cdg_token_logprobs_grad(
        lg, ld, tg, ib, rows, vocab, _dtype(dtype), float(scale), _dense(lse, rows, "float32", "lse"),
        _dense(entropy, rows, "float32", "entropy"), _dense(g_logp, rows, "float32", "g_logp"),
        _dense(g_entropy, rows, "float32", "g_entropy"), dl, ld_d, _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_token_logprobs_grad")


def embed(table, tokens, out, count: int, vocab: int, dim: int, dtype="bf16", scale: float = 1.0,
          ld_table: int | None = None, ld_out: int | None = None, stream=None) -> None:
    """out[i] = scale * table[tokens[i]], zeros where there is no token (cdg_embed)."""
    count, vocab, dim = int(count), int(vocab), int(dim)
    tb, ld_table = _matrix(table, vocab, dim, _TYPES.get(dtype), ld_table, "table")
    ou, ld_out = _matrix(out, count, dim, _TYPES.get(dtype), ld_out, "out")
    tk, ib = _tokens(tokens, count, "tokens")
    rc = load_library().cdg_embed(tb, ld_table, tk, ib, count, vocab, dim, _dtype(dtype), float(scale), ou, ld_out,
                                  _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_embed")


def embed_grad_workspace_bytes(count: int, vocab: int, dim: int) -> int:
    """Bytes of embed_grad's workspace (cdg_embed_grad_workspace_bytes)."""
    n = int(load_library().cdg_embed_grad_workspace_bytes(int(count), int(vocab), int(dim)))
    if n == 0:
        raise CdgError(ERR_INVALID_ARG, "cdg_embed_grad_workspace_bytes")
    return n


def embed_grad(dout, tokens, dtable, workspace, count: int, vocab: int, dim: int, dtype="bf16", scale: float = 1.0,
               out_f32: bool = False, accumulate: bool = False, ld_dout: int | None = None,
               ld_dtable: int | None = None, stream=None) -> None:
    """dtable[v] = scale * the sum of dout[i] over the i with tokens[i] = v
    (cdg_embed_grad); accumulate=True adds to the rows that tokens point to."""
    count, vocab, dim = int(count), int(vocab), int(dim)
    do, ld_dout = _matrix(dout, count, dim, _TYPES.get(dtype), ld_dout, "dout")
    dt, ld_dtable = _matrix(dtable, vocab, dim, "float32" if out_f32 else _TYPES.get(dtype), ld_dtable, "dtable")
    tk, ib = _tokens(tokens, count, "tokens")
    if workspace is not None and not isinstance(workspace, int):
        _check_buffer(workspace, embed_grad_workspace_bytes(count, vocab, dim), "workspace")
    rc = load_library().cdg_embed_grad(do, ld_dout, tk, ib, count, vocab, dim, _dtype(dtype), float(scale), dt,
                                       ld_dtable, int(bool(out_f32)), int(bool(accumulate)), _addr(workspace),
                                       _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_embed_grad")


# ---- the weight update from an orthogonalised gradient


class MuonInfo(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int), ("n", ctypes.c_int), ("transposed", ctypes.c_int),
                ("gram", ctypes.c_int), ("launches", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class MuonPlan:
    """One planned shape of the orthogonalised weight update (a ``cdg_muon_t``):
    a batch of rows x cols matrices, e.g. filters stored KRSC as K x (R*S*C)."""

    def __init__(self, rows, cols, batch=1, dtype="bf16", steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7,
                 host_sms: int | None = None):
        self.lib = load_library()
        self.shape = dict(batch=int(batch), rows=int(rows), cols=int(cols))
        self.dtype = dtype
        a, b, c = coefficients
        h = ctypes.c_void_p()
        args = (batch, rows, cols, _dtype(dtype), steps, a, b, c, eps)
        if host_sms is None:
            rc = self.lib.cdg_muon_plan(*args, ctypes.byref(h))
        else:
            rc = self.lib.cdg_muon_plan_host(*args, host_sms, ctypes.byref(h))
        if rc != OK:
            raise CdgError(rc, "cdg_muon_plan")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.lib.cdg_muon_destroy(self.handle)
        self.handle = None

    def __del__(self):
        self.close()

    @property
    def workspace_bytes(self) -> int:
        return int(self.lib.cdg_muon_workspace_bytes(self.handle))

    def info(self) -> dict:
        inf = MuonInfo()
        rc = self.lib.cdg_muon_get_info(self.handle, ctypes.byref(inf))
        if rc != OK:
            raise CdgError(rc, "cdg_muon_get_info")
        return inf.as_dict()

    def _elements(self) -> int:
        d = self.shape
        return d["batch"] * d["rows"] * d["cols"]

    def orthogonalize(self, U, O, workspace, stream=None) -> None:
        """O = the Newton-Schulz orthogonalisation of every matrix of U (cdg_muon_orthogonalize)."""
        n, kind = self._elements(), _TYPES.get(self.dtype)
        _check_buffer(workspace, self.workspace_bytes, "workspace")
        rc = self.lib.cdg_muon_orthogonalize(self.handle, _dense(U, n, kind, "U"), _dense(O, n, kind, "O"),
                                             _addr(workspace), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_muon_orthogonalize")

    def step(self, W, G, M, W_out, M_out, workspace, lr: float, momentum: float = 0.95, weight_decay: float = 0.0,
             update_scale: float = 1.0, nesterov: bool = True, stream=None) -> None:
        """The weight update (cdg_muon_step): M_out = momentum * M + G, W_out =
        (1 - lr * weight_decay) * W - lr * update_scale * orthogonalize(U).
        W_out may be W and M_out may be M."""
        n = self._elements()
        _check_buffer(workspace, self.workspace_bytes, "workspace")
        rc = self.lib.cdg_muon_step(
            self.handle, _dense(W, n, "float32", "W"), _dense(G, n, _TYPES.get(self.dtype), "G"), _dense(M, n, "float32", "M"),
            _dense(W_out, n, "float32", "W_out"), _dense(M_out, n, "float32", "M_out"), float(lr), float(momentum),
            float(weight_decay), float(update_scale), int(bool(nesterov)), _addr(workspace), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_muon_step")

    def device_status(self, stream=None) -> int:
        return int(self.lib.cdg_muon_device_status(self.handle, _stream(stream)))


def muon_plan(rows, cols, batch=1, dtype="bf16", steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7) -> MuonPlan:
    return MuonPlan(rows, cols, batch, dtype, steps, coefficients, eps)


def muon_plan_host(rows, cols, batch=1, dtype="bf16", steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7,
                   num_sms=148) -> MuonPlan:
    return MuonPlan(rows, cols, batch, dtype, steps, coefficients, eps, host_sms=num_sms)


# ---- attention over packed sequences, and its gradient


class AttentionPlan:
    """Heads and mask of an attention (a ``cdg_attention_t``)."""

    def __init__(self, heads, kv_heads, dim, dtype="bf16", causal=True, window=0, scale: float | None = None,
                 host_only: bool = False):
        self.lib = load_library()
        self.heads, self.kv_heads, self.dim, self.dtype = int(heads), int(kv_heads), int(dim), dtype
        if scale is None:
            scale = max(self.dim, 1) ** -0.5
        make = self.lib.cdg_attention_plan_host if host_only else self.lib.cdg_attention_plan
        # (the C argument is an int: a larger window hides nothing either, and would lose its upper bits)
        window = max(-1, min(int(window), (1 << 31) - 1))
        h = ctypes.c_void_p()
        rc = make(self.heads, self.kv_heads, self.dim, _dtype(dtype), int(bool(causal)), window, float(scale),
                  ctypes.byref(h))
        if rc != OK:
            raise CdgError(rc, "cdg_attention_plan")
        self.handle = h
        self._need: dict = {}  # bytes of workspace, by the sizes that calls have had

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            self.lib.cdg_attention_destroy(self.handle)
        self.handle = None

    def __del__(self):
        self.close()

    def workspace_bytes(self, q_tokens: int, k_tokens: int, sequences: int = 1) -> int:
        """Bytes of attend's workspace (cdg_attention_workspace_bytes)."""
        return self._bytes(self.lib.cdg_attention_workspace_bytes, q_tokens, k_tokens, sequences)

    def grad_workspace_bytes(self, q_tokens: int, k_tokens: int, sequences: int = 1) -> int:
        """Bytes of attend_grad's workspace (cdg_attention_grad_workspace_bytes)."""
        return self._bytes(self.lib.cdg_attention_grad_workspace_bytes, q_tokens, k_tokens, sequences)

    def _bytes(self, fn, *sizes) -> int:
        n = int(fn(self.handle, *(int(v) for v in sizes)))
        if n == 0:
            raise CdgError(ERR_INVALID_ARG, fn.__name__)
        return n

    def attend(self, q, k, v, o, lse, workspace, q_tokens: int, k_tokens: int, q_offsets=None, k_offsets=None,
               sequences: int | None = None, ld_q=None, ld_k=None, ld_v=None, ld_o=None, stream=None) -> None:
        """o and lse (heads x q_tokens, fp32) of the queries over the keys and
        values (cdg_attention).  Offsets are int32 or int64 tensors of
        sequences + 1 numbers; without them all rows are one sequence."""
        nq, nk = int(q_tokens), int(k_tokens)
        qo, ko, ib, n = _offsets(q_offsets, k_offsets, sequences)
        _check_workspace(workspace, self._need, self.workspace_bytes, nq, nk, n)
        wq, wk = self.heads * self.dim, self.kv_heads * self.dim
        m = _matrices(_TYPES.get(self.dtype), (q, nq, wq, ld_q, "q"), (k, nk, wk, ld_k, "k"), (v, nk, wk, ld_v, "v"),
                      (o, nq, wq, ld_o, "o"))
        rc = self.lib.cdg_attention(self.handle, *m[:6], nq, nk, qo, ko, ib, n, m[6], m[7],
                                    *_vectors(self.heads * nq, (lse, "lse")), _addr(workspace), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_attention")

    def attend_grad(self, q, k, v, o, lse, do, dq, dk, dv, workspace, q_tokens: int, k_tokens: int, q_offsets=None,
                    k_offsets=None, sequences: int | None = None, ld_q=None, ld_k=None, ld_v=None, ld_o=None, ld_do=None,
                    ld_dq=None, ld_dk=None, ld_dv=None, stream=None) -> None:
        """dq, dk and dv for the gradient do of o (cdg_attention_grad); o and
        lse as attend wrote them."""
        nq, nk = int(q_tokens), int(k_tokens)
        qo, ko, ib, n = _offsets(q_offsets, k_offsets, sequences)
        _check_workspace(workspace, self._need, self.grad_workspace_bytes, nq, nk, n)
        wq, wk = self.heads * self.dim, self.kv_heads * self.dim
        m = _matrices(_TYPES.get(self.dtype), (q, nq, wq, ld_q, "q"), (k, nk, wk, ld_k, "k"), (v, nk, wk, ld_v, "v"),
                      (o, nq, wq, ld_o, "o"), (do, nq, wq, ld_do, "do"), (dq, nq, wq, ld_dq, "dq"), (dk, nk, wk, ld_dk, "dk"),
                      (dv, nk, wk, ld_dv, "dv"))
        rc = self.lib.cdg_attention_grad(self.handle, *m[:8], *_vectors(self.heads * nq, (lse, "lse")), m[8], m[9], nq, nk, qo, ko,
                                         ib, n, *m[10:], _addr(workspace), _stream(stream))
        if rc != OK:
            raise CdgError(rc, "cdg_attention_grad")

    def device_status(self, stream=None) -> int:
        return int(self.lib.cdg_attention_device_status(self.handle, _stream(stream)))


def _check_workspace(t, known: dict, need, *sizes) -> None:
    """Checks a workspace of need(*sizes) bytes; known holds what need has
    answered (its own call takes as long as all of the tensor's checks)."""
    if t is None or isinstance(t, int):
        return
    key = (need.__name__, sizes)
    n = known.get(key)
    if n is None:
        if len(known) > 64:
            known.clear()
        n = known[key] = need(*sizes)
    if type(t) is _tensor and t.nbytes >= n and t.is_contiguous() and t.get_device() == _cuda_device():
        return  # what the check below finds, without its cost
    _check_buffer(t, n, "workspace")


def _offsets(q_offsets, k_offsets, sequences) -> tuple:
    """Addresses of two offset lists, bytes per number, and the number of
    sequences (of raw addresses, which hold int64 numbers: as given, or one)."""
    if type(q_offsets) is _tensor and type(k_offsets) is _tensor and sequences is None and q_offsets.dtype is k_offsets.dtype:
        n = q_offsets.nbytes
        size = {"int32": 4, "int64": 8}.get(_type_names.get(q_offsets.dtype), 0)
        if size and n > 0 and k_offsets.nbytes >= n and q_offsets.is_contiguous() and k_offsets.is_contiguous() and \
                q_offsets.get_device() == k_offsets.get_device() == _cuda_device():
            return q_offsets.data_ptr(), k_offsets.data_ptr(), size, n // size - 1  # as below
    n = sequences
    for t in (q_offsets, k_offsets):
        if n is None and t is not None and not isinstance(t, int):
            n = t.numel() - 1
    n = 1 if n is None else int(n)
    qo, qb = _tokens(q_offsets, n + 1, "q_offsets")
    ko, kb = _tokens(k_offsets, n + 1, "k_offsets")
    if q_offsets is None:
        qb = kb
    elif k_offsets is not None and qb != kb:
        raise ValueError("q_offsets and k_offsets must hold numbers of one type")
    return qo, ko, qb, n


def attention_plan(heads, kv_heads, dim, dtype="bf16", causal=True, window=0, scale: float | None = None) -> AttentionPlan:
    """Attention of `heads` query heads over `kv_heads` key and value heads of
    width dim; scale defaults to dim ** -0.5."""
    return AttentionPlan(heads, kv_heads, dim, dtype, causal, window, scale)


def attention_plan_host(heads, kv_heads, dim, dtype="bf16", causal=True, window=0, scale: float | None = None) -> AttentionPlan:
    return AttentionPlan(heads, kv_heads, dim, dtype, causal, window, scale, host_only=True)


# ---- norms of queries and keys with the position rotation, and their gradient


def rope_frequencies(rot: int, base: float = 10000.0, stretch: float = 1.0, trained: int = 0, low: float = 1.0,
                     high: float = 32.0) -> list:
    """inv_freq for qk_rope (cdg_rope_frequencies): rot / 2 numbers, stretched
    for contexts longer than the `trained` tokens a model has seen."""
    out = (ctypes.c_float * max(1, int(rot) // 2))()
    rc = load_library().cdg_rope_frequencies(int(rot), float(base), float(stretch), int(trained), float(low), float(high), out)
    if rc != OK:
        raise CdgError(rc, "cdg_rope_frequencies")
    return list(out)[: int(rot) // 2]


def _rope_args(m, positions, inv_freq, tokens, heads, kv_heads, dim, dtype, rot, interleaved, factor, norm, eps, w_q, w_k):
    """The arguments that qk_rope and qk_rope_grad share; m: q's and k's addresses and row strides."""
    at, ib = _tokens(positions, tokens, "positions")
    return (*m, at, ib, tokens, heads, kv_heads, dim, _dtype(dtype), *_vectors(rot // 2, (inv_freq, "inv_freq")), rot,
            int(bool(interleaved)), float(factor), int(bool(norm)), float(eps), *_vectors(dim, (w_q, "w_q"), (w_k, "w_k")))


_rope_need: dict = {}  # bytes of qk_rope_grad's workspace, by the sizes that calls have had


def qk_rope(q, k, positions, inv_freq, q_out, k_out, tokens: int, heads: int, kv_heads: int, dim: int, dtype="bf16",
            rot: int | None = None, interleaved: bool = False, factor: float = 1.0, norm: bool = False, eps: float = 1e-6,
            w_q=None, w_k=None, ld_q=None, ld_k=None, ld_qo=None, ld_ko=None, stream=None) -> None:
    """Norms of queries and keys for each head (norm=True: weights w_q, w_k, or
    ones) and the position rotation of a head's first `rot` values (all of them
    by default) in one pass (cdg_qk_rope).  positions: int32 or int64, None for
    the token's number.  q_out may be q, and k_out k."""
    tokens, heads, kv_heads, dim = int(tokens), int(heads), int(kv_heads), int(dim)
    rot = dim if rot is None else int(rot)
    wq, wk = heads * dim, kv_heads * dim
    m = _matrices(_TYPES.get(dtype), (q if heads else None, tokens, wq, ld_q, "q"), (k if kv_heads else None, tokens, wk, ld_k, "k"),
                  (q_out if heads else None, tokens, wq, ld_qo, "q_out"), (k_out if kv_heads else None, tokens, wk, ld_ko, "k_out"))
    rc = load_library().cdg_qk_rope(*_rope_args(m[:4], positions, inv_freq, tokens, heads, kv_heads, dim, dtype, rot, interleaved,
                                                factor, norm, eps, w_q, w_k), *m[4:], _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_qk_rope")


def qk_rope_grad_workspace_bytes(tokens: int, heads: int, kv_heads: int, dim: int) -> int:
    """Bytes of qk_rope_grad's workspace (cdg_qk_rope_grad_workspace_bytes)."""
    n = int(load_library().cdg_qk_rope_grad_workspace_bytes(int(tokens), int(heads), int(kv_heads), int(dim)))
    if n == 0:
        raise CdgError(ERR_INVALID_ARG, "cdg_qk_rope_grad_workspace_bytes")
    return n


def qk_rope_grad(q, k, positions, inv_freq, dq_out, dk_out, dq, dk, workspace, tokens: int, heads: int, kv_heads: int, dim: int,
                 dtype="bf16", rot: int | None = None, interleaved: bool = False, factor: float = 1.0, norm: bool = False,
                 eps: float = 1e-6, w_q=None, w_k=None, dw_q=None, dw_k=None, ld_q=None, ld_k=None, ld_dqo=None, ld_dko=None,
                 ld_dq=None, ld_dk=None, stream=None) -> None:
    """The gradient of qk_rope (cdg_qk_rope_grad): dq and dk for the gradients
    dq_out and dk_out of its outputs, and with norm=True the weights' gradients
    dw_q and dw_k (fp32; None: not wanted).  q and k are qk_rope's inputs, not
    read without the norm.  dq may be dq_out, and dk dk_out."""
    tokens, heads, kv_heads, dim = int(tokens), int(heads), int(kv_heads), int(dim)
    rot = dim if rot is None else int(rot)
    wq, wk, qs, ks = heads * dim, kv_heads * dim, heads > 0, kv_heads > 0
    m = _matrices(_TYPES.get(dtype), (q if norm and qs else None, tokens, wq, ld_q, "q"),
                  (k if norm and ks else None, tokens, wk, ld_k, "k"),
                  (dq_out if qs else None, tokens, wq, ld_dqo, "dq_out"), (dk_out if ks else None, tokens, wk, ld_dko, "dk_out"),
                  (dq if qs else None, tokens, wq, ld_dq, "dq"), (dk if ks else None, tokens, wk, ld_dk, "dk"))
    _check_workspace(workspace, _rope_need, qk_rope_grad_workspace_bytes, tokens, heads, kv_heads, dim)
    rc = load_library().cdg_qk_rope_grad(*_rope_args(m[:4], positions, inv_freq, tokens, heads, kv_heads, dim, dtype, rot,
                                                     interleaved, factor, norm, eps, w_q, w_k), *m[4:],
                                         *_vectors(dim, (dw_q, "dw_q"), (dw_k, "dw_k")), _addr(workspace), _stream(stream))
    if rc != OK:
        raise CdgError(rc, "cdg_qk_rope_grad")
