"""Python binding of the fftconv C ABI (include/fftconv.h).

Argument marshalling only: every step of the convolution runs in the CUDA
library.  PyTorch supplies device memory and the current stream.  If the
library cannot be loaded, every call raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

from .build import LIB_PATH, build as build_library

F16, BF16 = 0, 1
PATH_FUSED, PATH_MULTIPASS = 0, 1
STATUS = {0: "OK", 1: "ERR_INVALID", 2: "ERR_UNSUPPORTED", 3: "ERR_ALIGN", 4: "ERR_WORKSPACE",
          5: "ERR_CUDA", 6: "ERR_ALLOC", 7: "ERR_TIMEOUT"}

EXPORTED = ["fftconv_plan_query", "fftconv_plan_create", "fftconv_plan_destroy", "fftconv_plan_get_info",
            "fftconv_kf_bytes", "fftconv_workspace_bytes", "fftconv_set_workspace", "fftconv_kernel_fft",
            "fftconv_forward", "fftconv_forward_gated", "fftconv_forward_noalloc", "fftconv_host_scratch_bytes",
            "fftconv_forward_host", "fftconv_kernel_fft_adjoint", "fftconv_backward_du",
            "fftconv_backward_du_gated", "fftconv_backward_dk_scratch_bytes", "fftconv_backward_dk",
            "fftconv_partial_scratch_bytes", "fftconv_forward_partial", "fftconv_circular_scratch_bytes",
            "fftconv_forward_circular", "fftconv_selftest_wait", "fftconv_plan_create_sparse",
            "fftconv_plan_get_band", "fftconv_sparse_query", "fftconv_circular_query",
            "fftconv_plan_create_circular", "fftconv_delta_create", "fftconv_delta_destroy",
            "fftconv_delta_status", "fftconv_delta_saved_bytes", "fftconv_delta_scratch_bytes",
            "fftconv_delta_forward", "fftconv_delta_backward", "fftconv_delta_step", "fftconv_qknorm_forward",
            "fftconv_qknorm_scratch_bytes", "fftconv_qknorm_backward", "fftconv_linattn_create",
            "fftconv_linattn_destroy", "fftconv_linattn_status", "fftconv_linattn_scratch_bytes",
            "fftconv_linattn_forward", "fftconv_linattn_backward", "fftconv_linattn_step",
            "fftconv_layernorm_forward", "fftconv_layernorm_scratch_bytes", "fftconv_layernorm_backward",
            "fftconv_device_status", "fftconv_status_string", "fftconv_version"]


class FFTConvError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("M", ctypes.c_int64), ("order", ctypes.c_int32),
                ("factors", ctypes.c_int32 * 8), ("path", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("kf_bytes_per_channel", ctypes.c_int64), ("workspace_bytes_per_row", ctypes.c_int64)]

    def as_dict(self):
        return {"N": self.N, "M": self.M, "order": self.order,
                "factors": list(self.factors[: self.order]), "path": self.path, "dtype": self.dtype,
                "kf_bytes_per_channel": self.kf_bytes_per_channel,
                "workspace_bytes_per_row": self.workspace_bytes_per_row}


class View(ctypes.Structure):
    """fftconv_view_t: a [B, T, H, D] (or [B, T, H]) tensor by its strides."""
    _fields_ = [("ptr", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class DeltaArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64), ("Hv", ctypes.c_int64),
                ("nseq", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("q", View), ("k", View), ("v", View), ("g", View), ("beta", View)]


class QKNormArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("norm", ctypes.c_int32), ("D", ctypes.c_int32), ("R", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("q", View), ("k", View), ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p),
                ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("table_rows", ctypes.c_int64),
                ("positions", ctypes.c_void_p)]


class LinAttnArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64), ("Hv", ctypes.c_int64),
                ("nseq", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("decay", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("q", View), ("k", View), ("v", View)]


class LayerNormArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("D", ctypes.c_int32), ("eps", ctypes.c_float),
                ("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("x", View),
                ("w", ctypes.c_void_p), ("b", ctypes.c_void_p)]


_lib = None


def lib(auto_build: bool = True):
    """Load (building first if needed) the CUDA library."""
    global _lib
    if _lib is None:
        if auto_build:
            build_library()
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"fftconv CUDA library not built: {LIB_PATH}")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.fftconv_plan_query.argtypes = [i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(PlanInfo)]
        L.fftconv_plan_create.argtypes = [ctypes.POINTER(vp), i64, ctypes.c_int, ctypes.c_int]
        L.fftconv_plan_create_sparse.argtypes = [ctypes.POINTER(vp), i64, ctypes.c_int, ctypes.c_int,
                                                 ctypes.POINTER(ctypes.c_int32), ctypes.c_int]
        L.fftconv_sparse_query.argtypes = [i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int32),
                                           ctypes.c_int, ctypes.POINTER(ctypes.c_int32),
                                           ctypes.POINTER(ctypes.c_int32)]
        L.fftconv_circular_query.argtypes = [i64, ctypes.c_int, ctypes.POINTER(PlanInfo)]
        L.fftconv_plan_create_circular.argtypes = [ctypes.POINTER(vp), i64, ctypes.c_int]
        L.fftconv_plan_get_band.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                            ctypes.POINTER(ctypes.c_int32)]
        L.fftconv_plan_destroy.argtypes = [vp]
        L.fftconv_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
        L.fftconv_kf_bytes.argtypes = [vp, i64]
        L.fftconv_kf_bytes.restype = sz
        L.fftconv_workspace_bytes.argtypes = [vp, i64, i64]
        L.fftconv_workspace_bytes.restype = sz
        L.fftconv_set_workspace.argtypes = [vp, vp, sz]
        L.fftconv_kernel_fft.argtypes = [vp, vp, vp, i64, vp]
        L.fftconv_forward.argtypes = [vp, vp, vp, vp, i64, i64, vp]
        L.fftconv_forward_gated.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp]
        L.fftconv_forward_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, vp]
        L.fftconv_host_scratch_bytes.argtypes = [vp, i64, i64, ctypes.c_int]
        L.fftconv_host_scratch_bytes.restype = sz
        L.fftconv_forward_host.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp, sz, vp]
        L.fftconv_kernel_fft_adjoint.argtypes = [vp, vp, vp, i64, vp]
        L.fftconv_backward_du.argtypes = [vp, vp, vp, vp, i64, i64, vp]
        L.fftconv_backward_du_gated.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp]
        L.fftconv_backward_dk_scratch_bytes.argtypes = [vp, i64, i64]
        L.fftconv_backward_dk_scratch_bytes.restype = sz
        L.fftconv_backward_dk.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp, sz, vp]
        L.fftconv_partial_scratch_bytes.argtypes = [vp, i64, i64, i64, ctypes.c_int]
        L.fftconv_partial_scratch_bytes.restype = sz
        L.fftconv_forward_partial.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
        L.fftconv_circular_scratch_bytes.argtypes = [vp, i64, i64, ctypes.c_int]
        L.fftconv_circular_scratch_bytes.restype = sz
        L.fftconv_forward_circular.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp, sz, vp]
        L.fftconv_selftest_wait.argtypes = [vp, ctypes.c_int, vp]
        da, qa, cint = ctypes.POINTER(DeltaArgs), ctypes.POINTER(QKNormArgs), ctypes.c_int
        L.fftconv_delta_create.argtypes = [ctypes.POINTER(vp), cint, cint, cint]
        L.fftconv_delta_destroy.argtypes = [vp]
        L.fftconv_delta_status.argtypes = [vp, vp, ctypes.POINTER(cint)]
        L.fftconv_delta_saved_bytes.argtypes = [vp, i64, i64, i64, i64]
        L.fftconv_delta_saved_bytes.restype = sz
        L.fftconv_delta_scratch_bytes.argtypes = [vp, i64, i64, i64, i64, i64, cint]
        L.fftconv_delta_scratch_bytes.restype = sz
        L.fftconv_delta_forward.argtypes = [vp, da, vp, View, vp, vp, vp, sz, vp]
        L.fftconv_delta_backward.argtypes = [vp, da, View, vp, vp, View, View, View, View, View, vp, vp, sz, vp]
        L.fftconv_delta_step.argtypes = [vp, da, vp, vp, i64, vp, View, vp]
        L.fftconv_qknorm_forward.argtypes = [qa, View, View, vp]
        L.fftconv_qknorm_scratch_bytes.argtypes = [qa]
        L.fftconv_qknorm_scratch_bytes.restype = sz
        L.fftconv_qknorm_backward.argtypes = [qa, View, View, View, View, vp, vp, vp, sz, vp]
        la, ln = ctypes.POINTER(LinAttnArgs), ctypes.POINTER(LayerNormArgs)
        L.fftconv_linattn_create.argtypes = [ctypes.POINTER(vp), cint, cint, cint]
        L.fftconv_linattn_destroy.argtypes = [vp]
        L.fftconv_linattn_status.argtypes = [vp, vp, ctypes.POINTER(cint)]
        L.fftconv_linattn_scratch_bytes.argtypes = [vp, i64, i64, i64, i64, i64, cint]
        L.fftconv_linattn_scratch_bytes.restype = sz
        L.fftconv_linattn_forward.argtypes = [vp, la, vp, View, vp, vp, sz, vp]
        L.fftconv_linattn_backward.argtypes = [vp, la, vp, View, vp, View, View, View, vp, vp, sz, vp]
        L.fftconv_linattn_step.argtypes = [vp, la, vp, vp, i64, vp, View, vp]
        L.fftconv_layernorm_forward.argtypes = [ln, View, vp]
        L.fftconv_layernorm_scratch_bytes.argtypes = [ln]
        L.fftconv_layernorm_scratch_bytes.restype = sz
        L.fftconv_layernorm_backward.argtypes = [ln, View, View, vp, vp, vp, sz, vp]
        L.fftconv_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int)]
        L.fftconv_status_string.argtypes = [ctypes.c_int]
        L.fftconv_status_string.restype = ctypes.c_char_p
        L.fftconv_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(st: int, what: str):
    if st != 0:
        raise FFTConvError(st, what)


def query(N: int, dtype: int, order: int = 0) -> dict:
    info = PlanInfo()
    _check(lib().fftconv_plan_query(N, dtype, order, ctypes.byref(info)), "fftconv_plan_query")
    return info.as_dict()


def circular_query(C: int, dtype: int) -> dict:
    """The plan a circular convolution of length C would use (no GPU)."""
    info = PlanInfo()
    _check(lib().fftconv_circular_query(C, dtype, ctypes.byref(info)), "fftconv_circular_query")
    return info.as_dict()


def sparse_query(N: int, dtype: int, band, order: int = 0) -> dict:
    """Pairs of sub-rows a frequency-sparse plan would transform (no GPU)."""
    arr = (ctypes.c_int32 * max(1, len(band)))(*[int(b) for b in band])
    run, tot = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fftconv_sparse_query(N, dtype, order, arr, len(band), ctypes.byref(run), ctypes.byref(tot)),
           "fftconv_sparse_query")
    return {"pairs_run": run.value, "pairs_total": tot.value}


def _dtype_code(torch_dtype) -> int:
    import torch
    if torch_dtype == torch.float16:
        return F16
    if torch_dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {torch_dtype}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, dev=None) -> Optional[int]:
    """A call's stream: the current one of GPU dev (None: of the current GPU) by default."""
    if stream is not None:
        return stream.cuda_stream
    import torch  # torch.cuda.current_stream() takes 12 us
    return torch._C._cuda_getCurrentRawStream(_current_device() if dev is None else dev)


class Plan:
    """A plan for one sequence length N and dtype (torch.float16 / bfloat16)."""

    def __init__(self, N: int, dtype, order: int = 0, band=None, circular: bool = False):
        """band: one int per factor (outer first) for a frequency-sparse plan;
        None for the dense convolution.  circular: a plan for the circular
        convolution of length N (rows of N samples, k of N taps)."""
        self.N = int(N)
        self.torch_dtype = dtype
        self.dtype = _dtype_code(dtype)
        self.circular = bool(circular)
        h = ctypes.c_void_p()
        if circular:
            if band is not None or order != 0:
                raise ValueError("a circular plan takes no band and no order")
            _check(lib().fftconv_plan_create_circular(ctypes.byref(h), self.N, self.dtype),
                   "fftconv_plan_create_circular")
        elif band is None:
            _check(lib().fftconv_plan_create(ctypes.byref(h), self.N, self.dtype, order), "fftconv_plan_create")
        else:
            arr = (ctypes.c_int32 * max(1, len(band)))(*[int(b) for b in band])
            _check(lib().fftconv_plan_create_sparse(ctypes.byref(h), self.N, self.dtype, order, arr, len(band)),
                   "fftconv_plan_create_sparse")
        self._h = h
        info = PlanInfo()
        _check(lib().fftconv_plan_get_info(self._h, ctypes.byref(info)), "fftconv_plan_get_info")
        self.info = info.as_dict()
        self._workspace = None
        self._host_scratch = None

    def band(self) -> dict:
        """The plan's band per factor and the pass-B pairs that run / exist."""
        b = (ctypes.c_int32 * 8)()
        run, tot = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().fftconv_plan_get_band(self._h, b, ctypes.byref(run), ctypes.byref(tot)), "fftconv_plan_get_band")
        return {"band": list(b[: self.info["order"]]), "pairs_run": run.value, "pairs_total": tot.value}

    def close(self):
        if getattr(self, "_h", None):
            lib().fftconv_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def kf_bytes(self, H: int) -> int:
        return int(lib().fftconv_kf_bytes(self._h, H))

    def workspace_bytes(self, B: int, H: int) -> int:
        return int(lib().fftconv_workspace_bytes(self._h, B, H))

    def set_workspace(self, buf) -> None:
        """Attach a caller-owned device buffer (a torch tensor kept alive here)."""
        self._workspace = buf
        n = 0 if buf is None else buf.numel() * buf.element_size()
        _check(lib().fftconv_set_workspace(self._h, _ptr(buf), n), "fftconv_set_workspace")

    def kernel_fft(self, k, k_f=None, stream=None):
        """k: float32 [H, N] on the GPU -> opaque k_f (uint8 tensor)."""
        import torch
        H = k.shape[0]
        if k.dtype != torch.float32 or not k.is_contiguous() or k.shape[-1] != self.N:
            raise ValueError("k must be contiguous float32 [H, N]")
        if k_f is None:
            k_f = torch.empty(self.kf_bytes(H), dtype=torch.uint8, device=k.device)
        _check(lib().fftconv_kernel_fft(self._h, _ptr(k), _ptr(k_f), H, _stream(stream)), "fftconv_kernel_fft")
        return k_f

    def _ensure_workspace(self, B, H, device):
        import torch
        need = self.workspace_bytes(B, H)
        if need and (self._workspace is None or self._workspace.numel() < need):
            self.set_workspace(torch.empty(need, dtype=torch.uint8, device=device))

    def forward(self, u, k_f, y=None, stream=None):
        """u: [B, H, N] (plan dtype, GPU) -> y = causal conv with k."""
        import torch
        B, H, N = u.shape
        if y is None:
            y = torch.empty_like(u)
        self._ensure_workspace(B, H, u.device)
        _check(lib().fftconv_forward(self._h, _ptr(u), _ptr(k_f), _ptr(y), B, H, _stream(stream)),
               "fftconv_forward")
        return y

    def forward_gated(self, u, w_in, w_out, k_f, y=None, stream=None):
        """y = w_out * conv(u * w_in, k)."""
        import torch
        B, H, N = u.shape
        if y is None:
            y = torch.empty_like(u)
        self._ensure_workspace(B, H, u.device)
        _check(lib().fftconv_forward_gated(self._h, _ptr(u), _ptr(w_in), _ptr(w_out), _ptr(k_f), _ptr(y),
                                           B, H, _stream(stream)), "fftconv_forward_gated")
        return y

    def forward_host(self, u, k_f, w_in=None, w_out=None, y=None, stream=None):
        """u (and w_in, w_out): host tensors [B, H, N] in the plan dtype,
        page-locked for the copies to overlap -> y (host).  Chunks of rows are
        copied in, convolved and copied back with the three steps overlapped;
        y is complete once the stream has been synchronised."""
        import torch
        for t in (u, w_in, w_out, y):
            if t is not None and (t.is_cuda or not t.is_contiguous() or t.dtype != self.torch_dtype):
                raise ValueError("host tensors must be contiguous CPU tensors of the plan dtype")
        if (w_in is None) != (w_out is None):
            raise ValueError("w_in and w_out go together")
        B, H, N = u.shape
        if y is None:
            y = torch.empty(u.shape, dtype=u.dtype, pin_memory=True)
        gated = w_in is not None
        need = int(lib().fftconv_host_scratch_bytes(self._h, B, H, int(gated)))
        if need and (self._host_scratch is None or self._host_scratch.numel() < need):
            self._host_scratch = torch.empty(need, dtype=torch.uint8, device=k_f.device)
        n = 0 if self._host_scratch is None else self._host_scratch.numel()
        _check(lib().fftconv_forward_host(self._h, _ptr(u), _ptr(w_in), _ptr(w_out), _ptr(k_f), _ptr(y), B, H,
                                          _ptr(self._host_scratch), n, _stream(stream)), "fftconv_forward_host")
        return y

    # ---- partial convolution (kernels of at most N/2 taps, sequences of any multiple of N/2)

    def kernel_fft_partial(self, k, k_f=None, stream=None):
        """k: float32 [H, T] with T <= N/2 taps -> k_f for forward_partial."""
        import torch
        H, T = k.shape
        if T > self.N // 2:
            raise ValueError(f"a partial-convolution kernel has at most {self.N // 2} taps")
        kp = torch.zeros(H, self.N, dtype=torch.float32, device=k.device)
        kp[:, :T] = k
        return self.kernel_fft(kp, k_f=k_f, stream=stream)

    def forward_partial(self, u, k_f, w_in=None, w_out=None, y=None, stream=None):
        """u: [B, H, N'] with N' a multiple of N/2 -> the causal convolution with
        the kernel of kernel_fft_partial (gated when w_in, w_out are given)."""
        import torch
        B, H, Np = u.shape
        if y is None:
            y = torch.empty_like(u)
        gated = w_in is not None
        need = int(lib().fftconv_partial_scratch_bytes(self._h, B, H, Np, int(gated)))
        scratch = torch.empty(max(need, 16), dtype=torch.uint8, device=u.device)
        _check(lib().fftconv_forward_partial(self._h, _ptr(u), _ptr(w_in), _ptr(w_out), _ptr(k_f), _ptr(y), B, H, Np,
                                             _ptr(scratch), need, _stream(stream)), "fftconv_forward_partial")
        return y

    def forward_circular(self, u, k_f, w_in=None, w_out=None, y=None, stream=None):
        """u: [B, H, N/2] -> circular convolution of length N/2 with the kernel
        of kernel_fft_partial (its N/2 taps)."""
        import torch
        B, H, C = u.shape
        if C != self.N // 2:
            raise ValueError(f"circular length must be {self.N // 2} for this plan")
        if y is None:
            y = torch.empty_like(u)
        gated = w_in is not None
        need = int(lib().fftconv_circular_scratch_bytes(self._h, B, H, int(gated)))
        scratch = torch.empty(max(need, 16), dtype=torch.uint8, device=u.device)
        _check(lib().fftconv_forward_circular(self._h, _ptr(u), _ptr(w_in), _ptr(w_out), _ptr(k_f), _ptr(y), B, H,
                                              _ptr(scratch), need, _stream(stream)), "fftconv_forward_circular")
        return y

    # ---- backward (gradients in u and k)

    def kernel_fft_adjoint(self, k, k_f=None, stream=None):
        """k: float32 [H, N] -> opaque adjoint k_f (correlation with k)."""
        import torch
        H = k.shape[0]
        if k.dtype != torch.float32 or not k.is_contiguous() or k.shape[-1] != self.N:
            raise ValueError("k must be contiguous float32 [H, N]")
        if k_f is None:
            k_f = torch.empty(self.kf_bytes(H), dtype=torch.uint8, device=k.device)
        _check(lib().fftconv_kernel_fft_adjoint(self._h, _ptr(k), _ptr(k_f), H, _stream(stream)),
               "fftconv_kernel_fft_adjoint")
        return k_f

    def backward_du(self, dy, k_f_adj, w_in=None, w_out=None, du=None, stream=None):
        """du = corr(dy, k) (gated: w_in * corr(w_out * dy, k))."""
        import torch
        B, H, N = dy.shape
        if du is None:
            du = torch.empty_like(dy)
        self._ensure_workspace(B, H, dy.device)
        if w_in is None:
            st = lib().fftconv_backward_du(self._h, _ptr(dy), _ptr(k_f_adj), _ptr(du), B, H, _stream(stream))
        else:
            st = lib().fftconv_backward_du_gated(self._h, _ptr(dy), _ptr(w_in), _ptr(w_out), _ptr(k_f_adj),
                                                 _ptr(du), B, H, _stream(stream))
        _check(st, "fftconv_backward_du")
        return du

    def backward_dk(self, u, dy, w_in=None, w_out=None, dk=None, stream=None):
        """dk [H, N] float32 = sum_b corr(w_out * dy_b, w_in * u_b)."""
        import torch
        B, H, N = u.shape
        if dk is None:
            dk = torch.empty(H, N, dtype=torch.float32, device=u.device)
        need = int(lib().fftconv_backward_dk_scratch_bytes(self._h, B, H))
        scratch = torch.empty(max(need, 16), dtype=torch.uint8, device=u.device)
        _check(lib().fftconv_backward_dk(self._h, _ptr(u), _ptr(dy), _ptr(w_in), _ptr(w_out), _ptr(dk), B, H,
                                         _ptr(scratch), need, _stream(stream)), "fftconv_backward_dk")
        return dk

    def device_status(self, stream=None) -> int:
        v = ctypes.c_int()
        _check(lib().fftconv_device_status(self._h, _stream(stream), ctypes.byref(v)), "fftconv_device_status")
        return v.value


def status_string(code: int) -> str:
    return lib().fftconv_status_string(code).decode()


# ---- token mixers with a state: strided token-major tensors [B, T, H, D]
#
# A decoding step is a few microseconds of GPU work, so these calls keep their
# own work small: each tensor is looked at once, and the argument structures
# are packed in one go.  All tensors of a call are on the current GPU (checked).

_DELTA_ARGS = struct.Struct("=5qQf4x" + "Q3q" * 5)
_NORM_ARGS = struct.Struct("=5if4q" + "Q3q" * 2 + "4QqQ")
_LINATTN_ARGS = struct.Struct("=5qQQf4x" + "Q3q" * 3)
_LAYERNORM_ARGS = struct.Struct("=2if4x3q" + "Q3q" + "2Q")


def _current_device() -> int:
    import torch
    return torch._C._cuda_getDevice()


def _device(t, what: str) -> int:
    """The GPU of a call's first tensor, which has to be the current one: that is
    where the call's stream, its outputs and its scratch are."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"{what} must be a CUDA tensor on the current GPU")
    return dev


def _elsewhere(t, dev) -> bool:
    """Whether t is not on GPU dev (None: any)."""
    return not t.is_cuda if dev is None else t.get_device() != dev


def _strides(t, what: str, dtype, shape, dev=None):
    """A tensor's address and its first three strides, checked against dtype, shape and GPU."""
    st = t.stride()
    if t.shape != shape or t.dtype is not dtype or _elsewhere(t, dev) or (len(st) == 4 and st[3] != 1 and shape[3] > 1):
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)} on the call's GPU, contiguous in its features")
    return (t.data_ptr(), *st[:3])


def _new(t):
    """An uninitialised contiguous tensor like t, and its view."""
    import torch
    o = torch.empty_like(t, memory_format=torch.contiguous_format)
    return o, View(o.data_ptr(), *o.stride()[:3])


def _dense(t, what: str, dtype, shape, dev=None) -> int:
    """The address of a contiguous tensor of the given shape and GPU (None: 0)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or _elsewhere(t, dev) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the call's GPU")
    return t.data_ptr()


def _slots_of(state) -> int:
    """How many states a step's pool holds."""
    if state is None or state.dim() != 4:
        raise ValueError("state must be float32 [slots, Hv, Dk, Dv]")
    return state.shape[0]


def _on(stream):
    """Allocations made inside belong to the stream that the call runs on."""
    import torch
    return torch.cuda.stream(stream)


class DeltaRule:
    """The gated delta rule for head sizes Dk, Dv (64 or 128) and one dtype:

        S~ = exp(g_t) S;  u = beta_t (v_t - S~^T k_t);  S = S~ + k_t u^T;  o_t = scale S^T q_t

    q, k: [B, T, Hk, Dk]; v: [B, T, Hv, Dv]; g (log decay), beta: [B, T, Hv];
    Hv a multiple of Hk.  States: float32 [sequences, Hv, Dk, Dv].  offsets:
    int32 [n + 1] on the GPU for n sequences packed into one row (B = 1).
    scale defaults to Dk ** -0.5."""

    def __init__(self, Dk: int, Dv: int, dtype):
        self.Dk, self.Dv, self.torch_dtype = int(Dk), int(Dv), dtype
        self._scale = self.Dk ** -0.5
        h = ctypes.c_void_p()
        _check(lib().fftconv_delta_create(ctypes.byref(h), self.Dk, self.Dv, _dtype_code(dtype)),
               "fftconv_delta_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().fftconv_delta_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _args(self, q, k, v, g, beta, offsets, scale) -> DeltaArgs:
        import torch
        dt = self.torch_dtype
        if q.dim() != 4 or v.dim() != 4 or q.shape[3] != self.Dk:
            raise ValueError("q, k must be [B, T, Hk, Dk] and v [B, T, Hv, Dv]")
        B, T, Hk, _ = qs = q.shape
        Hv = v.shape[2]
        gs = (B, T, Hv)
        dev = _device(q, "q")
        nseq, off = B, 0
        if offsets is not None:
            if offsets.dim() != 1 or offsets.numel() < 1:
                raise ValueError("offsets must be [n + 1]")
            nseq = offsets.numel() - 1
            off = _dense(offsets, "offsets", torch.int32, offsets.shape, dev)
        return DeltaArgs.from_buffer_copy(_DELTA_ARGS.pack(
            B, T, Hk, Hv, nseq, off, self._scale if scale is None else scale, *_strides(q, "q", dt, qs, dev),
            *_strides(k, "k", dt, qs, dev), *_strides(v, "v", dt, (B, T, Hv, self.Dv), dev),
            *_strides(g, "g", dt, gs, dev), *_strides(beta, "beta", dt, gs, dev)))

    def _scratch(self, a, which, device):
        import torch
        n = int(lib().fftconv_delta_scratch_bytes(self._h, a.B, a.T, a.Hk, a.Hv, a.nseq, which))
        return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n

    def forward(self, q, k, v, g, beta, state=None, offsets=None, scale=None, save=False, stream=None):
        """Whole sequences from `state` (None: zero) -> (o, final states), and
        with save=True also what backward needs: (o, final states, saved)."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.forward(q, k, v, g, beta, state, offsets, scale, save)
        a = self._args(q, k, v, g, beta, offsets, scale)
        shape = (a.nseq, a.Hv, self.Dk, self.Dv)
        sin = _dense(state, "state", torch.float32, shape, q.get_device())
        o, vo = _new(v)
        out = torch.empty(shape, dtype=torch.float32, device=v.device)
        saved = None
        if save:
            n = int(lib().fftconv_delta_saved_bytes(self._h, a.B, a.T, a.Hv, a.nseq))
            saved = torch.empty(n, dtype=torch.uint8, device=v.device)
        scratch, n = self._scratch(a, 2 if save else 0, v.device)
        _check(lib().fftconv_delta_forward(self._h, ctypes.byref(a), sin, vo, out.data_ptr(), _ptr(saved),
                                           _ptr(scratch), n, _stream(None)), "fftconv_delta_forward")
        return (o, out, saved) if save else (o, out)

    def backward(self, do, q, k, v, g, beta, saved, dstate=None, offsets=None, scale=None, stream=None):
        """Gradients (dq, dk, dv, dg, dbeta, gradient of the initial states)
        from do [B, T, Hv, Dv] and, if the final states were used, dstate;
        `saved` and the other arguments as in forward."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.backward(do, q, k, v, g, beta, saved, dstate, offsets, scale)
        a = self._args(q, k, v, g, beta, offsets, scale)
        dt, dev = self.torch_dtype, q.get_device()
        shape = (a.nseq, a.Hv, self.Dk, self.Dv)
        dsin = _dense(dstate, "dstate", torch.float32, shape, dev)
        vdo = View(*_strides(do, "do", dt, v.shape, dev))
        sv = _dense(saved, "saved", torch.uint8,
                    (int(lib().fftconv_delta_saved_bytes(self._h, a.B, a.T, a.Hv, a.nseq)),), dev)
        grads, views = zip(*(_new(t) for t in (q, k, v, g, beta)))
        dst = torch.empty(shape, dtype=torch.float32, device=v.device)
        scratch, n = self._scratch(a, 1, v.device)
        _check(lib().fftconv_delta_backward(self._h, ctypes.byref(a), vdo, dsin, sv, *views, dst.data_ptr(), _ptr(scratch), n,
                                            _stream(None)), "fftconv_delta_backward")
        return (*grads, dst)

    def step(self, q, k, v, g, beta, state, state_out=None, slots=None, scale=None, stream=None):
        """The recurrent form: B rows of a few tokens, row b against
        state[slots[b]] (slots: int32 [B] on the GPU, distinct; None: state[b])
        -> o.  The updated states go to state_out, by default back to state."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.step(q, k, v, g, beta, state, state_out, slots, scale)
        a = self._args(q, k, v, g, beta, None, scale)
        shape = (_slots_of(state), v.shape[2], self.Dk, self.Dv)
        sin = _dense(state, "state", torch.float32, shape, q.get_device())
        sout = sin if state_out is None else _dense(state_out, "state_out", torch.float32, shape, q.get_device())
        sl = _dense(slots, "slots", torch.int32, (q.shape[0],), q.get_device())
        o, vo = _new(v)
        _check(lib().fftconv_delta_step(self._h, ctypes.byref(a), sin, sout, shape[0], sl, vo, _stream(None)),
               "fftconv_delta_step")
        return o

    def device_status(self, stream=None) -> int:
        v = ctypes.c_int()
        _check(lib().fftconv_delta_status(self._h, _stream(stream), ctypes.byref(v)), "fftconv_delta_status")
        return v.value


class QKNorm:
    """Norm of queries and keys for each head, with the position rotation of
    the first `rotary` features in the same pass.  norm: "rms" or "l2"."""

    def __init__(self, D: int, dtype, norm: str = "rms", eps: float = 1e-6, rotary: int = 0, interleaved: bool = False):
        if norm not in ("rms", "l2"):
            raise ValueError('norm must be "rms" or "l2"')
        self.D, self.torch_dtype, self.norm, self.eps = int(D), dtype, norm, float(eps)
        self.rotary, self.interleaved = int(rotary), bool(interleaved)
        self._code, self._norm = _dtype_code(dtype), int(norm == "l2")

    def _args(self, q, k, wq, wk, cos, sin, positions) -> QKNormArgs:
        import torch
        dt, D, R, f32 = self.torch_dtype, self.D, self.rotary, torch.float32
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("q must be [B, T, Hq, D] and k [B, T, Hk, D]")
        B, T, Hq, _ = q.shape
        Hk = k.shape[2]
        pc = ps = pp = rows = 0
        dev = _device(q, "q")
        if R:
            if cos is None or sin is None:
                raise ValueError("a rotation needs cos and sin")
            rows = cos.shape[0]
            pc, ps = _dense(cos, "cos", f32, (rows, R // 2), dev), _dense(sin, "sin", f32, (rows, R // 2), dev)
            pp = _dense(positions, "positions", torch.int32, (B, T), dev)
        return QKNormArgs.from_buffer_copy(_NORM_ARGS.pack(
            self._code, self._norm, D, R, self.interleaved, self.eps, B, T, Hq, Hk,
            *_strides(q, "q", dt, (B, T, Hq, D), dev), *_strides(k, "k", dt, (B, T, Hk, D), dev),
            _dense(wq, "wq", f32, (D,), dev), _dense(wk, "wk", f32, (D,), dev), pc, ps, rows, pp))

    def forward(self, q, k, wq=None, wk=None, cos=None, sin=None, positions=None, qo=None, ko=None, stream=None):
        """q: [B, T, Hq, D], k: [B, T, Hk, D] -> the normed and rotated (q, k).
        wq, wk: float32 [D] or None (ones); cos, sin: float32 [rows, rotary/2];
        positions: int32 [B, T] (None: the token's index).  qo, ko: where to
        write (q and k themselves are allowed)."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.forward(q, k, wq, wk, cos, sin, positions, qo, ko)
        args = ctypes.byref(self._args(q, k, wq, wk, cos, sin, positions))
        dt, dev = self.torch_dtype, q.get_device()
        qo, vq = _new(q) if qo is None else (qo, View(*_strides(qo, "qo", dt, q.shape, dev)))
        ko, vk = _new(k) if ko is None else (ko, View(*_strides(ko, "ko", dt, k.shape, dev)))
        _check(lib().fftconv_qknorm_forward(args, vq, vk, _stream(None)), "fftconv_qknorm_forward")
        return qo, ko

    def backward(self, dqo, dko, q, k, wq=None, wk=None, cos=None, sin=None, positions=None, stream=None):
        """Gradients (dq, dk, dwq, dwk) from those of forward's outputs; dwq
        (dwk) is None where wq (wk) is."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.backward(dqo, dko, q, k, wq, wk, cos, sin, positions)
        args = ctypes.byref(self._args(q, k, wq, wk, cos, sin, positions))
        dt, dev = self.torch_dtype, q.get_device()
        vdq = View(*_strides(dqo, "dqo", dt, q.shape, dev))
        vdk = View(*_strides(dko, "dko", dt, k.shape, dev))
        (dq, oq), (dk, ok) = _new(q), _new(k)
        dwq, dwk = (None if w is None else torch.empty(self.D, dtype=torch.float32, device=q.device)
                    for w in (wq, wk))
        n = int(lib().fftconv_qknorm_scratch_bytes(args)) if (wq is not None or wk is not None) else 0
        scratch = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
        _check(lib().fftconv_qknorm_backward(args, vdq, vdk, oq, ok, _ptr(dwq), _ptr(dwk), _ptr(scratch), n,
                                             _stream(None)), "fftconv_qknorm_backward")
        return dq, dk, dwq, dwk


class LinearAttention:
    """Linear attention with a fixed decay for each head, for head sizes Dk, Dv
    (64 or 128) and one dtype:

        S = exp(decay) S + k_t v_t^T;  o_t = scale S^T q_t

    q, k: [B, T, Hk, Dk]; v: [B, T, Hv, Dv]; decay: float32 [Hv], logarithms
    (taken as at most 0; constants of the layer, without a gradient); Hv a
    multiple of Hk.  States: float32 [sequences, Hv, Dk, Dv].  offsets: int32
    [n + 1] on the GPU for n sequences packed into one row (B = 1).  scale
    defaults to Dk ** -0.5."""

    def __init__(self, Dk: int, Dv: int, dtype):
        self.Dk, self.Dv, self.torch_dtype = int(Dk), int(Dv), dtype
        self._scale = self.Dk ** -0.5
        h = ctypes.c_void_p()
        _check(lib().fftconv_linattn_create(ctypes.byref(h), self.Dk, self.Dv, _dtype_code(dtype)),
               "fftconv_linattn_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().fftconv_linattn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _args(self, q, k, v, decay, offsets, scale) -> LinAttnArgs:
        import torch
        dt = self.torch_dtype
        if q.dim() != 4 or v.dim() != 4 or q.shape[3] != self.Dk:
            raise ValueError("q, k must be [B, T, Hk, Dk] and v [B, T, Hv, Dv]")
        B, T, Hk, _ = qs = q.shape
        Hv = v.shape[2]
        dev = _device(q, "q")
        nseq, off = B, 0
        if offsets is not None:
            if offsets.dim() != 1 or offsets.numel() < 1:
                raise ValueError("offsets must be [n + 1]")
            nseq = offsets.numel() - 1
            off = _dense(offsets, "offsets", torch.int32, offsets.shape, dev)
        if decay is None:
            raise ValueError("decay must be float32 [Hv]")
        return LinAttnArgs.from_buffer_copy(_LINATTN_ARGS.pack(
            B, T, Hk, Hv, nseq, off, _dense(decay, "decay", torch.float32, (Hv,), dev),
            self._scale if scale is None else scale, *_strides(q, "q", dt, qs, dev), *_strides(k, "k", dt, qs, dev),
            *_strides(v, "v", dt, (B, T, Hv, self.Dv), dev)))

    def _scratch(self, a, backward, device):
        import torch
        n = int(lib().fftconv_linattn_scratch_bytes(self._h, a.B, a.T, a.Hk, a.Hv, a.nseq, backward))
        return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n

    def forward(self, q, k, v, decay, state=None, offsets=None, scale=None, stream=None):
        """Whole sequences from `state` (None: zero) -> (o, final states)."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.forward(q, k, v, decay, state, offsets, scale)
        a = self._args(q, k, v, decay, offsets, scale)
        shape = (a.nseq, a.Hv, self.Dk, self.Dv)
        dev = q.get_device()
        sin = _dense(state, "state", torch.float32, shape, dev)
        o, vo = _new(v)
        out = torch.empty(shape, dtype=torch.float32, device=v.device)
        scratch, n = self._scratch(a, 0, v.device)
        _check(lib().fftconv_linattn_forward(self._h, ctypes.byref(a), sin, vo, out.data_ptr(), _ptr(scratch), n,
                                             _stream(None, dev)), "fftconv_linattn_forward")
        return o, out

    def backward(self, do, q, k, v, decay, state=None, dstate=None, offsets=None, scale=None, stream=None):
        """Gradients (dq, dk, dv, gradient of the initial states) from do
        [B, T, Hv, Dv] and, if the final states were used, dstate; the last is
        None where state is.  The other arguments as in forward, which keeps
        nothing for this call."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.backward(do, q, k, v, decay, state, dstate, offsets, scale)
        a = self._args(q, k, v, decay, offsets, scale)
        dev = q.get_device()
        shape = (a.nseq, a.Hv, self.Dk, self.Dv)
        sin = _dense(state, "state", torch.float32, shape, dev)
        dsin = _dense(dstate, "dstate", torch.float32, shape, dev)
        vdo = View(*_strides(do, "do", self.torch_dtype, v.shape, dev))
        (dq, oq), (dk, ok), (dv, ov) = _new(q), _new(k), _new(v)
        dst = None if state is None else torch.empty(shape, dtype=torch.float32, device=v.device)
        scratch, n = self._scratch(a, 1, v.device)
        _check(lib().fftconv_linattn_backward(self._h, ctypes.byref(a), sin, vdo, dsin, oq, ok, ov, _ptr(dst),
                                              _ptr(scratch), n, _stream(None, dev)), "fftconv_linattn_backward")
        return dq, dk, dv, dst

    def step(self, q, k, v, decay, state, state_out=None, slots=None, scale=None, stream=None):
        """The recurrent form: B rows of a few tokens, row b against
        state[slots[b]] (slots: int32 [B] on the GPU, distinct; None: state[b])
        -> o.  The updated states go to state_out, by default back to state."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.step(q, k, v, decay, state, state_out, slots, scale)
        a = self._args(q, k, v, decay, None, scale)
        shape, dev = (_slots_of(state), v.shape[2], self.Dk, self.Dv), q.get_device()
        sin = _dense(state, "state", torch.float32, shape, dev)
        sout = sin if state_out is None else _dense(state_out, "state_out", torch.float32, shape, dev)
        sl = _dense(slots, "slots", torch.int32, (q.shape[0],), dev)
        o, vo = _new(v)
        _check(lib().fftconv_linattn_step(self._h, ctypes.byref(a), sin, sout, shape[0], sl, vo, _stream(None, dev)),
               "fftconv_linattn_step")
        return o

    def device_status(self, stream=None) -> int:
        v = ctypes.c_int()
        _check(lib().fftconv_linattn_status(self._h, _stream(stream), ctypes.byref(v)), "fftconv_linattn_status")
        return v.value


class LayerNorm:
    """Layer norm of rows of D features:

        y = (x - mean) / sqrt(var + eps) * w + b

    x: [N, D] or [B, T, D] (rows of a hidden state) with w, b float32 [D], or
    [B, T, H, D] (a mixer's heads, normed one by one) with w, b float32 [H, D];
    either may be None (ones, zeros)."""

    def __init__(self, D: int, dtype, eps: float = 1e-5):
        self.D, self.torch_dtype, self.eps = int(D), dtype, float(eps)
        self._code = _dtype_code(dtype)

    def _new(self, x, a):
        """An uninitialised contiguous tensor like x, and its view."""
        import torch
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        return y, View(y.data_ptr(), a.T * a.H * self.D, a.H * self.D, self.D)

    def _view(self, t, what, shape, dev):
        """A tensor's address and its batch, token and head strides."""
        st = t.stride()
        if t.shape != shape or t.dtype is not self.torch_dtype or t.get_device() != dev or (st[-1] != 1 and shape[-1] > 1):
            raise ValueError(f"{what} must be a {self.torch_dtype} tensor of shape {tuple(shape)} on the call's GPU, "
                             "contiguous in its features")
        n = len(st)
        if n == 4:
            return t.data_ptr(), st[0], st[1], st[2]
        return (t.data_ptr(), st[0], st[1], self.D) if n == 3 else (t.data_ptr(), self.D, st[0], self.D)

    def _args(self, x, w, b) -> LayerNormArgs:
        import torch
        shape, n, D = x.shape, x.dim(), self.D
        if n < 2 or n > 4 or shape[-1] != D:
            raise ValueError("x must be [N, D], [B, T, D] or [B, T, H, D]")
        dev = _device(x, "x")
        B, T, H = (1, shape[0], 1) if n == 2 else (shape[0], shape[1], shape[2] if n == 4 else 1)
        ws = (H, D) if n == 4 else (D,)
        return LayerNormArgs.from_buffer_copy(_LAYERNORM_ARGS.pack(
            self._code, D, self.eps, B, T, H, *self._view(x, "x", shape, dev),
            _dense(w, "w", torch.float32, ws, dev), _dense(b, "b", torch.float32, ws, dev)))

    def forward(self, x, w=None, b=None, y=None, stream=None):
        """The normed rows.  y: where to write (x itself is allowed)."""
        if stream is not None:
            with _on(stream):
                return self.forward(x, w, b, y)
        a, dev = self._args(x, w, b), x.get_device()
        if y is None:
            y, vy = self._new(x, a)
        else:
            vy = View(*self._view(y, "y", x.shape, dev))
        _check(lib().fftconv_layernorm_forward(ctypes.byref(a), vy, _stream(None, dev)), "fftconv_layernorm_forward")
        return y

    def backward(self, dy, x, w=None, b=None, stream=None):
        """Gradients (dx, dw, db) from that of forward's output; dw (db) is
        None where w (b) is."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.backward(dy, x, w, b)
        a, dev = self._args(x, w, b), x.get_device()
        vdy = View(*self._view(dy, "dy", x.shape, dev))
        dx, vdx = self._new(x, a)
        dw, db = (None if t is None else torch.empty_like(t) for t in (w, b))
        n = int(lib().fftconv_layernorm_scratch_bytes(ctypes.byref(a))) if (w is not None or b is not None) else 0
        scratch = x.new_empty(n, dtype=torch.uint8) if n else None
        _check(lib().fftconv_layernorm_backward(ctypes.byref(a), vdy, vdx, _ptr(dw), _ptr(db), _ptr(scratch), n,
                                                _stream(None, dev)), "fftconv_layernorm_backward")
        return dx, dw, db
