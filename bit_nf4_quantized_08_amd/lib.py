"""Thin Python binding of ``libqlora_nf4.so`` (argument marshalling only).

Every function here checks dtypes/devices/shapes of torch tensors, hands raw
device pointers, sizes and torch's current HIP stream to the C ABI declared in
``include/qlora_nf4.h``, and raises on a non-zero status.  All arithmetic runs
in the library's HIP kernels; there is no CPU or PyTorch fallback.

Names follow the C ABI: ``nf4_quantize``, ``nf4_double_quant``, ``nf4_dequant``,
``qlora_linear_fwd``, ``qlora_linear_bwd``, ``qn_codebook``; dropout on the
adapter's input (``Dropout``, ``dropout``, ``qlora_linear_fwd_dropout``,
``qlora_linear_bwd_dropout``); and the microscaled base (``mxfp4_quantize``,
``mxfp4_dequant``, ``qlora_mx_linear_fwd``, ``qlora_mx_linear_bwd``).
"""

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# QN_LIBRARY names another build of the same library (the host-sanitizer build
# that the ABI tests load in a child process); by default the in-tree one.
LIB_PATH = os.environ.get("QN_LIBRARY") or os.path.join(_PKG, "libqlora_nf4.so")

QN_OK = 0
QN_F32, QN_BF16 = 0, 1
QN_NF4, QN_FP4 = 0, 1
QUANT_TYPES = {"nf4": QN_NF4, "fp4": QN_FP4}
QN_OP_FWD, QN_OP_BWD, QN_OP_FWD_DROPOUT, QN_OP_BWD_DROPOUT = 0, 1, 2, 3
QN_ERR_SCRATCH = 8
QN_ERR_MEMORY = 9
QN_NOALLOC_SCRATCH_BYTES = 16 << 20
QN_BLOCK, QN_GROUP, QN_MAX_RANK, QN_MAX_GROUP = 64, 256, 64, 8
QN_ADAMW_MULTI = 32
QN_MX_BLOCK, QN_MX_CHUNK = 32, 256

_lib = None


class QNError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")


class NF4WeightStruct(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("absmax", ctypes.c_void_p),
        ("absmax_q", ctypes.c_void_p),
        ("scale2", ctypes.c_void_p),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("quant_type", ctypes.c_int32),
    ]


class FwdProblemStruct(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p),
        ("M", ctypes.c_int64),
        ("W", NF4WeightStruct),
        ("A", ctypes.c_void_p),
        ("B", ctypes.c_void_p),
        ("r", ctypes.c_int64),
        ("alpha", ctypes.c_float),
        ("Y", ctypes.c_void_p),
        ("H_out", ctypes.c_void_p),
    ]


class AdamWConfigStruct(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("step", ctypes.c_int64),
    ]


class AdamWTensorStruct(ctypes.Structure):
    """qn_adamw_tensor: one tensor of a multi-tensor step."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("m_q", ctypes.c_void_p), ("m_step", ctypes.c_void_p), ("u_q", ctypes.c_void_p),
                ("u_step", ctypes.c_void_p)]


class DropoutStruct(ctypes.Structure):
    """qn_dropout_config."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("offset_dev", ctypes.c_void_p)]


class MXMatrixStruct(ctypes.Structure):
    """qn_mx_matrix."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


def load():
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m bit_nf4_quantized_08_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    sig = {
        "qn_codebook": (i32, [ctypes.POINTER(ctypes.c_float)]),
        "qn_table": (i32, [i32, ctypes.POINTER(ctypes.c_float)]),
        "qn_quantize_4bit": (i32, [vp, i32, i64, i64, i32, vp, vp, vp, vp, vp]),
        "nf4_quantize": (i32, [vp, i32, i64, i64, vp, vp, vp]),
        "nf4_double_quant": (i32, [vp, i64, vp, vp, vp]),
        "nf4_dequant": (i32, [ctypes.POINTER(NF4WeightStruct), vp, i32, vp]),
        "qn_adamw8_step": (i32, [vp, vp, i64, vp, vp, vp, vp, ctypes.POINTER(AdamWConfigStruct), vp]),
        "qn_adamw8_step_multi": (i32, [i32, ctypes.POINTER(AdamWTensorStruct), ctypes.POINTER(AdamWConfigStruct), vp]),
        "qlora_merge": (i32, [ctypes.POINTER(NF4WeightStruct), vp, vp, i64, f32, vp, i32, vp]),
        "qlora_workspace_size": (ctypes.c_size_t, [i32, i64, i64, i64, i64]),
        "qlora_linear_fwd": (i32, [vp, i64, ctypes.POINTER(NF4WeightStruct), vp, vp, i64, f32, vp, vp, vp,
                                   ctypes.c_size_t, vp]),
        "qlora_workspace_size_grouped": (ctypes.c_size_t, [i32, ctypes.POINTER(FwdProblemStruct)]),
        "qlora_linear_fwd_grouped": (i32, [i32, ctypes.POINTER(FwdProblemStruct), vp, ctypes.c_size_t, vp]),
        "qlora_linear_fwd_noalloc": (i32, [vp, i64, ctypes.POINTER(NF4WeightStruct), vp, vp, i64, f32, vp, vp, vp]),
        "qlora_linear_bwd": (i32, [vp, vp, vp, i64, ctypes.POINTER(NF4WeightStruct), vp, vp, i64, f32, vp, vp,
                                   vp, vp, ctypes.c_size_t, vp]),
        "qn_dropout": (i32, [vp, i32, i64, ctypes.POINTER(DropoutStruct), vp, vp]),
        "qlora_linear_fwd_dropout": (i32, [vp, i64, ctypes.POINTER(NF4WeightStruct), vp, vp, i64, f32,
                                           ctypes.POINTER(DropoutStruct), vp, vp, vp, ctypes.c_size_t, vp]),
        "qlora_linear_bwd_dropout": (i32, [vp, vp, vp, i64, ctypes.POINTER(NF4WeightStruct), vp, vp, i64, f32,
                                           ctypes.POINTER(DropoutStruct), vp, vp, vp, vp, ctypes.c_size_t, vp]),
        "qn_mxfp4_quantize": (i32, [vp, i32, i64, i64, vp, vp, vp]),
        "qn_mxfp4_dequant": (i32, [ctypes.POINTER(MXMatrixStruct), vp, i32, vp]),
        "qlora_mx_workspace_size": (ctypes.c_size_t, [i32, i64, i64, i64, i64]),
        "qlora_mx_linear_fwd": (i32, [vp, i64, ctypes.POINTER(MXMatrixStruct), vp, vp, i64, f32,
                                      ctypes.POINTER(DropoutStruct), vp, vp, vp, ctypes.c_size_t, vp]),
        "qlora_mx_linear_bwd": (i32, [vp, vp, vp, i64, ctypes.POINTER(MXMatrixStruct), vp, vp, i64, f32,
                                      ctypes.POINTER(DropoutStruct), vp, vp, vp, vp, ctypes.c_size_t, vp]),
        "qn_status_string": (ctypes.c_char_p, [i32]),
        "qn_trace_enable": (i32, [i32]),
        "qn_set_gemm_variant": (i32, [i32]),
        "qn_trace_read": (i32, [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float), i32]),
        "qn_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def exported_symbols():
    return ["qn_codebook", "qn_table", "qn_quantize_4bit", "nf4_quantize", "nf4_double_quant", "nf4_dequant", "qlora_merge", "qn_adamw8_step", "qn_adamw8_step_multi",
            "qlora_workspace_size",
            "qlora_linear_fwd", "qlora_linear_fwd_noalloc", "qlora_workspace_size_grouped",
            "qlora_linear_fwd_grouped", "qlora_linear_bwd", "qn_status_string", "qn_version", "qn_set_gemm_variant", "qn_trace_enable",
            "qn_trace_read", "qn_dropout", "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout", "qn_mxfp4_quantize",
            "qn_mxfp4_dequant", "qlora_mx_workspace_size", "qlora_mx_linear_fwd", "qlora_mx_linear_bwd"]


def status_string(status):
    return load().qn_status_string(int(status)).decode()


def _check(fn, status):
    if status != QN_OK:
        raise QNError(fn, status)


def qn_codebook():
    """The library's NF4 table (host call, no device work): numpy float32[16]."""
    out = (ctypes.c_float * 16)()
    _check("qn_codebook", load().qn_codebook(out))
    return np.frombuffer(out, dtype=np.float32).copy()


def qn_table(quant_type="nf4"):
    """The library's table of a 4-bit type ("nf4" or "fp4"), by code: numpy float32[16]."""
    out = (ctypes.c_float * 16)()
    _check("qn_table", load().qn_table(QUANT_TYPES[quant_type], out))
    return np.frombuffer(out, dtype=np.float32).copy()


# ------------------------------------------------------------------ torch glue
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream():
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, name, dtype=None, ndim=None, device_cuda=True):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device_cuda and t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got {t.dim()}-D")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@dataclass
class NF4Weight:
    """A frozen weight W[N, K] in NF4 form (device tensors)."""
    codes: "object"                 # uint8 [ceil(N*K/2)]
    absmax: Optional[object]        # fp32 [nb] (kept after double quantisation too)
    absmax_q: Optional[object]      # uint8 [nb] or None
    scale2: Optional[object]        # fp32 [ceil(nb/256)] or None
    N: int
    K: int
    quant_type: int = QN_NF4        # QN_NF4 or QN_FP4: the table the codes index

    def struct(self, use_double_quant=True):
        dq = use_double_quant and self.absmax_q is not None
        return NF4WeightStruct(
            self.codes.data_ptr(),
            self.absmax.data_ptr() if (self.absmax is not None and not dq) else 0,
            self.absmax_q.data_ptr() if dq else 0,
            self.scale2.data_ptr() if dq else 0,
            self.N, self.K, self.quant_type)


def nf4_quantize(W, codes=None, absmax=None):
    """Blockwise NF4 quantisation of a 2-D fp32 or bf16 device tensor."""
    torch = _torch()
    _need(W, "W", ndim=2)
    if W.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("W must be float32 or bfloat16")
    N, K = W.shape
    n = N * K
    if codes is None:
        codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=W.device)
    if absmax is None:
        absmax = torch.empty((n + 63) // 64, dtype=torch.float32, device=W.device)
    dt = QN_BF16 if W.dtype == torch.bfloat16 else QN_F32
    _check("nf4_quantize", load().nf4_quantize(_ptr(W), dt, N, K, _ptr(codes), _ptr(absmax), _stream()))
    return codes, absmax


def nf4_double_quant(absmax, absmax_q=None, scale2=None):
    torch = _torch()
    _need(absmax, "absmax", dtype=torch.float32, ndim=1)
    nb = absmax.numel()
    if absmax_q is None:
        absmax_q = torch.empty(nb, dtype=torch.uint8, device=absmax.device)
    if scale2 is None:
        scale2 = torch.empty((nb + 255) // 256, dtype=torch.float32, device=absmax.device)
    _check("nf4_double_quant", load().nf4_double_quant(_ptr(absmax), nb, _ptr(absmax_q), _ptr(scale2), _stream()))
    return absmax_q, scale2


def quantize_4bit(W, quant_type="nf4", codes=None, absmax=None, absmax_q=None, scale2=None, double_quant=True):
    """qn_quantize_4bit: blockwise 4-bit quantisation of a 2-D fp32 or bf16 device
    tensor, with the block scales double-quantised in the same launch when
    ``double_quant``.  Returns an NF4Weight (absmax kept either way)."""
    torch = _torch()
    _need(W, "W", ndim=2)
    if W.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("W must be float32 or bfloat16")
    N, K = W.shape
    n = N * K
    nb = (n + 63) // 64
    if codes is None:
        codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=W.device)
    if absmax is None:
        absmax = torch.empty(nb, dtype=torch.float32, device=W.device)
    if double_quant:
        if absmax_q is None:
            absmax_q = torch.empty(nb, dtype=torch.uint8, device=W.device)
        if scale2 is None:
            scale2 = torch.empty((nb + 255) // 256, dtype=torch.float32, device=W.device)
    else:
        absmax_q = scale2 = None
    dt = QN_BF16 if W.dtype == torch.bfloat16 else QN_F32
    qt = QUANT_TYPES[quant_type]
    _check("qn_quantize_4bit", load().qn_quantize_4bit(_ptr(W), dt, N, K, qt, _ptr(codes), _ptr(absmax),
                                                       _ptr(absmax_q), _ptr(scale2), _stream()))
    return NF4Weight(codes, absmax, absmax_q, scale2, int(N), int(K), qt)


def quantize_weight(W, double_quant=True, quant_type="nf4", fused=True):
    """W (2-D device tensor) -> NF4Weight, optionally double-quantised: by default
    in one launch (qn_quantize_4bit); ``fused=False`` (NF4 only) runs
    nf4_quantize and then nf4_double_quant."""
    if fused or quant_type != "nf4":
        return quantize_4bit(W, quant_type, double_quant=double_quant)
    codes, absmax = nf4_quantize(W)
    aq = s2 = None
    if double_quant:
        aq, s2 = nf4_double_quant(absmax)
    return NF4Weight(codes, absmax, aq, s2, int(W.shape[0]), int(W.shape[1]))


def nf4_dequant(w: NF4Weight, out_dtype="bf16", use_double_quant=True, out=None):
    torch = _torch()
    dt = {"bf16": (QN_BF16, torch.bfloat16), "f32": (QN_F32, torch.float32)}[out_dtype]
    if out is None:
        out = torch.empty((w.N, w.K), dtype=dt[1], device=w.codes.device)
    st = w.struct(use_double_quant)
    _check("nf4_dequant", load().nf4_dequant(ctypes.byref(st), _ptr(out), dt[0], _stream()))
    return out


def qlora_merge(w: NF4Weight, A, B, alpha, out_dtype="bf16", use_double_quant=True, out=None):
    """The adapter merged into the dequantised base: [N, K] bf16 (or fp32)."""
    torch = _torch()
    _need(A, "A", torch.bfloat16, 2)
    _need(B, "B", torch.bfloat16, 2)
    r = A.shape[0]
    if A.shape[1] != w.K or B.shape != (w.N, r):
        raise ValueError("A must be [r, K] and B [N, r]")
    dt = {"bf16": (QN_BF16, torch.bfloat16), "f32": (QN_F32, torch.float32)}[out_dtype]
    if out is None:
        out = torch.empty((w.N, w.K), dtype=dt[1], device=w.codes.device)
    st = w.struct(use_double_quant)
    _check("qlora_merge", load().qlora_merge(ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha), _ptr(out), dt[0],
                                             _stream()))
    return out


class AdamW8State:
    """8-bit block-wise AdamW state of one bf16 tensor (zeros: before the first step).

    host=True places the state in pinned host memory mapped for the device
    (the "paged" placement: none of its bytes occupy device memory, and the
    step reads and writes it across the host link)."""

    def __init__(self, n, device="cuda", host=False):
        torch = _torch()
        nb = (n + 63) // 64
        self.n = n
        self.host = bool(host)
        kw = dict(device="cpu", pin_memory=True) if self.host else dict(device=device)
        self.m_q = torch.zeros(n, dtype=torch.int8, **kw)
        self.m_step = torch.zeros(nb, dtype=torch.float32, **kw)
        self.u_q = torch.zeros(n, dtype=torch.uint8, **kw)
        self.u_step = torch.zeros(nb, dtype=torch.float32, **kw)
        self.step = 0


def adamw8_step(param, grad, state: AdamW8State, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                step=None):
    """One qn_adamw8_step on a bf16 tensor in place; advances state.step
    unless an explicit step number is given."""
    torch = _torch()
    _need(param, "param", torch.bfloat16)
    _need(grad, "grad", torch.bfloat16)
    if param.numel() != state.n or grad.numel() != state.n:
        raise ValueError("param, grad and state sizes differ")
    if step is None:
        state.step += 1
        step = state.step
    cfg = AdamWConfigStruct(lr, beta1, beta2, eps, weight_decay, int(step))
    _check("qn_adamw8_step", load().qn_adamw8_step(
        _ptr(param), _ptr(grad), state.n, _ptr(state.m_q), _ptr(state.m_step), _ptr(state.u_q), _ptr(state.u_step),
        ctypes.byref(cfg), _stream()))
    return param


def adamw8_step_multi(params, grads, states, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                      step=None):
    """One qn_adamw8_step_multi over several bf16 tensors in place (one launch
    per QN_ADAMW_MULTI tensors); all states advance to the same step unless an
    explicit step number is given."""
    torch = _torch()
    if not (len(params) == len(grads) == len(states)) or not params:
        raise ValueError("params, grads and states must be non-empty lists of one length")
    arr = (AdamWTensorStruct * len(params))()
    for i, (p, g, st) in enumerate(zip(params, grads, states)):
        _need(p, "param", torch.bfloat16)
        _need(g, "grad", torch.bfloat16)
        if p.numel() != st.n or g.numel() != st.n:
            raise ValueError("param, grad and state sizes differ")
        arr[i] = AdamWTensorStruct(_ptr(p), _ptr(g), st.n, _ptr(st.m_q), _ptr(st.m_step), _ptr(st.u_q),
                                   _ptr(st.u_step))
    if step is None:
        step = states[0].step + 1
    for st in states:
        st.step = int(step)
    cfg = AdamWConfigStruct(lr, beta1, beta2, eps, weight_decay, int(step))
    _check("qn_adamw8_step_multi", load().qn_adamw8_step_multi(len(params), arr, ctypes.byref(cfg), _stream()))
    return params


def workspace_size(op, M, N, K, r):
    return int(load().qlora_workspace_size(op, M, N, K, r))


def workspace(op, M, N, K, r, device="cuda"):
    torch = _torch()
    nbytes = workspace_size(op, M, N, K, r)
    if nbytes == 0:
        raise QNError("qlora_workspace_size", 2)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def qlora_linear_fwd(X, w: NF4Weight, A, B, alpha, want_H=False, use_double_quant=True, Y=None, ws=None, H=None):
    """Y = X bf16(dequant(W))^T + (alpha/r) (X A^T) B^T; returns Y (and H).

    ``H`` (optional, fp32 [M, r]) receives X A^T; passing it implies want_H."""
    torch = _torch()
    _need(X, "X", torch.bfloat16, 2)
    _need(A, "A", torch.bfloat16, 2)
    _need(B, "B", torch.bfloat16, 2)
    M, K = X.shape
    r = A.shape[0]
    if K != w.K or A.shape[1] != w.K or B.shape != (w.N, r):
        raise ValueError("shape mismatch between X, W, A, B")
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=X.device)
    _need(Y, "Y", torch.bfloat16, 2)
    if Y.shape != (M, w.N):
        raise ValueError("Y must be [M, N]")
    if H is not None:
        _need(H, "H", torch.float32, 2)
        if H.shape != (M, r):
            raise ValueError("H must be [M, r]")
        want_H = True
    elif want_H:
        H = torch.empty((M, r), dtype=torch.float32, device=X.device)
    if ws is None:
        ws = workspace(QN_OP_FWD, M, w.N, w.K, r, X.device)
    st = w.struct(use_double_quant)
    _check("qlora_linear_fwd", load().qlora_linear_fwd(
        _ptr(X), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha), _ptr(Y), _ptr(H),
        _ptr(ws), ws.numel(), _stream()))
    return (Y, H) if want_H else Y


class FwdGroup:
    """A fixed set of independent forwards for qlora_linear_fwd_grouped.

    ``problems`` is a list of (X, w, A, B, alpha, Y, H) with H optional (None);
    the descriptor array and the workspace are built once, so that run() only
    enqueues (and can be captured into a HIP graph)."""

    def __init__(self, problems, use_double_quant=True, ws=None):
        torch = _torch()
        n = len(problems)
        if not 1 <= n <= QN_MAX_GROUP:
            raise ValueError(f"1 to {QN_MAX_GROUP} problems per group")
        self._keep = problems
        arr = (FwdProblemStruct * n)()
        for i, (X, w, A, B, alpha, Y, H) in enumerate(problems):
            _need(X, "X", torch.bfloat16, 2)
            _need(A, "A", torch.bfloat16, 2)
            _need(B, "B", torch.bfloat16, 2)
            _need(Y, "Y", torch.bfloat16, 2)
            M, K = X.shape
            r = A.shape[0]
            if K != w.K or A.shape[1] != w.K or B.shape != (w.N, r) or Y.shape != (M, w.N):
                raise ValueError(f"problem {i}: shape mismatch between X, W, A, B, Y")
            if H is not None:
                _need(H, "H", torch.float32, 2)
                if H.shape != (M, r):
                    raise ValueError(f"problem {i}: H must be [M, r]")
            arr[i] = FwdProblemStruct(X.data_ptr(), M, w.struct(use_double_quant), A.data_ptr(), B.data_ptr(), r,
                                      float(alpha), Y.data_ptr(), H.data_ptr() if H is not None else 0)
        self._arr, self._n = arr, n
        nbytes = int(load().qlora_workspace_size_grouped(n, arr))
        if nbytes == 0:
            raise QNError("qlora_workspace_size_grouped", 2)
        self.ws = ws if ws is not None else torch.empty(nbytes, dtype=torch.uint8, device=problems[0][0].device)

    def run(self):
        _check("qlora_linear_fwd_grouped", load().qlora_linear_fwd_grouped(
            self._n, self._arr, _ptr(self.ws), self.ws.numel(), _stream()))


def qlora_linear_fwd_grouped(problems, use_double_quant=True):
    """Run independent forwards [(X, w, A, B, alpha, Y, H or None), ...] in one call."""
    FwdGroup(problems, use_double_quant).run()


def qlora_linear_fwd_noalloc(X, w: NF4Weight, A, B, alpha, Y, H=None, use_double_quant=True):
    """qlora_linear_fwd without a workspace: the library's static scratch array
    is the workspace.  Y (and H) are caller-provided; nothing is allocated."""
    torch = _torch()
    _need(X, "X", torch.bfloat16, 2)
    _need(A, "A", torch.bfloat16, 2)
    _need(B, "B", torch.bfloat16, 2)
    _need(Y, "Y", torch.bfloat16, 2)
    M, K = X.shape
    r = A.shape[0]
    if K != w.K or A.shape[1] != w.K or B.shape != (w.N, r) or Y.shape != (M, w.N):
        raise ValueError("shape mismatch between X, W, A, B, Y")
    if H is not None:
        _need(H, "H", torch.float32, 2)
        if H.shape != (M, r):
            raise ValueError("H must be [M, r]")
    st = w.struct(use_double_quant)
    _check("qlora_linear_fwd_noalloc", load().qlora_linear_fwd_noalloc(
        _ptr(X), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha), _ptr(Y), _ptr(H), _stream()))
    return Y


def qlora_linear_bwd(dY, X, w: NF4Weight, A, B, alpha, want_dX=True, use_double_quant=True, out=None, ws=None,
                     H=None):
    """Returns (dX or None, dA, dB) for the upstream gradient dY.

    ``H`` (optional, fp32 [M, r]) is X A^T as the forward returned it with
    ``want_H=True``; given, the call does not recompute it from X."""
    torch = _torch()
    _need(dY, "dY", torch.bfloat16, 2)
    _need(X, "X", torch.bfloat16, 2)
    _need(A, "A", torch.bfloat16, 2)
    _need(B, "B", torch.bfloat16, 2)
    M, K = X.shape
    r = A.shape[0]
    if dY.shape != (M, w.N) or K != w.K or A.shape[1] != w.K or B.shape != (w.N, r):
        raise ValueError("shape mismatch between dY, X, W, A, B")
    if H is not None:
        _need(H, "H", torch.float32, 2)
        if H.shape != (M, r):
            raise ValueError("H must be [M, r]")
    if out is None:
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=X.device) if want_dX else None
        dA = torch.empty((r, K), dtype=torch.bfloat16, device=X.device)
        dB = torch.empty((w.N, r), dtype=torch.bfloat16, device=X.device)
    else:
        dX, dA, dB = out
    if ws is None:
        ws = workspace(QN_OP_BWD, M, w.N, w.K, r, X.device)
    st = w.struct(use_double_quant)
    _check("qlora_linear_bwd", load().qlora_linear_bwd(
        _ptr(dY), _ptr(X), _ptr(H), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha), _ptr(dX), _ptr(dA),
        _ptr(dB), _ptr(ws), ws.numel(), _stream()))
    return dX, dA, dB


# ------------------------------------------------- dropout and the MXFP4 base
def _operand(t, name, dtype, shape=None):
    """Check a GPU operand (type, contiguity, shape); its address.  The quick test
    comes first: these calls are short, and a full report is made only to raise."""
    if not (getattr(t, "is_cuda", False) and t.dtype == dtype and t.is_contiguous()):
        _need(t, name, dtype)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _launch(tensors, fn, *args):
    """Call fn(*args, stream) on the current stream of the one GPU that all the
    tensors (None skipped) lie on."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if dev is not None:
                    raise ValueError(f"tensors on different devices: cuda:{dev} and {t.device}")
                dev = d
    call = getattr(_lib or load(), fn)
    device, stream = _cuda_lookups or _find_lookups()
    if dev == device():
        _check(fn, call(*args, stream(dev)))
    else:
        with _torch().cuda.device(dev):
            _check(fn, call(*args, stream(dev)))


_cuda_lookups = None   # (current device, hipStream_t of a device's current stream)


def _find_lookups():
    """torch's own lookups where it has them: without the initialisation check of
    torch.cuda.current_device and the Stream object of torch.cuda.current_stream
    (a GPU tensor is at hand, so the runtime is up)."""
    global _cuda_lookups
    torch = _torch()
    _cuda_lookups = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                     getattr(torch._C, "_cuda_getCurrentRawStream",
                             lambda dev: torch.cuda.current_stream(dev).cuda_stream))
    return _cuda_lookups


@dataclass
class Dropout:
    """qn_dropout_config: probability, seed, and the offset that picks the mask
    within a seed.  ``offset_dev`` (optional, a one-element int64 GPU tensor) is
    added to the offset when the kernels run: advance it between the replays of
    a captured graph, and keep it unchanged from a forward to its backward."""
    p: float
    seed: int
    offset: int = 0
    offset_dev: Optional[object] = None

    def struct(self):
        seed, offset, dev = int(self.seed), int(self.offset), 0
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be in [0, 2^64)")
        if not 0 <= offset < 1 << 64:
            raise ValueError("offset must be in [0, 2^64)")
        if self.offset_dev is not None:
            dev = _operand(self.offset_dev, "offset_dev", _torch().int64)
            if self.offset_dev.numel() != 1:
                raise ValueError("offset_dev must hold one element")
        return DropoutStruct(float(self.p), seed, offset, dev)


def _need_drop(drop):
    if drop is None:
        raise ValueError("drop is required (p = 0 drops nothing)")


def _drop_ref(drop):
    return ctypes.byref(drop.struct()) if drop is not None else None


def dropout(x, drop: Dropout, out=None):
    """qn_dropout of a contiguous fp32 or bf16 tensor of any shape; ``out`` may be
    ``x``.  Applied to a gradient with the same ``drop`` it is the backward."""
    _need_drop(drop)
    px, dt = _codec_operand(x, "x")
    if out is None:
        out = _torch().empty_like(x)
    po = _operand(out, "out", x.dtype, x.shape)
    _launch((x, out, drop.offset_dev), "qn_dropout", px, dt, x.numel(), _drop_ref(drop), po)
    return out


_codec_types = {}   # torch type -> QN type


def _codec_operand(t, name, shape=None):
    """Check an fp32 or bf16 operand; (its address, its QN type)."""
    if not _codec_types:
        torch = _torch()
        _codec_types.update({torch.bfloat16: QN_BF16, torch.float32: QN_F32})
    dt = _codec_types.get(getattr(t, "dtype", None))
    if dt is None:
        _need(t, name)
        raise ValueError(f"{name} must be float32 or bfloat16")
    return _operand(t, name, t.dtype, shape), dt


@dataclass
class MXMatrix:
    """A matrix [rows, cols] in MXFP4 form (device tensors)."""
    codes: "object"                 # uint8 [rows, 128 C], C = ceil(cols / 256)
    scales: "object"                # uint8 [C, rows, 8]
    rows: int
    cols: int

    @staticmethod
    def empty(rows, cols, device="cuda"):
        """Storage of a matrix, not yet written (mxfp4_quantize's ``out``)."""
        torch = _torch()
        C = -(-cols // QN_MX_CHUNK)
        return MXMatrix(torch.empty((rows, 128 * C), dtype=torch.uint8, device=device),
                        torch.empty((C, rows, 8), dtype=torch.uint8, device=device), int(rows), int(cols))

    @property
    def N(self):
        return self.rows

    @property
    def K(self):
        return self.cols

    def addresses(self):
        """Check the tensors; the addresses of codes and scales."""
        u8 = _torch().uint8
        C = -(-self.cols // QN_MX_CHUNK)
        return (_operand(self.codes, "codes", u8, (self.rows, 128 * C)),
                _operand(self.scales, "scales", u8, (C, self.rows, 8)))

    def struct(self):
        return MXMatrixStruct(*self.addresses(), self.rows, self.cols)


def mxfp4_quantize(X, out: Optional[MXMatrix] = None):
    """qn_mxfp4_quantize of a 2-D fp32 or bf16 device tensor -> MXMatrix."""
    px, dt = _codec_operand(X, "X")
    if X.dim() != 2:
        _need(X, "X", ndim=2)
    rows, cols = X.shape
    if out is None:
        out = MXMatrix.empty(rows, cols, X.device)
    if out.rows != rows or out.cols != cols:
        raise ValueError("out must have X's shape")
    codes, scales = out.addresses()
    _launch((X, out.codes, out.scales), "qn_mxfp4_quantize", px, dt, rows, cols, codes, scales)
    return out


def mxfp4_dequant(w: MXMatrix, out_dtype="bf16", out=None):
    """The values an MXMatrix stands for, [rows, cols] bf16 (or fp32); a given
    ``out`` decides the type."""
    st = w.struct()
    if out is None:
        torch = _torch()
        out = torch.empty((w.rows, w.cols), dtype={"bf16": torch.bfloat16, "f32": torch.float32}[out_dtype],
                          device=w.codes.device)
    po, dt = _codec_operand(out, "out", (w.rows, w.cols))
    _launch((w.codes, w.scales, out), "qn_mxfp4_dequant", ctypes.byref(st), po, dt)
    return out


def mx_workspace_size(op, M, N, K, r):
    return int(load().qlora_mx_workspace_size(op, M, N, K, r))


def mx_workspace(op, M, N, K, r, device="cuda"):
    """Workspace of the MXFP4 linear for op QN_OP_FWD or QN_OP_BWD (r = 0: no adapter)."""
    torch = _torch()
    nbytes = mx_workspace_size(op, M, N, K, r)
    if nbytes == 0:
        raise QNError("qlora_mx_workspace_size", 2)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _addr(t):
    return t.data_ptr() if t is not None else 0


def _linear_args(X, w, A, B, H, other, name):
    """Check a linear's operands; (M, r).  A and B are both None for r = 0."""
    bf = _torch().bfloat16
    _need(X, "X", bf, 2)
    M, K = X.shape
    if K != w.K:
        raise ValueError("X must be [M, K]")
    if (A is None) != (B is None):
        raise ValueError("A and B go together")
    r = 0
    if A is not None:
        r = A.shape[0]
        _operand(A, "A", bf, (r, K))
        _operand(B, "B", bf, (w.N, r))
    if other is not None:
        _operand(other, name, bf, (M, w.N))
    if H is not None:
        if r == 0:
            raise ValueError("H needs an adapter")
        _operand(H, "H", _torch().float32, (M, r))
    return int(M), int(r)


def _outputs(X, w, M, r, Y, H, want_H):
    """A forward's (Y, H), allocated where not given; H None unless wanted."""
    torch = _torch()
    if Y is None:
        Y = torch.empty((M, w.N), dtype=torch.bfloat16, device=X.device)
    if want_H and H is None:
        if r == 0:
            raise ValueError("H needs an adapter")
        H = torch.empty((M, r), dtype=torch.float32, device=X.device)
    return Y, H


def _grads(out, want_dX, X, w, M, r):
    """The gradients' tensors (dX, dA, dB), checked or allocated."""
    torch = _torch()
    bf = torch.bfloat16
    shapes = ((M, w.K), (r, w.K), (w.N, r))
    if out is None:
        new = [torch.empty(s, dtype=bf, device=X.device) for s in shapes[:3 if r else 1]]
        return (new[0] if want_dX else None,) + (tuple(new[1:]) if r else (None, None))
    for t, name, shape in zip(out, ("dX", "dA", "dB"), shapes):
        if t is not None:
            _operand(t, name, bf, shape)
        elif name != "dX" and r:
            raise ValueError(f"{name} is required")
    return tuple(out)


def qlora_linear_fwd_dropout(X, w: NF4Weight, A, B, alpha, drop: Dropout, want_H=False, use_double_quant=True, Y=None,
                             ws=None, H=None):
    """qlora_linear_fwd with dropout on the adapter's input: H = c (keep * X) A^T,
    Y = X bf16(dequant(W))^T + (alpha/r) H B^T.  The workspace is
    ``workspace(QN_OP_FWD_DROPOUT, ...)``."""
    _need_drop(drop)
    if A is None or B is None:
        raise ValueError("A and B are required")
    M, r = _linear_args(X, w, A, B, H, Y, "Y")
    Y, H = _outputs(X, w, M, r, Y, H, want_H)
    if ws is None:
        ws = workspace(QN_OP_FWD_DROPOUT, M, w.N, w.K, r, X.device)
    pw = _operand(ws, "ws", _torch().uint8)
    st = w.struct(use_double_quant)
    _launch((X, A, B, Y, H, ws, w.codes, w.absmax, w.absmax_q, w.scale2, drop.offset_dev),
            "qlora_linear_fwd_dropout", X.data_ptr(), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(), r, float(alpha),
            _drop_ref(drop), Y.data_ptr(), _addr(H), pw, ws.numel())
    return Y if H is None else (Y, H)


def qlora_linear_bwd_dropout(dY, X, w: NF4Weight, A, B, alpha, drop: Dropout, want_dX=True, use_double_quant=True,
                             out=None, ws=None, H=None):
    """Backward of qlora_linear_fwd_dropout: (dX or None, dA, dB).  ``H`` is the
    (dropped) one that forward returned, or None to form it again.  The workspace
    is ``workspace(QN_OP_BWD_DROPOUT, ...)``; that of QN_OP_BWD does, slower where
    dX's contraction would be cut."""
    _need_drop(drop)
    if A is None or B is None:
        raise ValueError("A and B are required")
    if dY is None:
        raise ValueError("dY is required")
    M, r = _linear_args(X, w, A, B, H, dY, "dY")
    dX, dA, dB = _grads(out, want_dX, X, w, M, r)
    if ws is None:
        ws = workspace(QN_OP_BWD_DROPOUT, M, w.N, w.K, r, X.device)
    pw = _operand(ws, "ws", _torch().uint8)
    st = w.struct(use_double_quant)
    _launch((dY, X, A, B, H, ws, dX, dA, dB, w.codes, w.absmax, w.absmax_q, w.scale2, drop.offset_dev),
            "qlora_linear_bwd_dropout", dY.data_ptr(), X.data_ptr(), _addr(H), M, ctypes.byref(st), A.data_ptr(),
            B.data_ptr(), r, float(alpha), _drop_ref(drop), _addr(dX), dA.data_ptr(), dB.data_ptr(), pw, ws.numel())
    return dX, dA, dB


def qlora_mx_linear_fwd(X, w: MXMatrix, A=None, B=None, alpha=0.0, drop: Optional[Dropout] = None, want_H=False,
                        Y=None, ws=None, H=None):
    """Y = mx(X) W^T + (alpha/r) H B^T over an MXFP4 base, H = c (keep * X) A^T;
    returns Y (and H).  A = B = None: the base alone."""
    M, r = _linear_args(X, w, A, B, H, Y, "Y")
    Y, H = _outputs(X, w, M, r, Y, H, want_H)
    if ws is None:
        ws = mx_workspace(QN_OP_FWD, M, w.N, w.K, r, X.device)
    pw = _operand(ws, "ws", _torch().uint8)
    st = w.struct()
    _launch((X, A, B, Y, H, ws, w.codes, w.scales, drop.offset_dev if drop is not None else None),
            "qlora_mx_linear_fwd", X.data_ptr(), M, ctypes.byref(st), _addr(A), _addr(B), r, float(alpha),
            _drop_ref(drop), Y.data_ptr(), _addr(H), pw, ws.numel())
    return Y if H is None else (Y, H)


def qlora_mx_linear_bwd(dY, X, w: MXMatrix, A=None, B=None, alpha=0.0, drop: Optional[Dropout] = None, want_dX=True,
                        out=None, ws=None, H=None):
    """Backward of qlora_mx_linear_fwd: (dX or None, dA, dB); dA and dB are None
    without an adapter."""
    if dY is None:
        raise ValueError("dY is required")
    M, r = _linear_args(X, w, A, B, H, dY, "dY")
    dX, dA, dB = _grads(out, want_dX, X, w, M, r)
    if ws is None:
        ws = mx_workspace(QN_OP_BWD, M, w.N, w.K, r, X.device)
    pw = _operand(ws, "ws", _torch().uint8)
    st = w.struct()
    _launch((dY, X, A, B, H, ws, dX, dA, dB, w.codes, w.scales, drop.offset_dev if drop is not None else None),
            "qlora_mx_linear_bwd", dY.data_ptr(), X.data_ptr(), _addr(H), M, ctypes.byref(st), _addr(A), _addr(B), r,
            float(alpha), _drop_ref(drop), _addr(dX), _addr(dA), _addr(dB), pw, ws.numel())
    return dX, dA, dB


TRACE_KINDS = {1: "quantize", 2: "double_quant", 3: "dequant", 4: "gemv", 5: "gemm_fwd", 6: "gemm_dx",
               7: "gemm_db", 8: "gemm_da", 9: "lowrank", 10: "merge", 11: "adamw8", 12: "dropout",
               13: "mx_quantize", 14: "mx_dequant", 15: "mx_gemv", 16: "mx_gemm", 17: "mx_dx"}


def set_gemm_variant(variant):
    """Forward dequant-GEMM tiling for later calls: 0 automatic, 1 256x128, 2 256x256."""
    _check("qn_set_gemm_variant", load().qn_set_gemm_variant(int(variant)))


def trace_enable(on=True):
    _check("qn_trace_enable", load().qn_trace_enable(1 if on else 0))


def trace_read(cap=1 << 16):
    """Wait for the logged kernels; returns a list of (kind name, milliseconds)."""
    kinds = (ctypes.c_int * cap)()
    ms = (ctypes.c_float * cap)()
    n = load().qn_trace_read(kinds, ms, cap)
    if n < 0:
        raise QNError("qn_trace_read", -n)
    return [(TRACE_KINDS.get(kinds[i], str(kinds[i])), float(ms[i])) for i in range(n)]


def raw():
    """The ctypes library object (for callers passing raw pointers)."""
    return load()
