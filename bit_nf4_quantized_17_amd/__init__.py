"""MI355X (gfx950) QLoRA NF4 linear layer -- Python binding of libqlora_nf4.

Argument marshalling only: every step of the layer runs in the HIP kernels of
``libqlora_nf4.so`` behind the C ABI of ``include/qlora_nf4.h``.  PyTorch is
used for device memory and the current HIP stream.  There is no fallback: if
the library is missing or fails to load, every call raises.

Functions keep the C ABI's names:
  nf4_levels, nf4_storage_bytes, nf4_quantize, nf4_dequantize,
  qlora_fwd_workspace_bytes, qlora_linear_fwd,
  qlora_bwd_workspace_bytes, qlora_linear_bwd, qlora_linear_bwd_noalloc,
  qlora_multi_fwd, qlora_multi_bwd, qlora_multi_plan, qlora_adamw8_step,
  qlora_abi_version
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import importlib
import os
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqlora_nf4.so")

QL_DTYPE_BF16 = 1
QL_CODEBOOK_NF4 = 0
QL_CODEBOOK_INT4 = 1
CODEBOOKS = {"nf4": QL_CODEBOOK_NF4, "int4": QL_CODEBOOK_INT4}
QL_DQ_E4M3 = 0
QL_DQ_UINT8 = 1
DQ_FORMATS = {"e4m3": QL_DQ_E4M3, "uint8": QL_DQ_UINT8}
QL_DUAL_SEPARATE = 1
QL_DUAL_SWIGLU = 2
QLORA_MAX_RANK = 128
QLORA_MAX_ADAPTERS = 32768
QLORA_BWD_NOALLOC_MAX_BYTES = 32 << 20
_STATUS = {0: "QL_OK", -1: "QL_ERR_NULL", -2: "QL_ERR_SHAPE", -3: "QL_ERR_UNSUPPORTED",
           -4: "QL_ERR_ALIGN", -5: "QL_ERR_WORKSPACE", -6: "QL_ERR_HIP"}

_lib = None
_native_mod = None


class QLoRAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class _AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("master", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class _Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("qscale", ctypes.c_void_p),
                ("dscale", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("block", ctypes.c_int32), ("dq_block", ctypes.c_int32), ("codebook", ctypes.c_int32),
                ("dq_format", ctypes.c_int32)]


def lib() -> ctypes.CDLL:
    """Load libqlora_nf4.so (built by build.py); raises if it is not there."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run python -m bit_nf4_quantized_17_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    WP = ctypes.POINTER(_Weight)
    L.qlora_abi_version.argtypes, L.qlora_abi_version.restype = [], I
    L.qlora_last_error.argtypes, L.qlora_last_error.restype = [], ctypes.c_char_p
    L.nf4_levels.argtypes, L.nf4_levels.restype = [P], None
    L.nf4_storage_bytes.argtypes = [I64, I64, I, I, P, P, P]
    L.nf4_storage_bytes.restype = I
    L.nf4_quantize.argtypes = [P, I64, I64, I, I, P, P, P, P, P]
    L.nf4_quantize.restype = I
    L.qlora_quantize.argtypes = [P, I64, I64, I, I, I, P, P, P, P, P]
    L.qlora_quantize.restype = I
    L.qlora_codebook_levels.argtypes = [I, P]
    L.qlora_codebook_levels.restype = I
    L.nf4_dequantize.argtypes = [WP, P, P]
    L.nf4_dequantize.restype = I
    L.qlora_fwd_workspace_bytes.argtypes = [I64, I64, I64, I]
    L.qlora_fwd_workspace_bytes.restype = SZ
    L.qlora_linear_fwd.argtypes = [WP, P, I64, P, P, I, F, I, P, P, P, SZ, P]
    L.qlora_linear_fwd.restype = I
    L.qlora_dual_fwd.argtypes = [WP, WP, P, I64, P, P, P, P, I, F, I, I, P, P, P, P, P, P, SZ, P]
    L.qlora_dual_fwd.restype = I
    L.qlora_adamw_step.argtypes = [P, I, F, F, F, F, F, I, P]
    L.qlora_adamw_step.restype = I
    D = ctypes.c_double
    L.qlora_adamw8_step.argtypes = [P, I, D, D, D, D, D, I64, ctypes.c_uint32, P]
    L.qlora_adamw8_step.restype = I
    # (the many-adapter calls take their descriptors as packed bytes)
    for f in (L.qlora_multi_fwd_workspace_bytes, L.qlora_multi_bwd_workspace_bytes):
        f.argtypes, f.restype = [I64, I64, I64, I, I], SZ
    L.qlora_multi_fwd.argtypes = [P, P, I64, P, P, I, P, P, P, SZ, P]
    L.qlora_multi_fwd.restype = I
    L.qlora_multi_bwd.argtypes = [P, P, P, I64, P, P, I, P, P, P, P, P, SZ, P]
    L.qlora_multi_bwd.restype = I
    L.qlora_multi_plan.argtypes = [WP, I64, I, I, ctypes.POINTER(ctypes.c_int * 3)]
    L.qlora_multi_plan.restype = I
    L.qlora_bwd_workspace_bytes.argtypes = [I64, I64, I64, I]
    L.qlora_bwd_workspace_bytes.restype = SZ
    L.qlora_linear_bwd.argtypes = [WP, P, P, I64, P, P, I, F, I, P, P, P, P, P, SZ, P]
    L.qlora_linear_bwd.restype = I
    L.qlora_linear_bwd_noalloc.argtypes = [WP, P, P, I64, P, P, I, F, I, P, P, P, P, P]
    L.qlora_linear_bwd_noalloc.restype = I
    L.qlora_merge.argtypes = [WP, P, P, I, F, P, P]
    L.qlora_merge.restype = I
    L.qlora_unmerge.argtypes = [P, I64, I64, P, P, I, F, P, P]
    L.qlora_unmerge.restype = I
    L.qlora_set_timing_events.argtypes = [P, P, P, P]
    L.qlora_set_timing_events.restype = I
    _lib = L
    return L


def _native():
    """The native argument marshalling (built by build.py); raises if it is not there."""
    global _native_mod
    if _native_mod is None:
        import torch  # noqa: F401  (its libraries hold the symbols the module links to)
        _native_mod = importlib.import_module("._marshal", __name__)
    return _native_mod


def _check(rc: int):
    if rc != 0:
        raise QLoRAError(rc, lib().qlora_last_error().decode())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t, dtype, shape, name):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous cuda {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def qlora_set_timing_events(fwd_begin=None, fwd_end=None, dx_begin=None, dx_end=None) -> None:
    """Raw hipEvent_t handles (ints) recorded around the main GEMM kernels of
    later calls on this thread; all None clears the hook."""
    _check(lib().qlora_set_timing_events(fwd_begin, fwd_end, dx_begin, dx_end))


def qlora_abi_version() -> int:
    return lib().qlora_abi_version()


def nf4_levels():
    """The 16 fp32 NF4 levels in code order (a list of floats)."""
    buf = (ctypes.c_float * 16)()
    lib().nf4_levels(ctypes.cast(buf, ctypes.c_void_p))
    return list(buf)


def codebook_levels(codebook: str = "nf4"):
    """The 16 fp32 levels of a codebook ("nf4" or "int4") in code order."""
    buf = (ctypes.c_float * 16)()
    _check(lib().qlora_codebook_levels(CODEBOOKS[codebook], ctypes.cast(buf, ctypes.c_void_p)))
    return list(buf)


def nf4_storage_bytes(rows: int, cols: int, block: int = 64, dq_block: int = 256):
    c, q, d = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().nf4_storage_bytes(rows, cols, block, dq_block, ctypes.byref(c), ctypes.byref(q),
                                   ctypes.byref(d)))
    return c.value, q.value, d.value


@dataclasses.dataclass
class NF4Weight:
    """A quantized frozen weight [rows][cols] held in device tensors.  With
    double_quant the block scales are 8-bit codes in qscale (dq_format "e4m3" or
    "uint8") and group constants in dscale; without, qscale is None and dscale
    holds the fp32 block scales."""
    codes: "torch.Tensor"              # uint8 [rows*cols/2]
    qscale: Optional["torch.Tensor"]   # uint8 [rows*cols/64], or None
    dscale: "torch.Tensor"             # float32 [ceil(nb/256)], or [nb]
    rows: int
    cols: int
    codebook: str = "nf4"
    dq_format: str = "e4m3"

    @property
    def double_quant(self) -> bool:
        return self.qscale is not None

    def validate(self) -> None:
        """Raise ValueError unless every buffer is a contiguous cuda tensor of the
        dtype and element count nf4_storage_bytes gives for [rows][cols], all on
        one device: the kernels index these buffers by the descriptor's shape."""
        import torch
        if self.codebook not in CODEBOOKS:
            raise ValueError(f"unknown codebook {self.codebook!r}")
        if self.dq_format not in DQ_FORMATS:
            raise ValueError(f"unknown dq_format {self.dq_format!r}")
        c, q, d = nf4_storage_bytes(self.rows, self.cols, 64, 256 if self.double_quant else 0)
        _need(self.codes, torch.uint8, (c,), "codes")
        if self.qscale is not None:
            _need(self.qscale, torch.uint8, (q,), "qscale")
        _need(self.dscale, torch.float32, (d // 4,), "dscale")
        devs = {t.device for t in (self.codes, self.qscale, self.dscale) if t is not None}
        if len(devs) != 1:
            raise ValueError(f"weight buffers are on different devices: {sorted(map(str, devs))}")

    def descriptor(self) -> _Weight:
        self.validate()
        return _Weight(self.codes.data_ptr(), _ptr(self.qscale), self.dscale.data_ptr(),
                       self.rows, self.cols, 64, 256 if self.double_quant else 0,
                       CODEBOOKS[self.codebook], DQ_FORMATS[self.dq_format])

    @staticmethod
    def empty(rows: int, cols: int, device="cuda", codebook: str = "nf4",
              double_quant: bool = True, dq_format: str = "e4m3") -> "NF4Weight":
        import torch
        c, q, d = nf4_storage_bytes(rows, cols, 64, 256 if double_quant else 0)
        return NF4Weight(torch.empty(c, dtype=torch.uint8, device=device),
                         torch.empty(q, dtype=torch.uint8, device=device) if double_quant else None,
                         torch.empty(d // 4, dtype=torch.float32, device=device), rows, cols, codebook,
                         dq_format)


def nf4_quantize(W, out: Optional[NF4Weight] = None, absmax=None, stream=None,
                 codebook: str = "nf4", double_quant: bool = True,
                 dq_format: str = "e4m3") -> NF4Weight:
    """Quantize a cuda fp32 [rows, cols] weight with a codebook ("nf4" or "int4"),
    with double-quantized scales (default; dq_format "e4m3" or "uint8") or fp32
    block scales.  ``absmax`` (optional cuda fp32 [rows*cols/64]) receives the
    exact block scales."""
    import torch
    rows, cols = W.shape
    _need(W, torch.float32, (rows, cols), "W")
    if dq_format not in DQ_FORMATS:
        raise ValueError(f"unknown dq_format {dq_format!r}")
    if out is None:
        out = NF4Weight.empty(rows, cols, W.device, codebook, double_quant, dq_format)
    w = out
    if w.codebook != codebook or w.double_quant != double_quant or \
            (double_quant and w.dq_format != dq_format):
        raise ValueError("out has another codebook or scale format")
    if (w.rows, w.cols) != (rows, cols):
        raise ValueError(f"out holds a {w.rows}x{w.cols} weight, W is {rows}x{cols}")
    w.validate()
    if absmax is not None:
        _need(absmax, torch.float32, (rows * cols // 64,), "absmax")
    _check(lib().qlora_quantize(W.data_ptr(), rows, cols, CODEBOOKS[codebook],
                                256 if double_quant else 0, DQ_FORMATS[dq_format],
                                w.codes.data_ptr(), _ptr(w.qscale),
                                w.dscale.data_ptr(), _ptr(absmax), _stream(stream)))
    return w


def nf4_dequantize(w: NF4Weight, out=None, stream=None):
    """bf16 [rows, cols] dequantized weight."""
    import torch
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.codes.device)
    _need(out, torch.bfloat16, (w.rows, w.cols), "out")
    d = w.descriptor()
    _check(lib().nf4_dequantize(ctypes.byref(d), out.data_ptr(), _stream(stream)))
    return out


def qlora_merge(w: NF4Weight, A, B, alpha: float, out=None, stream=None):
    """bf16 [rows, cols] = bf16(W' + (alpha/r) B A): the adapter merged into the weight."""
    import torch
    r = A.shape[0]
    _need(A, torch.bfloat16, (r, w.cols), "A")
    _need(B, torch.bfloat16, (w.rows, r), "B")
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.codes.device)
    _need(out, torch.bfloat16, (w.rows, w.cols), "out")
    d = w.descriptor()
    _check(lib().qlora_merge(ctypes.byref(d), A.data_ptr(), B.data_ptr(), r, float(alpha),
                             out.data_ptr(), _stream(stream)))
    return out


def qlora_unmerge(W_merged, A, B, alpha: float, out=None, stream=None):
    """bf16 [rows, cols] = bf16(W_merged - (alpha/r) B A); out may be W_merged (in place)."""
    import torch
    rows, cols = W_merged.shape
    r = A.shape[0]
    _need(W_merged, torch.bfloat16, (rows, cols), "W_merged")
    _need(A, torch.bfloat16, (r, cols), "A")
    _need(B, torch.bfloat16, (rows, r), "B")
    if out is None:
        out = torch.empty_like(W_merged)
    _need(out, torch.bfloat16, (rows, cols), "out")
    _check(lib().qlora_unmerge(W_merged.data_ptr(), rows, cols, A.data_ptr(), B.data_ptr(), r, float(alpha),
                               out.data_ptr(), _stream(stream)))
    return out


def qlora_fwd_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return lib().qlora_fwd_workspace_bytes(M, N, K, r)


def qlora_bwd_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return lib().qlora_bwd_workspace_bytes(M, N, K, r)


def _workspace(nbytes: int, device, given):
    import torch
    if given is not None:
        return given
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def qlora_linear_fwd(w: NF4Weight, X, A, B, alpha: float, Y=None, T=None, workspace=None,
                     stream=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """Y = X W'^T + (alpha/r) (X A^T) B^T ; returns (Y [M, N] bf16, T [M, r] fp32)."""
    import torch
    M, K = X.shape
    r = A.shape[0]
    N = w.rows
    _need(X, torch.bfloat16, (M, w.cols), "X")
    _need(A, torch.bfloat16, (r, K), "A")
    _need(B, torch.bfloat16, (N, r), "B")
    Y = Y if Y is not None else torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
    T = T if T is not None else torch.empty(M, r, dtype=torch.float32, device=X.device)
    _need(Y, torch.bfloat16, (M, N), "Y")
    _need(T, torch.float32, (M, r), "T")
    nbytes = qlora_fwd_workspace_bytes(M, N, K, r)
    ws = _workspace(nbytes, X.device, workspace)
    d = w.descriptor()
    _check(lib().qlora_linear_fwd(ctypes.byref(d), X.data_ptr(), M, A.data_ptr(), B.data_ptr(), r,
                                  float(alpha), QL_DTYPE_BF16, Y.data_ptr(), T.data_ptr(), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)))
    return Y, T


def qlora_dual_fwd(w_gate: NF4Weight, w_up: NF4Weight, X, A_gate, B_gate, A_up, B_up,
                   alpha: float, swiglu: bool = False, workspace=None, stream=None):
    """Gate and up projections of one X in one kernel.  Returns
    (Y_gate, Y_up, T_gate, T_up), or with swiglu=True (H, T_gate, T_up) where
    H = bf16(silu(G) * U) from the fp32 sums."""
    import torch
    M, K = X.shape
    r = A_gate.shape[0]
    N = w_gate.rows
    _need(X, torch.bfloat16, (M, w_gate.cols), "X")
    for t, nm in ((A_gate, "A_gate"), (A_up, "A_up")):
        _need(t, torch.bfloat16, (r, K), nm)
    for t, nm in ((B_gate, "B_gate"), (B_up, "B_up")):
        _need(t, torch.bfloat16, (N, r), nm)
    dev = X.device
    Tg = torch.empty(M, r, dtype=torch.float32, device=dev)
    Tu = torch.empty(M, r, dtype=torch.float32, device=dev)
    if swiglu:
        H = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        Yg = Yu = None
    else:
        Yg = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        Yu = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        H = None
    ws = _workspace(qlora_fwd_workspace_bytes(M, N, K, r), dev, workspace)
    dg, du = w_gate.descriptor(), w_up.descriptor()
    _check(lib().qlora_dual_fwd(ctypes.byref(dg), ctypes.byref(du), X.data_ptr(), M,
                                A_gate.data_ptr(), B_gate.data_ptr(), A_up.data_ptr(), B_up.data_ptr(),
                                r, float(alpha), QL_DTYPE_BF16,
                                QL_DUAL_SWIGLU if swiglu else QL_DUAL_SEPARATE,
                                _ptr(Yg), _ptr(Yu), _ptr(H), Tg.data_ptr(), Tu.data_ptr(), _ptr(ws),
                                0 if ws is None else ws.numel(), _stream(stream)))
    return (H, Tg, Tu) if swiglu else (Yg, Yu, Tg, Tu)


def qlora_adamw_step(params, grads, exp_avgs, exp_avg_sqs, lr: float, betas=(0.9, 0.999),
                     eps: float = 1e-8, weight_decay: float = 0.0, step: int = 1, masters=None,
                     stream=None) -> None:
    """One AdamW step over lists of tensors, in place: bf16 params (cuda),
    bf16 grads, fp32 moments, optional fp32 master copies (a list with None
    entries allowed)."""
    import torch
    n = len(params)
    masters = masters if masters is not None else [None] * n
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == len(masters) == n):
        raise ValueError("tensor lists differ in length")
    arr = (_AdamwTensor * max(1, n))()
    for i, (p, g, m, v, w) in enumerate(zip(params, grads, exp_avgs, exp_avg_sqs, masters)):
        shape = tuple(p.shape)
        _need(p, torch.bfloat16, shape, f"params[{i}]")
        _need(g, torch.bfloat16, shape, f"grads[{i}]")
        _need(m, torch.float32, shape, f"exp_avgs[{i}]")
        _need(v, torch.float32, shape, f"exp_avg_sqs[{i}]")
        if w is not None:
            _need(w, torch.float32, shape, f"masters[{i}]")
        arr[i] = _AdamwTensor(p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), _ptr(w), p.numel())
    _check(lib().qlora_adamw_step(ctypes.cast(arr, ctypes.c_void_p), n, float(lr), float(betas[0]),
                                  float(betas[1]), float(eps), float(weight_decay), int(step),
                                  _stream(stream)))


def qlora_linear_bwd(w: NF4Weight, X, dY, A, B, alpha: float, T=None, want_dX: bool = True,
                     dX=None, dA=None, dB=None, workspace=None, stream=None):
    """Returns (dX [M, K] or None, dA [r, K], dB [N, r]) in bf16."""
    import torch
    M, K = X.shape
    r = A.shape[0]
    N = w.rows
    _need(X, torch.bfloat16, (M, w.cols), "X")
    _need(dY, torch.bfloat16, (M, N), "dY")
    _need(A, torch.bfloat16, (r, K), "A")
    _need(B, torch.bfloat16, (N, r), "B")
    if T is not None:
        _need(T, torch.float32, (M, r), "T")
    if want_dX and dX is None:
        dX = torch.empty(M, K, dtype=torch.bfloat16, device=X.device)
    if dX is not None:
        _need(dX, torch.bfloat16, (M, K), "dX")
    dA = dA if dA is not None else torch.empty(r, K, dtype=torch.bfloat16, device=X.device)
    dB = dB if dB is not None else torch.empty(N, r, dtype=torch.bfloat16, device=X.device)
    _need(dA, torch.bfloat16, (r, K), "dA")
    _need(dB, torch.bfloat16, (N, r), "dB")
    ws = _workspace(qlora_bwd_workspace_bytes(M, N, K, r), X.device, workspace)
    d = w.descriptor()
    _check(lib().qlora_linear_bwd(ctypes.byref(d), X.data_ptr(), dY.data_ptr(), M, A.data_ptr(),
                                  B.data_ptr(), r, float(alpha), QL_DTYPE_BF16, _ptr(T), _ptr(dX),
                                  dA.data_ptr(), dB.data_ptr(), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)))
    return dX, dA, dB


def qlora_linear_bwd_noalloc(w: NF4Weight, X, dY, A, B, alpha: float, dX, dA, dB, T=None,
                             stream=None):
    """The backward over the library's fixed per-GPU scratch (no workspace,
    nothing allocated here either: dX (or None), dA [r, K] and dB [N, r] are
    the caller's bf16 outputs).  Calls that can overlap on one GPU race."""
    import torch
    M, K = X.shape
    r = A.shape[0]
    N = w.rows
    _need(X, torch.bfloat16, (M, w.cols), "X")
    _need(dY, torch.bfloat16, (M, N), "dY")
    _need(A, torch.bfloat16, (r, K), "A")
    _need(B, torch.bfloat16, (N, r), "B")
    if T is not None:
        _need(T, torch.float32, (M, r), "T")
    if dX is not None:
        _need(dX, torch.bfloat16, (M, K), "dX")
    _need(dA, torch.bfloat16, (r, K), "dA")
    _need(dB, torch.bfloat16, (N, r), "dB")
    d = w.descriptor()
    _check(lib().qlora_linear_bwd_noalloc(ctypes.byref(d), X.data_ptr(), dY.data_ptr(), M,
                                          A.data_ptr(), B.data_ptr(), r, float(alpha),
                                          QL_DTYPE_BF16, _ptr(T), _ptr(dX), dA.data_ptr(),
                                          dB.data_ptr(), _stream(stream)))
    return dX, dA, dB


# ---------------------------------------------------------------------------
# many adapters on one weight
# ---------------------------------------------------------------------------
_HERE = contextlib.nullcontext()


def _on(device, stream):
    """The stream to launch on and a context under which allocations belong to
    it: the given stream, or `device`'s current one, whichever device is
    current."""
    import torch
    current = torch.cuda.current_stream(device)
    if stream is None:
        stream = current
    elif stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    elif stream != current:
        return stream, torch.cuda.stream(stream)
    return stream, _HERE if device.index == torch.cuda.current_device() else torch.cuda.stream(stream)


def _need_on(t, dtype, shape, name, device):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda or t.device != device:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}, contiguous {t.is_contiguous()}")


@dataclasses.dataclass
class AdapterSet:
    """LoRA adapters of one weight [N, K]: A bf16 [count, r, K], B bf16
    [count, N, r], scale fp32 [count] (alpha / rank of each).  An adapter of a
    rank below r has zeros in its other rows of A and columns of B."""
    A: "torch.Tensor"
    B: "torch.Tensor"
    scale: "torch.Tensor"

    def check(self, w: NF4Weight) -> None:
        """Raise ValueError unless the tensors fit the weight."""
        import torch
        if self.A.dim() != 3:
            raise ValueError(f"A: expected [count, r, K], got {tuple(self.A.shape)}")
        count, r, _ = self.A.shape
        dev = w.codes.device
        _need_on(self.A, torch.bfloat16, (count, r, w.cols), "A", dev)
        _need_on(self.B, torch.bfloat16, (count, w.rows, r), "B", dev)
        _need_on(self.scale, torch.float32, (count,), "scale", dev)


def _multi_workspace(nbytes: int, device, given):
    import torch
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if given.dtype != torch.uint8 or not given.is_contiguous() or given.device != device:
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {device}")
    return given


def qlora_multi_fwd_workspace_bytes(M: int, N: int, K: int, r: int, count: int) -> int:
    return lib().qlora_multi_fwd_workspace_bytes(M, N, K, r, count)


def qlora_multi_bwd_workspace_bytes(M: int, N: int, K: int, r: int, count: int) -> int:
    return lib().qlora_multi_bwd_workspace_bytes(M, N, K, r, count)


def qlora_multi_plan(w: NF4Weight, M: int, r: int, backward: bool = False) -> Tuple[str, int, int]:
    """The kernel that the product with the weight takes for M tokens (dX's with
    `backward`): ("stream", "fused" or "generic", rows of a tile, parts of the
    contraction)."""
    out = (ctypes.c_int * 3)()
    _check(lib().qlora_multi_plan(ctypes.byref(w.descriptor()), M, r, int(backward), ctypes.byref(out)))
    return ("stream", "fused", "generic")[out[0]], out[1], out[2]


def _layer(w, adapters, X, ids, stream):
    """Descriptors, sizes, raw stream and allocation context of a call over
    many adapters; raises where an argument does not fit."""
    got = _native().layer(w, adapters, X, ids)
    if got is None:   # find out why
        import torch
        M, _ = X.shape
        w.validate()
        adapters.check(w)
        _need_on(X, torch.bfloat16, (M, w.cols), "X", w.codes.device)
        _need_on(ids, torch.int32, (M,), "ids", w.codes.device)
        raise ValueError("w, adapters, X and ids have to be an NF4Weight, an AdapterSet and plain tensors")
    *desc, handle, here = got
    if stream is None and here:
        return *desc, handle, _HERE
    stream, ctx = _on(X.device, stream)
    return *desc, stream.cuda_stream, ctx


def qlora_multi_fwd(w: NF4Weight, X, adapters: AdapterSet, ids, Y=None, T=None, workspace=None,
                    stream=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """Tokens of many requests through one weight, each with its own adapter:
    Y[m] = X[m] W'^T + scale[a] (X[m] A[a]^T) B[a]^T, a = ids[m] (int32 [M] on
    the GPU; outside 0 .. count - 1: no adapter).  Returns (Y [M, N] bf16,
    T [M, r] fp32); T is what qlora_multi_bwd takes."""
    import torch
    wd, ad, M, N, K, r, count, handle, ctx = _layer(w, adapters, X, ids, stream)
    dev = X.device
    with ctx:
        if Y is None:
            Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        else:
            _need_on(Y, torch.bfloat16, (M, N), "Y", dev)
        if T is None:
            T = torch.empty(M, r, dtype=torch.float32, device=dev)
        else:
            _need_on(T, torch.float32, (M, r), "T", dev)
        ws = _multi_workspace(lib().qlora_multi_fwd_workspace_bytes(M, N, K, r, count), dev, workspace)
        _check(lib().qlora_multi_fwd(wd, X.data_ptr(), M, ad, ids.data_ptr(), QL_DTYPE_BF16, Y.data_ptr(),
                                     T.data_ptr(), ws.data_ptr(), ws.numel(), handle))
    return Y, T


def qlora_multi_bwd(w: NF4Weight, X, dY, adapters: AdapterSet, ids, T=None, want_dX: bool = True, dX=None,
                    dA=None, dB=None, workspace=None, stream=None):
    """Gradients of qlora_multi_fwd: (dX [M, K] or None, dA [count, r, K],
    dB [count, N, r]) in bf16; zeros for an adapter that no token names."""
    import torch
    wd, ad, M, N, K, r, count, handle, ctx = _layer(w, adapters, X, ids, stream)
    dev = X.device
    _need_on(dY, torch.bfloat16, (M, N), "dY", dev)
    if T is not None:
        _need_on(T, torch.float32, (M, r), "T", dev)
    with ctx:
        if dX is not None:
            _need_on(dX, torch.bfloat16, (M, K), "dX", dev)
        elif want_dX:
            dX = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        if dA is None:
            dA = torch.empty(count, r, K, dtype=torch.bfloat16, device=dev)
        else:
            _need_on(dA, torch.bfloat16, (count, r, K), "dA", dev)
        if dB is None:
            dB = torch.empty(count, N, r, dtype=torch.bfloat16, device=dev)
        else:
            _need_on(dB, torch.bfloat16, (count, N, r), "dB", dev)
        ws = _multi_workspace(lib().qlora_multi_bwd_workspace_bytes(M, N, K, r, count), dev, workspace)
        _check(lib().qlora_multi_bwd(wd, X.data_ptr(), dY.data_ptr(), M, ad, ids.data_ptr(), QL_DTYPE_BF16, _ptr(T),
                                     _ptr(dX), dA.data_ptr(), dB.data_ptr(), ws.data_ptr(), ws.numel(), handle))
    return dX, dA, dB


# ---------------------------------------------------------------------------
# AdamW with 8-bit moments
# ---------------------------------------------------------------------------
ADAMW8_BLOCK = 256


@dataclasses.dataclass
class AdamW8State:
    """One tensor's 8-bit moments: E4M3 codes (uint8, the parameter's element
    count) of the first moment and of the root of the second, and their fp32
    scales, one per 256 elements."""
    exp_avg: "torch.Tensor"
    exp_root: "torch.Tensor"
    exp_avg_scale: "torch.Tensor"
    exp_root_scale: "torch.Tensor"

    @staticmethod
    def zeros(param) -> "AdamW8State":
        """The state before the first step."""
        import torch
        n, dev = param.numel(), param.device
        nb = -(-n // ADAMW8_BLOCK)
        return AdamW8State(torch.zeros(n, dtype=torch.uint8, device=dev), torch.zeros(n, dtype=torch.uint8, device=dev),
                           torch.zeros(nb, dtype=torch.float32, device=dev),
                           torch.zeros(nb, dtype=torch.float32, device=dev))

    def moments(self):
        """(first moment, second moment) in fp32, for checkpoints and inspection."""
        import torch

        def value(codes, scale):
            return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(ADAMW8_BLOCK)[: codes.numel()]
        return value(self.exp_avg, self.exp_avg_scale), value(self.exp_root, self.exp_root_scale) ** 2


def _explain_adamw8(params, grads, states, masters, dev):
    """Raise the ValueError of lists that _marshal.adamw8 did not take."""
    import torch
    written = []   # first byte, order, end, name
    for i, (p, g, s, w) in enumerate(zip(params, grads, states, masters)):
        blocks = (-(-p.numel() // ADAMW8_BLOCK),)
        _need_on(p, torch.bfloat16, p.shape, f"params[{i}]", dev)
        _need_on(g, torch.bfloat16, p.shape, f"grads[{i}]", dev)
        _need_on(s.exp_avg, torch.uint8, (p.numel(),), f"states[{i}].exp_avg", dev)
        _need_on(s.exp_root, torch.uint8, (p.numel(),), f"states[{i}].exp_root", dev)
        _need_on(s.exp_avg_scale, torch.float32, blocks, f"states[{i}].exp_avg_scale", dev)
        _need_on(s.exp_root_scale, torch.float32, blocks, f"states[{i}].exp_root_scale", dev)
        if w is not None:
            _need_on(w, torch.float32, p.shape, f"masters[{i}]", dev)
        for t, name in ((p, "params"), (s.exp_avg, "states"), (s.exp_root, "states"), (s.exp_avg_scale, "states"),
                        (s.exp_root_scale, "states"), (w, "masters")):
            if t is None or not t.numel() or not _native().has_memory(t):   # (a tracer's have no address to ask for)
                continue
            written.append((t.data_ptr(), len(written), t.data_ptr() + t.numel() * t.element_size(), f"{name}[{i}]"))
    written.sort()
    for (a, _, end, other), (b, _, _, name) in zip(written, written[1:]):
        if a == b:
            raise ValueError(f"{name}: the same tensor twice")
        if b < end:
            raise ValueError(f"{name}: shares memory with {other}")
    raise ValueError("params, grads, states and masters have to be lists of plain tensors")


def qlora_adamw8_step(params, grads, states, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                      weight_decay: float = 0.0, step: int = 1, seed: Optional[int] = None, masters=None,
                      stream=None) -> None:
    """One AdamW step over lists of tensors, in place, with 8-bit moments: bf16
    params and grads, AdamW8State per tensor, optional fp32 masters (None
    entries allowed).  seed (32 bits; the step number if None) drives the
    stochastic rounding of the second moment.  It has to differ from step to
    step: under one seed an element meets the same threshold every time, and a
    second moment that shrinks by less than a code a step stays where it is.
    A captured call replays its seed and its step's bias correction, so a graph
    is one step, not a loop's."""
    import torch
    n = len(params)
    masters = masters if masters is not None else [None] * n
    if not (len(grads) == len(states) == len(masters) == n):
        raise ValueError("tensor lists differ in length")
    if n == 0:
        return
    seed = step if seed is None else seed
    dev = params[0].device
    table = _native().adamw8(list(params), list(grads), list(states), list(masters),
                             dev.index if dev.type == "cuda" else -1)
    if table is None:
        _explain_adamw8(params, grads, states, masters, dev)
    stream, ctx = _on(dev, stream)
    with ctx:
        _check(lib().qlora_adamw8_step(table, n, float(lr), float(betas[0]),
                                       float(betas[1]), float(eps), float(weight_decay), int(step),
                                       int(seed) & 0xFFFFFFFF, ctypes.c_void_p(stream.cuda_stream)))
