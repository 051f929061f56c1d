"""ctypes binding of libqlora_nf4.so (the C ABI in include/qlora_nf4.h).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  There is
no fallback: if the library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import functools
import inspect
import os
import re

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "qlora_nf4.h")

QLORA_F32, QLORA_BF16 = 0, 1
STATUS_BYTES = 256
GEMV_MAX_M = 16

STATUS_NAMES = {
    0: "QLORA_OK", 1: "QLORA_ERR_INVALID_ARGUMENT", 2: "QLORA_ERR_UNSUPPORTED_SHAPE",
    3: "QLORA_ERR_MISALIGNED", 4: "QLORA_ERR_WORKSPACE_TOO_SMALL", 5: "QLORA_ERR_NONFINITE",
    6: "QLORA_ERR_TIMEOUT", 7: "QLORA_ERR_CUDA", 8: "QLORA_ERR_NO_DEVICE",
}


class QLoRAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")


class NF4TensorC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scale_codes", ctypes.c_void_p), ("c2", ctypes.c_void_p), ("scale_format", ctypes.c_int32)]


# qlora_scale_format
SCALE_FORMATS = {"e4m3": 0, "e5m2": 1, "u8": 2}


class LoraC(ctypes.Structure):
    _fields_ = [("r", ctypes.c_int32), ("alpha", ctypes.c_float), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p)]


class AdamWC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float)]


class PoolC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("r", ctypes.c_int32), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class TensorC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grad", ctypes.c_void_p), ("param", ctypes.c_void_p),
                ("param_bf16", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p), ("lr_scale", ctypes.c_float)]


class TensorListC(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_tensors", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("n_chunks", ctypes.c_int64)]


_lib = None


def lib():
    """Loads the library once; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with `python -m bit_nf4_quantized_27_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pT, pL = ctypes.POINTER(NF4TensorC), ctypes.POINTER(LoraC)
    pP, pTL = ctypes.POINTER(PoolC), ctypes.POINTER(TensorListC)
    sigs = {
        "qlora_abi_version": (ctypes.c_int, []),
        "qlora_nf4_codebook": (None, [ctypes.POINTER(ctypes.c_float)]),
        "qlora_nf4_storage_bytes": (sz, [i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]),
        "qlora_workspace_bytes": (sz, [i64, i64, i64, i32, ctypes.c_int]),
        "qlora_workspace_bytes_multi": (sz, [i64, i64, i64, i32]),
        "qlora_nf4_quantize": (ctypes.c_int, [vp, ctypes.c_int, pT, vp, vp]),
        "qlora_nf4_dequantize": (ctypes.c_int, [pT, vp, ctypes.c_int, vp]),
        "qlora_linear_fwd": (ctypes.c_int, [pT, pL, vp, i64, vp, ctypes.c_int, vp, vp, sz, vp]),
        "qlora_linear_bwd": (ctypes.c_int, [pT, pL, vp, vp, i64, vp, vp, ctypes.c_int, vp, vp, ctypes.c_int, vp,
                                            sz, vp]),
        "qlora_workspace_bytes_dropout": (sz, [i64, i64, i64, i32, ctypes.c_int]),
        "qlora_linear_fwd_dropout": (ctypes.c_int, [pT, pL, vp, vp, ctypes.c_float, i64, vp, ctypes.c_int, vp, vp,
                                                    sz, vp]),
        "qlora_linear_bwd_dropout": (ctypes.c_int, [pT, pL, vp, vp, vp, ctypes.c_float, i64, vp, vp, ctypes.c_int,
                                                    vp, vp, ctypes.c_int, vp, sz, vp]),
        "qlora_linear_fwd_multi": (ctypes.c_int, [pT, pL, i32, ctypes.POINTER(i32), vp, i64, vp, ctypes.c_int, vp,
                                                  sz, vp]),
        "qlora_lora_merge": (ctypes.c_int, [pT, pL, vp, vp]),
        "qlora_adamw_step": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, ctypes.POINTER(AdamWC), i64, vp]),
        "qlora_adapter_groups": (ctypes.c_int, [vp, i64, i32, vp, vp, vp, vp]),
        "qlora_workspace_bytes_adapters": (sz, [i64, i64, i64, i32, ctypes.c_int]),
        "qlora_adapters_fwd": (ctypes.c_int, [pP, vp, vp, vp, i64, i64, i64, i64, vp, i64, ctypes.c_int, vp, vp, sz, vp]),
        "qlora_adapters_bwd": (ctypes.c_int, [pP, vp, vp, vp, i64, vp, i64, i64, i64, i64, vp, vp, i64, ctypes.c_int, vp,
                                              vp, ctypes.c_int, vp, sz, vp]),
        "qlora_linear_fwd_pool": (ctypes.c_int, [pT, pP, vp, vp, vp, i64, vp, ctypes.c_int, vp, vp, sz, vp]),
        "qlora_linear_bwd_pool": (ctypes.c_int, [pT, pP, vp, vp, vp, vp, i64, vp, vp, ctypes.c_int, vp, vp, ctypes.c_int,
                                                 vp, sz, vp]),
        "qlora_tensor_list_bytes": (sz, [ctypes.POINTER(TensorC), i32]),
        "qlora_tensor_list_init": (ctypes.c_int, [ctypes.POINTER(TensorC), i32, ctypes.c_int, i32, vp, sz, pTL, vp]),
        "qlora_workspace_bytes_grad_norm": (sz, []),
        "qlora_grad_norm": (ctypes.c_int, [pTL, ctypes.c_float, vp, vp, sz, vp]),
        "qlora_adamw_multi": (ctypes.c_int, [pTL, ctypes.POINTER(AdamWC), i64, vp, ctypes.c_uint32, vp]),
        "qlora_selftest_bounded_wait": (ctypes.c_int, [vp, ctypes.c_uint32, vp]),
        "qlora_clear_status": (ctypes.c_int, [vp, vp]),
        "qlora_read_status": (ctypes.c_int, [vp, vp]),
        "qlora_read_library_status": (ctypes.c_int, [vp]),
        "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def header_functions() -> list[str]:
    """Names of the functions include/qlora_nf4.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(qlora_\w+)\s*\(", text)))


def _check(code: int, where: str):
    if code != 0:
        raise QLoRAError(code, where)


def _stream(stream=None):
    # the raw handle without building a Stream object, which costs more than some of the kernels
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on_its_stream(fn):
    """Gives fn a `stream` argument whose call runs with that stream as the current one.  What
    a call allocates, its scratch and the outputs that the caller did not pass, then
    belongs to the stream that its kernels run on: the scratch is zeroed in order with
    them, and memory freed at the return is not handed to another stream under them."""
    place = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kwargs):
        if "stream" not in kwargs and len(args) <= place:
            return fn(*args, **kwargs)
        with torch.cuda.stream(kwargs["stream"] if "stream" in kwargs else args[place]):  # no effect for None
            return fn(*args, **kwargs)

    return call


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype_code(dt):
    if dt == torch.float32:
        return QLORA_F32
    if dt == torch.bfloat16:
        return QLORA_BF16
    raise ValueError(f"unsupported dtype {dt}")


# ---------------------------------------------------------------------------
def codebook() -> list[float]:
    out = (ctypes.c_float * 16)()
    lib().qlora_nf4_codebook(out)
    return list(out)


def storage_bytes(rows: int, cols: int):
    c, s, g = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    total = lib().qlora_nf4_storage_bytes(rows, cols, ctypes.byref(c), ctypes.byref(s), ctypes.byref(g))
    return total, c.value, s.value, g.value


def workspace_bytes(m: int, n: int, k: int, r: int, backward: bool) -> int:
    return int(lib().qlora_workspace_bytes(m, n, k, r, 1 if backward else 0))


class NF4Weight:
    """A quantised [rows, cols] weight: three device buffers owned by torch."""

    def __init__(self, rows: int, cols: int, device="cuda", scale_format: str = "e4m3"):
        total, cb, sb, gb = storage_bytes(rows, cols)
        if total == 0:
            raise ValueError("cols must be a positive multiple of 64")
        if scale_format not in SCALE_FORMATS:
            raise ValueError(f"scale_format must be one of {sorted(SCALE_FORMATS)}")
        self.rows, self.cols = rows, cols
        self.scale_format = scale_format
        self.codes = torch.empty(cb, dtype=torch.uint8, device=device)
        self.scale_codes = torch.empty(sb, dtype=torch.uint8, device=device)
        self.c2 = torch.empty(gb // 4, dtype=torch.float32, device=device)

    def c_struct(self) -> NF4TensorC:
        return NF4TensorC(self.rows, self.cols, self.codes.data_ptr(), self.scale_codes.data_ptr(),
                          self.c2.data_ptr(), SCALE_FORMATS[self.scale_format])

    def nbytes(self) -> int:
        return self.codes.numel() + self.scale_codes.numel() + 4 * self.c2.numel()


def new_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    ws = torch.zeros(max(nbytes, STATUS_BYTES), dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


@_on_its_stream
def quantize(w: torch.Tensor, out: NF4Weight | None = None, ws: torch.Tensor | None = None,
             stream=None, scale_format: str | None = None) -> NF4Weight:
    """NF4 codes with double-quantised block scales; scale_format (default the
    weight's own, E4M3 for a new one) picks the 8-bit scale format."""
    assert w.is_cuda and w.is_contiguous() and w.dim() == 2
    q = out if out is not None else NF4Weight(w.shape[0], w.shape[1], w.device, scale_format or "e4m3")
    if scale_format is not None:
        q.scale_format = scale_format
    if ws is None:
        ws = new_workspace(STATUS_BYTES, w.device)
    t = q.c_struct()
    _check(lib().qlora_nf4_quantize(_ptr(w), _dtype_code(w.dtype), ctypes.byref(t), _ptr(ws), _stream(stream)),
           "qlora_nf4_quantize")
    q._status_ws = ws
    return q


@_on_its_stream
def dequantize(q: NF4Weight, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None):
    y = out if out is not None else torch.empty(q.rows, q.cols, dtype=dtype, device=q.codes.device)
    t = q.c_struct()
    _check(lib().qlora_nf4_dequantize(ctypes.byref(t), _ptr(y), _dtype_code(y.dtype), _stream(stream)),
           "qlora_nf4_dequantize")
    return y


def _lora(A: torch.Tensor, B: torch.Tensor, alpha: float) -> LoraC:
    assert A.dtype == torch.bfloat16 and B.dtype == torch.bfloat16
    assert A.is_contiguous() and B.is_contiguous()
    return LoraC(A.shape[0], float(alpha), A.data_ptr(), B.data_ptr())


@_on_its_stream
def linear_fwd(q: NF4Weight, A, B, alpha: float, X, y_dtype=torch.bfloat16, save_t: bool = True,
               ws: torch.Tensor | None = None, out: torch.Tensor | None = None, t_out=None, stream=None):
    """Y = X W'^T + (alpha/r) (X A^T) B^T.  Returns (Y, T or None); T is the
    [2, M, r] bf16 pair (hi, lo) with hi + lo = X A^T."""
    M = X.shape[0]
    r = A.shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and X.shape[1] == q.cols
    Y = out if out is not None else torch.empty(M, q.rows, dtype=y_dtype, device=X.device)
    T = t_out if t_out is not None else (torch.empty(2, M, r, dtype=torch.bfloat16, device=X.device) if save_t else None)
    need = workspace_bytes(M, q.rows, q.cols, r, False)
    if ws is None:
        ws = new_workspace(need, X.device)
    t, ad = q.c_struct(), _lora(A, B, alpha)
    _check(lib().qlora_linear_fwd(ctypes.byref(t), ctypes.byref(ad), _ptr(X), M, _ptr(Y), _dtype_code(Y.dtype),
                                  _ptr(T), _ptr(ws), ws.numel(), _stream(stream)), "qlora_linear_fwd")
    return Y, T


@_on_its_stream
def linear_bwd(q: NF4Weight, A, B, alpha: float, X, dY, T=None, dx_dtype=torch.bfloat16,
               grad_dtype=torch.bfloat16, ws: torch.Tensor | None = None, outs=None, stream=None):
    """Returns (dX, dA, dB) for upstream gradient dY."""
    M = X.shape[0]
    r = A.shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and X.shape[1] == q.cols
    assert dY.dtype == torch.bfloat16 and dY.is_contiguous() and dY.shape == (M, q.rows)
    if outs is not None:
        dX, dA, dB = outs
    else:
        dX = torch.empty(M, q.cols, dtype=dx_dtype, device=X.device)
        dA = torch.empty(r, q.cols, dtype=grad_dtype, device=X.device)
        dB = torch.empty(q.rows, r, dtype=grad_dtype, device=X.device)
    need = workspace_bytes(M, q.rows, q.cols, r, True)
    if ws is None:
        ws = new_workspace(need, X.device)
    t, ad = q.c_struct(), _lora(A, B, alpha)
    _check(lib().qlora_linear_bwd(ctypes.byref(t), ctypes.byref(ad), _ptr(X), _ptr(dY), M, _ptr(T), _ptr(dX),
                                  _dtype_code(dX.dtype), _ptr(dA), _ptr(dB), _dtype_code(dA.dtype), _ptr(ws),
                                  ws.numel(), _stream(stream)), "qlora_linear_bwd")
    return dX, dA, dB


def selftest_bounded_wait(ws: torch.Tensor, limit_us: int, stream=None):
    """Runs the device-side give-up protocol once: records QLORA_ERR_TIMEOUT in ws."""
    _check(lib().qlora_selftest_bounded_wait(_ptr(ws), int(limit_us), _stream(stream)),
           "qlora_selftest_bounded_wait")


def clear_status(ws: torch.Tensor, stream=None):
    _check(lib().qlora_clear_status(_ptr(ws), _stream(stream)), "qlora_clear_status")


def read_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the device status code (0 = ok)."""
    return int(lib().qlora_read_status(_ptr(ws), _stream(stream)))


def read_library_status(stream=None) -> int:
    """Synchronises the stream, returns and clears the status code of the calls
    without a workspace (the merged export) on the current device (0 = ok)."""
    return int(lib().qlora_read_library_status(_stream(stream)))


class QLoRALinearFunction(torch.autograd.Function):
    """Autograd wrapper: the frozen NF4 weight gets no gradient; A, B and X do."""

    @staticmethod
    def forward(ctx, X, A, B, q: NF4Weight, alpha: float):
        X = X.contiguous()  # the backward reads its rows one behind the other, too
        Y, T = linear_fwd(q, A, B, alpha, X)
        ctx.save_for_backward(X, A, B, T)
        ctx.q, ctx.alpha = q, alpha
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, A, B, T = ctx.saved_tensors
        dX, dA, dB = linear_bwd(ctx.q, A, B, ctx.alpha, X, dY.contiguous().to(torch.bfloat16), T)
        return dX, dA, dB, None, None


@_on_its_stream
def merge(q: NF4Weight, A, B, alpha: float, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Merged export W_merged [N, K] bf16 = bf16(W' + (alpha/r) B A)."""
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=torch.bfloat16, device=A.device)
    t, ad = q.c_struct(), _lora(A, B, alpha)
    _check(lib().qlora_lora_merge(ctypes.byref(t), ctypes.byref(ad), _ptr(out), _stream(stream)), "qlora_lora_merge")
    return out


def adamw_step(p: torch.Tensor, g: torch.Tensor, m: torch.Tensor, v: torch.Tensor, step: int, lr: float,
               beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
               p_bf16: torch.Tensor | None = None, stream=None) -> None:
    """One AdamW step in place on flat float32 tensors p, m, v with gradient g;
    writes bf16(p) to p_bf16 if given."""
    for t in (p, g, m, v):
        assert t.dtype == torch.float32 and t.is_contiguous() and t.numel() == p.numel()
    if p_bf16 is not None:
        assert p_bf16.dtype == torch.bfloat16 and p_bf16.is_contiguous() and p_bf16.numel() == p.numel()
    hp = AdamWC(lr, beta1, beta2, eps, weight_decay)
    _check(lib().qlora_adamw_step(_ptr(p), _ptr(p_bf16), _ptr(g), _ptr(m), _ptr(v), p.numel(), ctypes.byref(hp),
                                  step, _stream(stream)), "qlora_adamw_step")


@_on_its_stream
def linear_fwd_multi(q: NF4Weight, adapters, adapter_of_token, X, y_dtype=torch.bfloat16,
                     ws: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode forward of one base serving several adapters: adapters is a list of
    (A, B, alpha) of one rank; token t uses adapters[adapter_of_token[t]]."""
    M = X.shape[0]
    r = adapters[0][0].shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and X.shape[1] == q.cols
    Y = out if out is not None else torch.empty(M, q.rows, dtype=y_dtype, device=X.device)
    arr = (LoraC * len(adapters))(*[_lora(a, b, alpha) for a, b, alpha in adapters])
    idx = (ctypes.c_int32 * M)(*[int(i) for i in adapter_of_token])
    if ws is None:
        ws = new_workspace(workspace_bytes_multi(M, q.rows, q.cols, r), X.device)
    t = q.c_struct()
    _check(lib().qlora_linear_fwd_multi(ctypes.byref(t), arr, len(adapters), idx, _ptr(X), M, _ptr(Y),
                                        _dtype_code(Y.dtype), _ptr(ws), ws.numel(), _stream(stream)),
           "qlora_linear_fwd_multi")
    return Y


def workspace_bytes_multi(m: int, n: int, k: int, r: int) -> int:
    return int(lib().qlora_workspace_bytes_multi(m, n, k, r))


def workspace_bytes_dropout(m: int, n: int, k: int, r: int, backward: bool) -> int:
    return int(lib().qlora_workspace_bytes_dropout(m, n, k, r, 1 if backward else 0))


@_on_its_stream
def linear_fwd_dropout(q: NF4Weight, A, B, alpha: float, X, keep: torch.Tensor, p: float, y_dtype=torch.bfloat16,
                       save_t: bool = True, ws: torch.Tensor | None = None, stream=None):
    """Forward with LoRA dropout on the adapter input; keep is the packed
    uint8 [M, K/8] mask.  Returns (Y, T pair or None) as linear_fwd."""
    M, K = X.shape
    r = A.shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and K == q.cols
    assert keep.dtype == torch.uint8 and keep.is_contiguous() and tuple(keep.shape) == (M, K // 8)
    Y = torch.empty(M, q.rows, dtype=y_dtype, device=X.device)
    T = torch.empty(2, M, r, dtype=torch.bfloat16, device=X.device) if save_t else None
    if ws is None:
        ws = new_workspace(workspace_bytes_dropout(M, q.rows, q.cols, r, False), X.device)
    t, ad = q.c_struct(), _lora(A, B, alpha)
    _check(lib().qlora_linear_fwd_dropout(ctypes.byref(t), ctypes.byref(ad), _ptr(X), _ptr(keep), float(p), M,
                                          _ptr(Y), _dtype_code(Y.dtype), _ptr(T), _ptr(ws), ws.numel(),
                                          _stream(stream)), "qlora_linear_fwd_dropout")
    return Y, T


@_on_its_stream
def linear_bwd_dropout(q: NF4Weight, A, B, alpha: float, X, dY, keep: torch.Tensor, p: float, T=None,
                       dx_dtype=torch.bfloat16, grad_dtype=torch.bfloat16, ws: torch.Tensor | None = None, stream=None):
    """Gradients (dX, dA, dB) of linear_fwd_dropout for upstream dY."""
    M, K = X.shape
    r = A.shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and K == q.cols
    assert dY.dtype == torch.bfloat16 and dY.is_contiguous() and dY.shape == (M, q.rows)
    assert keep.dtype == torch.uint8 and keep.is_contiguous() and tuple(keep.shape) == (M, K // 8)
    dX = torch.empty(M, K, dtype=dx_dtype, device=X.device)
    dA = torch.empty(r, K, dtype=grad_dtype, device=X.device)
    dB = torch.empty(q.rows, r, dtype=grad_dtype, device=X.device)
    if ws is None:
        ws = new_workspace(workspace_bytes_dropout(M, q.rows, q.cols, r, True), X.device)
    t, ad = q.c_struct(), _lora(A, B, alpha)
    _check(lib().qlora_linear_bwd_dropout(ctypes.byref(t), ctypes.byref(ad), _ptr(X), _ptr(dY), _ptr(keep), float(p),
                                          M, _ptr(T), _ptr(dX), _dtype_code(dx_dtype), _ptr(dA), _ptr(dB),
                                          _dtype_code(grad_dtype), _ptr(ws), ws.numel(), _stream(stream)),
           "qlora_linear_bwd_dropout")
    return dX, dA, dB


# ---------------------------------------------------------------------------
# Many adapters on one base
# ---------------------------------------------------------------------------
def _here(*tensors):
    """The operands of a call lie on the current device, where its kernels run."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:  # -1 for a tensor on the CPU
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")


_increment_version = torch._C._increment_version  # torch.autograd.graph.increment_version without its own checks


def _wrote(*tensors):
    """The call has written these tensors of the caller's.  Autograd learns of it, so that a backward
    whose forward read what stood there before raises, as after any operation in place (a graph's
    replays write without a call, and do not tell)."""
    _increment_version([t for t in tensors if t is not None])


class AdapterPool:
    """n adapters side by side: A [n, r, K] and B [n, N, r] bf16, scales [n] float32,
    and, where ranks differ, ranks [n] int32 (adapter i is the first ranks[i] rows of
    A[i] and columns of B[i])."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scales: torch.Tensor, ranks: torch.Tensor | None = None):
        assert A.dtype == torch.bfloat16 and B.dtype == torch.bfloat16 and A.is_contiguous() and B.is_contiguous()
        assert A.dim() == 3 and B.dim() == 3 and A.shape[0] == B.shape[0] and A.shape[1] == B.shape[2]
        assert scales.dtype == torch.float32 and scales.is_contiguous() and scales.numel() == A.shape[0]
        assert scales.device == A.device == B.device
        if ranks is not None:
            assert ranks.dtype == torch.int32 and ranks.is_contiguous() and ranks.numel() == A.shape[0]
            assert ranks.device == A.device
        self.A, self.B, self.scales, self.ranks = A, B, scales, ranks
        self.n, self.r = A.shape[0], A.shape[1]
        self.cols, self.rows = A.shape[2], B.shape[1]  # K, N
        self._c = PoolC(self.n, self.r, A.data_ptr(), B.data_ptr(), None if ranks is None else ranks.data_ptr(),
                        scales.data_ptr())

        self._ref = ctypes.byref(self._c)

    def c_struct(self) -> PoolC:
        return self._c


def workspace_bytes_adapters(m: int, n: int, k: int, r: int, backward: bool) -> int:
    return int(lib().qlora_workspace_bytes_adapters(m, n, k, r, 1 if backward else 0))


@_on_its_stream
def adapter_groups(adapter_of_token: torch.Tensor, n: int, out=None, ws: torch.Tensor | None = None, stream=None):
    """(order [M], offsets [n + 1]) int32: the tokens grouped by adapter (-1: none, last).  Here and in the
    calls that take the groups, what the kernels find wrong (an index, a place or a rank out of range) stands in
    ws's status word, for read_status; a call without ws does not tell of it."""
    idx = adapter_of_token
    assert idx.dtype == torch.int32 and idx.is_contiguous() and idx.dim() == 1
    M = idx.numel()
    if out is None:
        order, offsets = idx.new_empty(M), idx.new_empty(n + 1)
    else:
        order, offsets = out
        assert order.dtype == offsets.dtype == torch.int32 and order.is_contiguous() and offsets.is_contiguous()
        assert order.numel() == M and offsets.numel() == n + 1
    _here(idx, order, offsets, ws)
    if ws is None:
        ws = new_workspace(STATUS_BYTES, idx.device)
    _check(lib().qlora_adapter_groups(idx.data_ptr(), M, n, order.data_ptr(), offsets.data_ptr(), ws.data_ptr(), _stream(stream)),
           "qlora_adapter_groups")
    if out is not None:
        _wrote(order, offsets)
    return order, offsets


def _group_ptrs(groups, pool: AdapterPool, m: int):
    order, offsets = groups
    assert order.dtype == offsets.dtype == torch.int32 and order.is_contiguous() and offsets.is_contiguous()
    assert order.numel() == m and offsets.numel() == pool.n + 1
    return order.data_ptr(), offsets.data_ptr()


def _row_stride(t: torch.Tensor) -> int:
    """Row stride of a [rows, cols] tensor whose rows are contiguous; that of a single row, which nothing
    goes by, is its length."""
    (rows, cols), (row, col) = t.shape, t.stride()
    assert cols == 1 or col == 1
    return row if rows > 1 else cols


@_on_its_stream
def adapters_fwd(pool: AdapterPool, groups, X: torch.Tensor, Y: torch.Tensor, save_t: bool = False, t_out=None,
                 ws: torch.Tensor | None = None, stream=None):
    """Adds every token's adapter term to Y in place: Y[t] += s_a (X[t] A_a^T) B_a^T, outside autograd
    (QLoRAPoolLinearFunction is the layer with gradients).
    groups: (order, offsets) of adapter_groups.  X and Y may be column slices of wider
    tensors.  Returns T, the bf16 [3, M, r] planes whose sum is X A^T, or None."""
    M, cols = X.shape
    assert X.dtype == torch.bfloat16 and cols == pool.cols and Y.shape == (M, pool.rows)
    order, offsets = _group_ptrs(groups, pool, M)
    T = t_out if t_out is not None else (torch.empty(3, M, pool.r, dtype=torch.bfloat16, device=X.device) if save_t else None)
    assert T is None or (T.dtype == torch.bfloat16 and T.is_contiguous() and T.numel() == 3 * M * pool.r)
    _here(X, Y, T, ws, pool.A, *groups)
    if ws is None:
        ws = new_workspace(workspace_bytes_adapters(M, pool.rows, pool.cols, pool.r, False), X.device)
    _check(lib().qlora_adapters_fwd(pool._ref, order, offsets, X.data_ptr(), _row_stride(X), M, pool.rows,
                                    pool.cols, Y.data_ptr(), _row_stride(Y), _dtype_code(Y.dtype), _ptr(T), ws.data_ptr(),
                                    ws.numel(), _stream(stream)), "qlora_adapters_fwd")
    _wrote(Y, t_out)
    return T


def _pool_grads(pool: AdapterPool, grad_dtype, outs, device):
    if outs is None:
        return (torch.empty(pool.n, pool.r, pool.cols, dtype=grad_dtype, device=device),
                torch.empty(pool.n, pool.rows, pool.r, dtype=grad_dtype, device=device))
    dA, dB = outs
    assert dA.dtype == dB.dtype and dA.is_contiguous() and dB.is_contiguous()
    assert dA.shape == pool.A.shape and dB.shape == pool.B.shape
    return dA, dB


@_on_its_stream
def adapters_bwd(pool: AdapterPool, groups, X: torch.Tensor, dY: torch.Tensor, T=None, dX: torch.Tensor | None = None,
                 need_grads: bool = True, grad_dtype=torch.float32, outs=None, ws: torch.Tensor | None = None, stream=None):
    """Gradients of adapters_fwd.  Adds the adapters' part to dX in place (if given) and
    returns (dA [n, r, K], dB [n, N, r]), or (None, None) without need_grads."""
    M = X.shape[0]
    assert X.dtype == torch.bfloat16 and X.shape[1] == pool.cols
    assert dY.dtype == torch.bfloat16 and dY.shape == (M, pool.rows)
    assert dX is None or dX.shape == (M, pool.cols)
    assert T is None or (T.dtype == torch.bfloat16 and T.is_contiguous() and T.numel() == 3 * M * pool.r)
    order, offsets = _group_ptrs(groups, pool, M)
    dA, dB = _pool_grads(pool, grad_dtype, outs, X.device) if need_grads else (None, None)
    _here(X, dY, T, dX, dA, dB, ws, pool.A, *groups)
    if ws is None:
        ws = new_workspace(workspace_bytes_adapters(M, pool.rows, pool.cols, pool.r, True), X.device)
    _check(lib().qlora_adapters_bwd(pool._ref, order, offsets, X.data_ptr(), _row_stride(X), dY.data_ptr(),
                                    _row_stride(dY), M, pool.rows, pool.cols, _ptr(T), _ptr(dX),
                                    0 if dX is None else _row_stride(dX), QLORA_F32 if dX is None else _dtype_code(dX.dtype),
                                    _ptr(dA), _ptr(dB), QLORA_F32 if dA is None else _dtype_code(dA.dtype), _ptr(ws),
                                    ws.numel(), _stream(stream)), "qlora_adapters_bwd")
    _wrote(dX, *(outs or ()))
    return dA, dB


@_on_its_stream
def linear_fwd_pool(q: NF4Weight, pool: AdapterPool, groups, X, y_dtype=torch.bfloat16, save_t: bool = True,
                    ws: torch.Tensor | None = None, out: torch.Tensor | None = None, t_out=None, stream=None):
    """Forward of the NF4 layer with every token's own adapter, outside autograd.  Returns (Y, T or
    None).  For a decode step of up to 16 tokens whose adapters the host knows, of one rank,
    linear_fwd_multi is faster."""
    M = X.shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and X.shape[1] == q.cols == pool.cols and pool.rows == q.rows
    Y = out if out is not None else torch.empty(M, q.rows, dtype=y_dtype, device=X.device)
    assert Y.is_contiguous() and tuple(Y.shape) == (M, q.rows)
    T = t_out if t_out is not None else (torch.empty(3, M, pool.r, dtype=torch.bfloat16, device=X.device) if save_t else None)
    assert T is None or (T.dtype == torch.bfloat16 and T.is_contiguous() and T.numel() == 3 * M * pool.r)
    order, offsets = _group_ptrs(groups, pool, M)
    _here(X, Y, T, ws, pool.A, q.codes, *groups)
    if ws is None:
        ws = new_workspace(workspace_bytes_adapters(M, q.rows, q.cols, pool.r, False), X.device)
    t = q.c_struct()
    _check(lib().qlora_linear_fwd_pool(ctypes.byref(t), pool._ref, order, offsets, _ptr(X), M, _ptr(Y),
                                       _dtype_code(Y.dtype), _ptr(T), _ptr(ws), ws.numel(), _stream(stream)),
           "qlora_linear_fwd_pool")
    if out is not None or t_out is not None:
        _wrote(out, t_out)
    return Y, T


@_on_its_stream
def linear_bwd_pool(q: NF4Weight, pool: AdapterPool, groups, X, dY, T=None, dx_dtype=torch.bfloat16,
                    grad_dtype=torch.bfloat16, ws: torch.Tensor | None = None, outs=None, stream=None,
                    need_grads: bool = True):
    """Returns (dX, dA [n, r, K], dB [n, N, r]) for upstream gradient dY, or (dX, None, None)
    without need_grads.  (dA and dB without dX, and so without the base product, are
    adapters_bwd's.)"""
    M = X.shape[0]
    assert X.dtype == torch.bfloat16 and X.is_contiguous() and X.shape[1] == q.cols == pool.cols and pool.rows == q.rows
    assert dY.dtype == torch.bfloat16 and dY.is_contiguous() and tuple(dY.shape) == (M, q.rows)
    assert T is None or (T.dtype == torch.bfloat16 and T.is_contiguous() and T.numel() == 3 * M * pool.r)
    dX = outs[0] if outs is not None else torch.empty(M, q.cols, dtype=dx_dtype, device=X.device)
    assert dX.is_contiguous() and tuple(dX.shape) == (M, q.cols)
    dA, dB = _pool_grads(pool, grad_dtype, None if outs is None else outs[1:], X.device) if need_grads else (None, None)
    order, offsets = _group_ptrs(groups, pool, M)
    _here(X, dY, T, dX, dA, dB, ws, pool.A, q.codes, *groups)
    if ws is None:
        ws = new_workspace(workspace_bytes_adapters(M, q.rows, q.cols, pool.r, True), X.device)
    t = q.c_struct()
    _check(lib().qlora_linear_bwd_pool(ctypes.byref(t), pool._ref, order, offsets, _ptr(X), _ptr(dY), M,
                                       _ptr(T), _ptr(dX), _dtype_code(dX.dtype), _ptr(dA), _ptr(dB),
                                       QLORA_F32 if dA is None else _dtype_code(dA.dtype), _ptr(ws), ws.numel(),
                                       _stream(stream)), "qlora_linear_bwd_pool")
    if outs is not None:
        _wrote(*outs)
    return dX, dA, dB


class QLoRAPoolLinearFunction(torch.autograd.Function):
    """Autograd wrapper of the NF4 layer with a pool: X, A [n, r, K] and B [n, N, r] get
    gradients, those of them that require one; groups, scales and ranks are the batch's and
    the pool's constants.  ws: a workspace of the backward's size, which both
    directions then use; its status word (read_status) tells of a bad group, a bad rank or a wait
    that ran out, and without one nothing does."""

    @staticmethod
    def forward(ctx, X, A, B, q: NF4Weight, groups, scales, ranks=None, ws: torch.Tensor | None = None):
        X = X.contiguous()
        grads = any(ctx.needs_input_grad[1:3])  # T is for them alone
        Y, T = linear_fwd_pool(q, AdapterPool(A, B, scales, ranks), groups, X, save_t=grads, ws=ws)
        ctx.save_for_backward(X, A, B, T, scales, *groups, *([] if ranks is None else [ranks]))
        ctx.q, ctx.ws = q, ws
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, A, B, T, scales, order, offsets, *ranks = ctx.saved_tensors
        pool = AdapterPool(A, B, scales, ranks[0] if ranks else None)
        groups, dY = (order, offsets), dY.contiguous().to(torch.bfloat16)
        need_x, need_a, need_b = ctx.needs_input_grad[:3]
        dX = None
        if need_x:
            dX, dA, dB = linear_bwd_pool(ctx.q, pool, groups, X, dY, T, need_grads=need_a or need_b, ws=ctx.ws)
        else:
            dA, dB = adapters_bwd(pool, groups, X, dY, T, grad_dtype=torch.bfloat16, ws=ctx.ws)
        return dX, dA if need_a else None, dB if need_b else None, None, None, None, None, None


# ---------------------------------------------------------------------------
# One optimiser step over a list of tensors
# ---------------------------------------------------------------------------
class TensorList:
    """The tensors of one optimiser step and its device table.  grads alone serve
    grad_norm; adamw_multi also needs params (float32) and the states: float32, or
    8-bit codes (uint8, or float8_e4m3fn for exp_avg and float8_e5m2 for exp_avg_sq)
    with a float32 scale per 256 elements.  The list keeps its tensors alive; they must
    not move (a gradient that is allocated anew needs a new list)."""

    @_on_its_stream
    def __init__(self, grads, params=None, exp_avg=None, exp_avg_sq=None, p_bf16=None, exp_avg_scale=None,
                 exp_avg_sq_scale=None, lr_scale=None, stream=None):
        grads = list(grads)
        count = len(grads)
        assert count > 0
        gdt = grads[0].dtype
        bits = 0 if params is None else (32 if exp_avg[0].dtype == torch.float32 else 8)
        columns = [grads, params, p_bf16, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale]
        columns = [None if c is None else list(c) for c in columns]
        for c in columns:
            assert c is None or len(c) == count
        grads, params, p_bf16, exp_avg, exp_avg_sq, ms, vs = columns
        code_m, code_v = (torch.uint8, torch.float8_e4m3fn), (torch.uint8, torch.float8_e5m2)
        for i, g in enumerate(grads):
            assert g.dtype == gdt and g.is_contiguous()
            if bits:
                n, nb = g.numel(), -(-g.numel() // 256)
                kinds = [(params, (torch.float32,), n), (p_bf16, (torch.bfloat16,), n),
                         (exp_avg, (torch.float32,) if bits == 32 else code_m, n),
                         (exp_avg_sq, (torch.float32,) if bits == 32 else code_v, n)]
                if bits == 8:
                    kinds += [(ms, (torch.float32,), nb), (vs, (torch.float32,), nb)]
                for col, types, size in kinds:
                    if col is None and col is p_bf16:
                        continue
                    t = col[i]
                    assert t.dtype in types and t.is_contiguous() and t.numel() == size and t.device == g.device
        _here(*(t for c in columns if c is not None for t in c))
        arr = (TensorC * count)()
        for i in range(count):
            p = [0 if c is None else c[i].data_ptr() for c in (grads, params, p_bf16, exp_avg, exp_avg_sq, ms, vs)]
            arr[i] = TensorC(grads[i].numel(), *p, 1.0 if lr_scale is None else float(lr_scale[i]))
        nbytes = int(lib().qlora_tensor_list_bytes(arr, count))
        if nbytes == 0:
            raise QLoRAError(2, "qlora_tensor_list_bytes")
        self.table = torch.empty(nbytes, dtype=torch.uint8, device=grads[0].device)
        self._c = TensorListC()
        _check(lib().qlora_tensor_list_init(arr, count, _dtype_code(gdt), bits, _ptr(self.table), nbytes,
                                            ctypes.byref(self._c), _stream(stream)), "qlora_tensor_list_init")
        self._keep = columns
        # what adamw_multi writes and a graph may have saved; views of one tensor share its version
        written = [t if t._base is None else t._base for c in (params, p_bf16) if bits and c is not None for t in c]
        self._written = list({id(t): t for t in written}.values())
        self.state_bits = bits
        self._ref = ctypes.byref(self._c)

    def c_struct(self) -> TensorListC:
        return self._c


def workspace_bytes_grad_norm() -> int:
    return int(lib().qlora_workspace_bytes_grad_norm())


@_on_its_stream
def grad_norm(tensors: TensorList, max_norm: float, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """float32 [2] on the device: the norm of all gradients and min(1, max_norm / (norm + 1e-6))."""
    result = torch.empty(2, dtype=torch.float32, device=tensors.table.device) if out is None else out
    assert result.dtype == torch.float32 and result.is_contiguous() and result.numel() == 2
    _here(tensors.table, result, ws)
    if ws is None:
        ws = new_workspace(workspace_bytes_grad_norm(), tensors.table.device)
    _check(lib().qlora_grad_norm(tensors._ref, float(max_norm), result.data_ptr(), ws.data_ptr(), ws.numel(),
                                 _stream(stream)), "qlora_grad_norm")
    if out is not None:
        _wrote(out)
    return result


def adamw_multi(tensors: TensorList, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                weight_decay: float = 0.0, clip: torch.Tensor | None = None, seed: int | None = None, stream=None) -> None:
    """One AdamW step in place on every tensor of the list.  clip: what grad_norm returned
    (gradients are multiplied by clip[1]; NaN there leaves everything as it is).  seed: the
    random bits of the 8-bit states' rounding, by default of the step; with the same ones at
    every step each element would always be rounded by the same threshold, and a
    slowly changing variance would not move.  A call captured into a graph keeps its step and
    seed."""
    assert clip is None or (clip.dtype == torch.float32 and clip.is_contiguous() and clip.numel() == 2)
    _here(tensors.table, clip)
    hp = AdamWC(lr, beta1, beta2, eps, weight_decay)
    _check(lib().qlora_adamw_multi(tensors._ref, ctypes.byref(hp), step, _ptr(clip),
                                   (step if seed is None else seed) & 0xffffffff,
                                   _stream(stream)), "qlora_adamw_multi")
    _wrote(*tensors._written)
