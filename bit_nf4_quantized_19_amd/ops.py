"""Python binding of libqlora_nf4 (argument marshalling only).

Every function here forwards torch device tensors (as raw pointers) and the
current HIP stream to the C ABI declared in ``include/qlora_nf4.h``; all
arithmetic runs in the library's gfx950 kernels. There is no fallback: if the
shared library is missing or fails to load, the first call raises.

bf16 tensors are ``torch.bfloat16`` (passed as their uint16 bit patterns).
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")
#: measurement build of the same sources with per-launch HIP events
#: (include/qlora_nf4_timing.h); loaded only inside ``timing_build()``
TIMING_LIB_PATH = os.path.join(_HERE, "libqlora_nf4_timing.so")

QLORA_OK, QLORA_ERR_INVALID_ARG, QLORA_ERR_UNSUPPORTED, QLORA_ERR_WORKSPACE, QLORA_ERR_HIP = (
    0, -1, -2, -3, -4)
OP_QUANTIZE, OP_FWD, OP_BWD, OP_FWD_MULTI, OP_QUANTIZE_RESIDUAL, OP_LOFTQ = 0, 1, 2, 3, 4, 5


class QLoRAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class NF4WeightC(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int64), ("k", ctypes.c_int64),
        ("blocksize", ctypes.c_int32), ("double_quant", ctypes.c_int32),
        ("dq_blocksize", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p),
        ("absmax_q", ctypes.c_void_p), ("absmax_scale", ctypes.c_void_p),
        ("absmax_offset", ctypes.c_void_p),
    ]


_lib = None
_timing_lib = None
_use_timing = False
_vp, _i64, _i32, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                              ctypes.c_float, ctypes.c_size_t)
_PW = ctypes.POINTER(NF4WeightC)

#: exported symbol -> (restype, argtypes); mirrors include/qlora_nf4.h and the
#: headers named below
SIGNATURES = {
    "qlora_nf4_quantize": (ctypes.c_int, [_vp, _PW, _vp, _sz, _vp]),
    "qlora_nf4_dequantize": (ctypes.c_int, [_PW, _vp, _vp]),
    "qlora_linear_fwd": (ctypes.c_int, [_PW, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp,
                                        _vp, _sz, _vp]),
    "qlora_linear_bwd": (ctypes.c_int, [_PW, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _sz, _vp]),
    "qlora_linear_fwd_ex": (ctypes.c_int, [_PW, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp,
                                           _vp, _sz, _vp]),
    "qlora_linear_bwd_ex": (ctypes.c_int, [_PW, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _sz, _vp]),
    "qlora_linear_fwd_multi": (ctypes.c_int, [_vp, _i32, _vp, _i64, _vp, _vp, _i32, _f32, _vp,
                                              _vp, _vp, _sz, _vp]),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [_PW, _vp, _i64, _vp, _vp, _i32, _f32, _vp, _vp,
                                                _vp]),
    "qlora_merge": (ctypes.c_int, [_PW, _vp, _vp, _i32, _f32, _vp, _vp]),
    "qlora_nf4_quantize_residual": (ctypes.c_int, [_vp, _vp, _vp, _i32, _f32, _PW, _vp, _sz,
                                                   _vp]),
    "qlora_loftq_init": (ctypes.c_int, [_vp, _vp, _i32, _f32, _i32, _i32, _PW, _vp, _vp, _vp,
                                        _vp, _sz, _vp]),
    "qlora_nf4_storage_bytes": (_sz, [_i64, _i64, _i32]),
    "qlora_workspace_bytes": (_sz, [_i32, _i64, _i64, _i64, _i32, _i32]),
    "qlora_nf4_codebook": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(ctypes.c_float)]),
    "qlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_adamw_step": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp]),
    "qlora_adamw_page_out": (ctypes.c_int, [_vp, _vp, _i32, _i64, _vp]),
    "qlora_adamw_page_in": (ctypes.c_int, [_vp, _vp, _i32, _i64, _vp]),
    # include/qlora_adapters.h
    "qlora_adapter_plan_bytes": (_sz, [_i64, _i32]),
    "qlora_adapter_plan_build": (ctypes.c_int, [_vp, _vp, _vp]),
    "qlora_adapters_workspace_bytes": (_sz, [_i32, _i64, _i64, _i64, _i32, _i32]),
    "qlora_linear_fwd_adapters": (ctypes.c_int, [_PW, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "qlora_linear_bwd_adapters": (ctypes.c_int, [_PW, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                 _sz, _vp]),
    # include/qlora_logprobs.h
    "qlora_token_logprobs_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32]),
    "qlora_token_logprobs": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz,
                                            _vp]),
    "qlora_token_logprobs_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
}

#: the timing build's extra symbols; mirrors include/qlora_nf4_timing.h
TIMING_SIGNATURES = {
    "qlora_profile_begin": (ctypes.c_int, [_i32, ctypes.c_uint32]),
    "qlora_profile_end": (ctypes.c_int, []),
    "qlora_profile_query": (ctypes.c_int, [_i32, ctypes.POINTER(ctypes.c_int32),
                                           ctypes.POINTER(ctypes.c_double)]),
    "qlora_profile_release": (ctypes.c_int, []),
}

#: kernel ids of the timing hooks (QLORA_K_* in include/qlora_nf4_timing.h);
#: ids 8 and 10 are reserved and never recorded
KERNELS = ["quantize", "double_quant", "dequantize", "gemm_fwd", "gemm_dx", "gemv",
           "gemv_epilogue", "lora_down", "lora_reduce", "lora_colacc", "lora_colacc_reduce",
           "merge", "layout", "adamw", "loftq_product", "loftq_small", "residual", "adapter_plan",
           "logprobs", "logprobs_grad"]


def _load(path: str, signatures: dict) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing; build it with "
                          "`python -m bit_nf4_quantized_19_amd.build`")
    L = ctypes.CDLL(path)
    for name, (res, args) in signatures.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def lib() -> ctypes.CDLL:
    """The library every call goes through: the product build, or the timing
    build inside ``timing_build()``. Loaded once; raises if it is not built."""
    global _lib
    if _use_timing:
        return timing_lib()
    if _lib is None:
        _lib = _load(LIB_PATH, SIGNATURES)
    return _lib


def timing_lib() -> ctypes.CDLL:
    """The timing build (same kernels and entry points plus qlora_profile_*)."""
    global _timing_lib
    if _timing_lib is None:
        _timing_lib = _load(TIMING_LIB_PATH, {**SIGNATURES, **TIMING_SIGNATURES})
    return _timing_lib


@contextlib.contextmanager
def timing_build():
    """Route every call of this module to the timing build while inside."""
    global _use_timing
    prev = _use_timing
    _use_timing = True
    try:
        yield timing_lib()
    finally:
        _use_timing = prev


def status_string(status: int) -> str:
    return lib().qlora_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != QLORA_OK:
        raise QLoRAError(status, what)


def _stream(stream=None) -> int:
    if stream is None:   # the handle itself, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dev_bf16(t: torch.Tensor, name: str):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")


# ---------------------------------------------------------------------------
@dataclass
class NF4Weight:
    """Quantised weight: packed codes plus absmax or its double-quantised form."""
    d: int
    k: int
    double_quant: bool
    codes: torch.Tensor                      # uint8 [d*k/2]
    absmax: torch.Tensor | None = None       # float32 [nb]
    absmax_q: torch.Tensor | None = None     # int8 [nb]
    absmax_scale: torch.Tensor | None = None  # float32 [ceil(nb/256)]
    absmax_offset: torch.Tensor | None = None  # float32 [1]

    def c_struct(self) -> NF4WeightC:
        return NF4WeightC(self.d, self.k, 64, int(self.double_quant), 256, 0,
                          _ptr(self.codes), _ptr(self.absmax), _ptr(self.absmax_q),
                          _ptr(self.absmax_scale), _ptr(self.absmax_offset))

    @staticmethod
    def empty(d: int, k: int, double_quant: bool, device="cuda") -> "NF4Weight":
        n = d * k
        nb = n // 64
        w = NF4Weight(d, k, double_quant, torch.empty(n // 2, dtype=torch.uint8, device=device))
        if double_quant:
            w.absmax_q = torch.empty(nb, dtype=torch.int8, device=device)
            w.absmax_scale = torch.empty(-(-nb // 256), dtype=torch.float32, device=device)
            w.absmax_offset = torch.empty(1, dtype=torch.float32, device=device)
        else:
            w.absmax = torch.empty(nb, dtype=torch.float32, device=device)
        return w


def storage_bytes(d: int, k: int, double_quant: bool) -> int:
    return int(lib().qlora_nf4_storage_bytes(d, k, int(double_quant)))


def workspace_bytes(op: int, d: int, k: int, M: int = 0, r: int = 0,
                    double_quant: bool = True) -> int:
    n = lib().qlora_workspace_bytes(op, d, k, M, r, int(double_quant))
    if n == ctypes.c_size_t(-1).value:
        raise QLoRAError(QLORA_ERR_UNSUPPORTED, "workspace_bytes")
    return int(n)


def codebook():
    lv = (ctypes.c_float * 16)()
    th = (ctypes.c_float * 15)()
    _check(lib().qlora_nf4_codebook(lv, th), "codebook")
    return list(lv), list(th)


def _workspace(nbytes: int, device, ws: torch.Tensor | None):
    if nbytes == 0:
        return None, 0
    if ws is not None:
        return ws, ws.numel() * ws.element_size()
    t = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-t.data_ptr()) % 256
    return t[off:off + nbytes], nbytes


def quantize(W0: torch.Tensor, double_quant: bool = True, out: NF4Weight | None = None,
             ws: torch.Tensor | None = None, stream=None) -> NF4Weight:
    _dev_bf16(W0, "W0")
    d, k = W0.shape
    w = out if out is not None else NF4Weight.empty(d, k, double_quant, W0.device)
    wsb = workspace_bytes(OP_QUANTIZE, d, k, 0, 0, double_quant)
    wst, wsn = _workspace(wsb, W0.device, ws)
    cw = w.c_struct()
    _check(lib().qlora_nf4_quantize(W0.data_ptr(), ctypes.byref(cw), _ptr(wst), wsn,
                                    _stream(stream)), "qlora_nf4_quantize")
    return w


def quantize_residual(W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, lora_alpha: float,
                      double_quant: bool = True, out: NF4Weight | None = None,
                      ws: torch.Tensor | None = None, stream=None) -> NF4Weight:
    """NF4 (+DQ) of bf16(W - (alpha/r) B A): the base of one LoftQ step."""
    for t, nm in ((W, "W"), (A, "A"), (B, "B")):
        _dev_bf16(t, nm)
    d, k = W.shape
    r = A.shape[0]
    w = out if out is not None else NF4Weight.empty(d, k, double_quant, W.device)
    wsb = workspace_bytes(OP_QUANTIZE_RESIDUAL, d, k, 0, r, double_quant)
    wst, wsn = _workspace(wsb, W.device, ws)
    cw = w.c_struct()
    _check(lib().qlora_nf4_quantize_residual(W.data_ptr(), A.data_ptr(), B.data_ptr(), r,
                                             float(lora_alpha), ctypes.byref(cw), _ptr(wst), wsn,
                                             _stream(stream)), "qlora_nf4_quantize_residual")
    return w


def loftq_init(W: torch.Tensor, omega: torch.Tensor, lora_alpha: float, iters: int = 1,
               power_iters: int = 4, double_quant: bool = True, ws: torch.Tensor | None = None,
               stream=None):
    """LoftQ: returns (NF4Weight, A (r x k bf16), B (d x r bf16), sigma (r fp32)).
    ``omega`` is the k x r float32 Gaussian test matrix (its column count is r)."""
    _dev_bf16(W, "W")
    if omega.dtype != torch.float32 or not omega.is_cuda or not omega.is_contiguous():
        raise ValueError("omega must be a contiguous float32 CUDA tensor")
    d, k = W.shape
    if omega.dim() != 2 or omega.shape[0] != k:
        raise ValueError("omega must be k x r")
    r = omega.shape[1]
    w = NF4Weight.empty(d, k, double_quant, W.device)
    A = torch.empty(r, k, dtype=torch.bfloat16, device=W.device)
    B = torch.empty(d, r, dtype=torch.bfloat16, device=W.device)
    sigma = torch.empty(r, dtype=torch.float32, device=W.device)
    wsb = workspace_bytes(OP_LOFTQ, d, k, 0, r, double_quant)
    wst, wsn = _workspace(wsb, W.device, ws)
    cw = w.c_struct()
    _check(lib().qlora_loftq_init(W.data_ptr(), omega.data_ptr(), r, float(lora_alpha), int(iters),
                                  int(power_iters), ctypes.byref(cw), A.data_ptr(), B.data_ptr(),
                                  sigma.data_ptr(), _ptr(wst), wsn, _stream(stream)),
           "qlora_loftq_init")
    return w, A, B, sigma


def dequantize(w: NF4Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    Y = out if out is not None else torch.empty(w.d, w.k, dtype=torch.bfloat16,
                                                device=w.codes.device)
    cw = w.c_struct()
    _check(lib().qlora_nf4_dequantize(ctypes.byref(cw), Y.data_ptr(), _stream(stream)),
           "qlora_nf4_dequantize")
    return Y


class LoraDropoutC(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("reserved", ctypes.c_uint32), ("seed", ctypes.c_uint64),
                ("mask", ctypes.c_void_p)]


def dropout_mask(M: int, k: int, device="cuda") -> torch.Tensor:
    """Buffer for the keep bits a forward stores for its backward (M*k/4 bytes)."""
    return torch.empty(M * k // 4, dtype=torch.uint8, device=device)


def _check_mask(mask, M: int, k: int):
    if mask is None:
        return
    if (mask.dtype != torch.uint8 or not mask.is_cuda or not mask.is_contiguous()
            or mask.numel() < M * k // 4):
        raise ValueError(f"mask: contiguous uint8 device tensor of at least {M * k // 4} "
                         "bytes (M*k/4) expected")


def linear_fwd(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
               lora_alpha: float, save_h: bool = True, Y: torch.Tensor | None = None,
               H: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None,
               dropout: float = 0.0, seed: int = 0, mask: torch.Tensor | None = None):
    """Y = X W'^T + (alpha/r) (X~ A^T) B^T with X~ the adapter input after
    dropout at rate `dropout` (keep bits from `seed`; 0 = none); with more than
    16 tokens the bits are also stored in `mask` (M*k/4 bytes, see
    dropout_mask) when given. Returns (Y, H or None)."""
    for t, nm in ((X, "X"), (A, "A"), (B, "B")):
        _dev_bf16(t, nm)
    M = X.shape[0]
    r = A.shape[0]
    if Y is None:
        Y = torch.empty(M, w.d, dtype=torch.bfloat16, device=X.device)
    if save_h and H is None:
        H = torch.empty(M, r, dtype=torch.float32, device=X.device)
    wsb = workspace_bytes(OP_FWD, w.d, w.k, M, r, w.double_quant)
    wst, wsn = _workspace(wsb, X.device, ws)
    cw = w.c_struct()
    if dropout:
        _check_mask(mask, M, w.k)
        dr = LoraDropoutC(float(dropout), 0, int(seed), _ptr(mask))
        _check(lib().qlora_linear_fwd_ex(ctypes.byref(cw), X.data_ptr(), M, A.data_ptr(),
                                         B.data_ptr(), r, float(lora_alpha), ctypes.addressof(dr),
                                         Y.data_ptr(), _ptr(H) if save_h else None, _ptr(wst),
                                         wsn, _stream(stream)), "qlora_linear_fwd_ex")
    else:
        _check(lib().qlora_linear_fwd(ctypes.byref(cw), X.data_ptr(), M, A.data_ptr(),
                                      B.data_ptr(), r, float(lora_alpha), Y.data_ptr(),
                                      _ptr(H) if save_h else None, _ptr(wst), wsn,
                                      _stream(stream)), "qlora_linear_fwd")
    return Y, (H if save_h else None)


NOALLOC_SCRATCH_BYTES = 16 << 20


def linear_fwd_noalloc(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                       lora_alpha: float, Y: torch.Tensor, H: torch.Tensor | None = None,
                       stream=None):
    """qlora_linear_fwd_noalloc: the forward into caller-given Y (and H)
    with the library's own 16 MiB device scratch instead of a workspace
    (nothing is allocated by the library or here)."""
    for t, nm in ((X, "X"), (A, "A"), (B, "B"), (Y, "Y")):
        _dev_bf16(t, nm)
    cw = w.c_struct()
    _check(lib().qlora_linear_fwd_noalloc(ctypes.byref(cw), X.data_ptr(), X.shape[0],
                                          A.data_ptr(), B.data_ptr(), A.shape[0],
                                          float(lora_alpha), Y.data_ptr(), _ptr(H),
                                          _stream(stream)), "qlora_linear_fwd_noalloc")
    return Y, H


def linear_fwd_multi(ws_: list, X: torch.Tensor, As: list, Bs: list, lora_alpha: float,
                     save_h: bool = True, Ys: list | None = None, ws: torch.Tensor | None = None,
                     stream=None, Hs: list | None = None):
    """Sibling projections: Y_i = X W_i'^T + (alpha/r) (X A_i^T) B_i^T for up
    to four weights reading the same X, in one call. Returns (Ys, Hs)."""
    nw = len(ws_)
    if not (1 <= nw <= 4) or len(As) != nw or len(Bs) != nw:
        raise ValueError("one to four weights, each with its A and B")
    _dev_bf16(X, "X")
    for i in range(nw):
        _dev_bf16(As[i], f"A[{i}]")
        _dev_bf16(Bs[i], f"B[{i}]")
    M, r = X.shape[0], As[0].shape[0]
    if Ys is None:
        Ys = [torch.empty(M, w.d, dtype=torch.bfloat16, device=X.device) for w in ws_]
    if save_h and Hs is None:
        Hs = [torch.empty(M, r, dtype=torch.float32, device=X.device) for _ in range(nw)]
    if not save_h:
        Hs = None
    dtot = sum(w.d for w in ws_)
    wsb = workspace_bytes(OP_FWD_MULTI, dtot, ws_[0].k, M, r, ws_[0].double_quant)
    wst, wsn = _workspace(wsb, X.device, ws)
    cws = [w.c_struct() for w in ws_]
    wp = (ctypes.c_void_p * nw)(*[ctypes.addressof(c) for c in cws])
    ap = (ctypes.c_void_p * nw)(*[a.data_ptr() for a in As])
    bp = (ctypes.c_void_p * nw)(*[b.data_ptr() for b in Bs])
    yp = (ctypes.c_void_p * nw)(*[y.data_ptr() for y in Ys])
    hp = (ctypes.c_void_p * nw)(*[h.data_ptr() for h in Hs]) if save_h else None
    _check(lib().qlora_linear_fwd_multi(wp, nw, X.data_ptr(), M, ap, bp, r, float(lora_alpha), yp,
                                        hp, _ptr(wst), wsn, _stream(stream)),
           "qlora_linear_fwd_multi")
    return Ys, Hs


def linear_bwd(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
               lora_alpha: float, dY: torch.Tensor, H: torch.Tensor | None = None,
               need_dx: bool = True, dX=None, dA=None, dB=None,
               ws: torch.Tensor | None = None, stream=None, dropout: float = 0.0, seed: int = 0,
               mask: torch.Tensor | None = None):
    """Returns (dX or None, dA, dB); `dropout`, `seed` and `mask` as given to the
    forward (with more than 16 tokens the forward stored the keep bits in
    `mask`, which the backward then reads instead of drawing them again)."""
    for t, nm in ((X, "X"), (A, "A"), (B, "B"), (dY, "dY")):
        _dev_bf16(t, nm)
    M = X.shape[0]
    r = A.shape[0]
    dev = X.device
    if need_dx and dX is None:
        dX = torch.empty(M, w.k, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(r, w.k, dtype=torch.bfloat16, device=dev)
    if dB is None:
        dB = torch.empty(w.d, r, dtype=torch.bfloat16, device=dev)
    wsb = workspace_bytes(OP_BWD, w.d, w.k, M, r, w.double_quant)
    wst, wsn = _workspace(wsb, dev, ws)
    cw = w.c_struct()
    if dropout:
        _check_mask(mask, M, w.k)
        dr = LoraDropoutC(float(dropout), 0, int(seed), _ptr(mask))
        _check(lib().qlora_linear_bwd_ex(ctypes.byref(cw), X.data_ptr(), M, A.data_ptr(),
                                         B.data_ptr(), r, float(lora_alpha), ctypes.addressof(dr),
                                         dY.data_ptr(), _ptr(H), _ptr(dX) if need_dx else None,
                                         dA.data_ptr(), dB.data_ptr(), _ptr(wst), wsn,
                                         _stream(stream)), "qlora_linear_bwd_ex")
    else:
        _check(lib().qlora_linear_bwd(ctypes.byref(cw), X.data_ptr(), M, A.data_ptr(),
                                      B.data_ptr(), r, float(lora_alpha), dY.data_ptr(), _ptr(H),
                                      _ptr(dX) if need_dx else None, dA.data_ptr(), dB.data_ptr(),
                                      _ptr(wst), wsn, _stream(stream)), "qlora_linear_bwd")
    return (dX if need_dx else None), dA, dB


def merge(w: NF4Weight, A: torch.Tensor, B: torch.Tensor, lora_alpha: float,
          out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev_bf16(A, "A")
    _dev_bf16(B, "B")
    r = A.shape[0]
    Wm = out if out is not None else torch.empty(w.d, w.k, dtype=torch.bfloat16,
                                                 device=A.device)
    cw = w.c_struct()
    _check(lib().qlora_merge(ctypes.byref(cw), A.data_ptr(), B.data_ptr(), r,
                             float(lora_alpha), Wm.data_ptr(), _stream(stream)), "qlora_merge")
    return Wm


class AdamWHParamsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double)]


def adamw_step(param: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
               grad: torch.Tensor, param_bf16: torch.Tensor, step: int, lr: float = 2e-4,
               beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.0, stream=None):
    """One AdamW step in place on (param, exp_avg, exp_avg_sq) (float32) with
    the bf16 gradient, writing the bf16 copy of the updated parameter.

    The float32 state may be CUDA tensors or page-locked host tensors
    (``pin_memory=True``; the paged-out state), which the kernel reads and
    writes in place over the host link."""
    n = param.numel()
    for t, name in ((param, "param"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq")):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be a CUDA tensor or page-locked host memory")
    for t, name in ((grad, "grad"), (param_bf16, "param_bf16")):
        _dev_bf16(t, name)
        if t.numel() != n:
            raise ValueError(f"{name} must have {n} elements")
    hp = AdamWHParamsC(lr, beta1, beta2, eps, weight_decay)
    _check(lib().qlora_adamw_step(_ptr(param), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(grad),
                                  _ptr(param_bf16), n, ctypes.addressof(hp), int(step),
                                  _stream(stream)), "qlora_adamw_step")


def _page(fn: str, dst, src, stream):
    if len(dst) != len(src) or not 1 <= len(dst) <= 3:
        raise ValueError("dst and src must list the same 1 to 3 buffers")
    n = dst[0].numel()
    for t in list(dst) + list(src):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"every buffer must be a contiguous float32 tensor of {n} elements")
    arr = ctypes.c_void_p * len(dst)
    d = arr(*[t.data_ptr() for t in dst])
    s = arr(*[t.data_ptr() for t in src])
    _check(getattr(lib(), fn)(d, s, len(dst), n, _stream(stream)), fn)


def adamw_page_out(host, dev, stream=None):
    """Enqueue copies of the optimiser state ``dev`` (CUDA float32 tensors:
    param, exp_avg, exp_avg_sq or a subset) into the page-locked host
    tensors ``host`` on the stream."""
    _page("qlora_adamw_page_out", host, dev, stream)


def adamw_page_in(dev, host, stream=None):
    """Enqueue copies of the paged-out state ``host`` (page-locked float32
    tensors) back into the CUDA tensors ``dev`` on the stream."""
    _page("qlora_adamw_page_in", dev, host, stream)


# ---------------------------------------------------------------------------
# many adapters on one base weight (include/qlora_adapters.h)
def _device_tensors(*named):
    """Every (tensor, name, dtype, shape) contiguous, of that type and shape,
    and on the current device (the one the stream belongs to)."""
    dev = named[0][0].get_device()
    for t, name, dtype, shape in named:
        if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
                or t.get_device() != dev or dev < 0):
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape "
                             f"{tuple(shape)} on the device of {named[0][1]}")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{named[0][1]} is on cuda:{dev}, not on the current device")
    return dev


def _beside(dev, *others):
    """Every (tensor, name) is on device number dev."""
    for t, name in others:
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev} like the call's other tensors")


def _on(stream):
    """Context in which what a call allocates belongs to its stream."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class AdapterPlanC(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("n", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("data", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class AdaptersC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("r", ctypes.c_int32), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


@dataclass
class AdapterPlan:
    """Which of ``n`` adapters each of ``M`` tokens uses, laid out on the
    device for the many-adapter linears of one batch (``adapter_plan``)."""
    M: int
    n: int
    data: torch.Tensor

    def c_struct(self) -> AdapterPlanC:
        return AdapterPlanC(self.M, self.n, 0, self.data.data_ptr(), self.data.nbytes)


def adapter_plan(ids: torch.Tensor, n: int, out: AdapterPlan | None = None,
                 stream=None) -> AdapterPlan:
    """Plan of a batch: ids (int32, one per token) is the adapter of each
    token, any value outside [0, n) meaning none. Built on the device in one
    launch; every linear the batch passes takes the same plan. ``out`` (a plan
    of the same M and n) is rebuilt in place."""
    M = ids.numel()
    _device_tensors((ids, "ids", torch.int32, (M,)))
    if out is None:
        nbytes = int(lib().qlora_adapter_plan_bytes(M, n))
        if nbytes == 0:
            raise QLoRAError(QLORA_ERR_UNSUPPORTED if M and n > 0 else QLORA_ERR_INVALID_ARG,
                             "adapter_plan")
        with _on(stream):
            out = AdapterPlan(M, n, torch.empty(nbytes, dtype=torch.uint8, device=ids.device))
    elif out.M != M or out.n != n:
        raise ValueError(f"out is a plan of {out.M} tokens and {out.n} adapters, not {M} and {n}")
    else:
        _beside(ids.get_device(), (out.data, "out"))
    c = out.c_struct()
    _check(lib().qlora_adapter_plan_build(ids.data_ptr(), ctypes.addressof(c), _stream(stream)),
           "qlora_adapter_plan_build")
    return out


def adapters_workspace_bytes(op: int, d: int, k: int, M: int, n: int, r: int) -> int:
    b = lib().qlora_adapters_workspace_bytes(op, d, k, M, n, r)
    if b == ctypes.c_size_t(-1).value:
        raise QLoRAError(QLORA_ERR_UNSUPPORTED, "adapters_workspace_bytes")
    return int(b)


def adapters_workspace(plan: AdapterPlan, d: int, k: int, r: int,
                       backward: bool = False) -> torch.Tensor:
    """Workspace of the forward (and of the backward too, when asked) of a
    d x k weight for the plan's batch; calls on one stream can share it."""
    b = adapters_workspace_bytes(OP_FWD, d, k, plan.M, plan.n, r)
    if backward:
        b = max(b, adapters_workspace_bytes(OP_BWD, d, k, plan.M, plan.n, r))
    return _workspace(b, plan.data.device, None)[0]


def _adapter_rank(A, plan: AdapterPlan) -> int:
    if A.dim() != 3:
        raise ValueError("A must be n x r x k")
    if plan.n != A.shape[0]:
        raise ValueError(f"the plan is for {plan.n} adapters, A holds {A.shape[0]}")
    return A.shape[1]


def _adapter_args(w: NF4Weight, X, A, B, scale, plan: AdapterPlan, r: int, ws, *more):
    """Checks of a call's tensors (``more`` as in ``_device_tensors``); its adapters."""
    n, k, bf = plan.n, w.k, torch.bfloat16
    dev = _device_tensors((X, "X", bf, (plan.M, k)), (A, "A", bf, (n, r, k)),
                          (B, "B", bf, (n, w.d, r)), (scale, "scale", torch.float32, (n,)), *more)
    _beside(dev, (w.codes, "w"), (plan.data, "plan"), (ws, "ws"))
    return AdaptersC(n, r, A.data_ptr(), B.data_ptr(), scale.data_ptr())


def linear_fwd_adapters(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        scale: torch.Tensor, plan: AdapterPlan, save_h: bool = True,
                        Y: torch.Tensor | None = None, H: torch.Tensor | None = None,
                        ws: torch.Tensor | None = None, stream=None):
    """Y[m] = X[m] W'^T + s_a (X[m] A_a^T) B_a^T with a the adapter of token m
    in ``plan``: A (n x r x k), B (n x d x r) bf16, scale (n) float32 holding
    s_a. Returns (Y, H or None); H (M x r float32) is what the backward needs."""
    r = _adapter_rank(A, plan)
    if Y is None or ws is None or (save_h and H is None):
        with _on(stream):
            if Y is None:
                Y = torch.empty(plan.M, w.d, dtype=torch.bfloat16, device=X.device)
            if save_h and H is None:
                H = torch.empty(plan.M, r, dtype=torch.float32, device=X.device)
            if ws is None:
                ws = adapters_workspace(plan, w.d, w.k, r)
    y = (Y, "Y", torch.bfloat16, (plan.M, w.d))
    if save_h:
        ad = _adapter_args(w, X, A, B, scale, plan, r, ws, y, (H, "H", torch.float32, (plan.M, r)))
    else:
        H = None
        ad = _adapter_args(w, X, A, B, scale, plan, r, ws, y)
    cw, cp = w.c_struct(), plan.c_struct()
    _check(lib().qlora_linear_fwd_adapters(ctypes.byref(cw), X.data_ptr(), ctypes.addressof(ad),
                                           ctypes.addressof(cp), Y.data_ptr(), _ptr(H),
                                           ws.data_ptr(), ws.nbytes, _stream(stream)),
           "qlora_linear_fwd_adapters")
    return Y, H


def linear_bwd_adapters(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        scale: torch.Tensor, plan: AdapterPlan, dY: torch.Tensor,
                        H: torch.Tensor | None = None, need_dx: bool = True, dX=None, dA=None,
                        dB=None, ws: torch.Tensor | None = None, stream=None):
    """Backward of ``linear_fwd_adapters``: (dX or None, dA (n x r x k), dB
    (n x d x r)); adapters without tokens get zero gradients. H as the forward
    returned it, or None to recompute it."""
    r = _adapter_rank(A, plan)
    with _on(stream):
        if need_dx and dX is None:
            dX = torch.empty_like(X)
        if dA is None:
            dA = torch.empty_like(A)
        if dB is None:
            dB = torch.empty_like(B)
        if ws is None:
            ws = adapters_workspace(plan, w.d, w.k, r, backward=True)
    more = [(dY, "dY", torch.bfloat16, (plan.M, w.d)), (dA, "dA", torch.bfloat16, A.shape),
            (dB, "dB", torch.bfloat16, B.shape)]
    if need_dx:
        more.append((dX, "dX", torch.bfloat16, X.shape))
    if H is not None:
        more.append((H, "H", torch.float32, (plan.M, r)))
    ad = _adapter_args(w, X, A, B, scale, plan, r, ws, *more)
    cw, cp = w.c_struct(), plan.c_struct()
    _check(lib().qlora_linear_bwd_adapters(ctypes.byref(cw), X.data_ptr(), ctypes.addressof(ad),
                                           ctypes.addressof(cp), dY.data_ptr(), _ptr(H),
                                           dX.data_ptr() if need_dx else None, dA.data_ptr(),
                                           dB.data_ptr(), ws.data_ptr(), ws.nbytes,
                                           _stream(stream)), "qlora_linear_bwd_adapters")
    return (dX if need_dx else None), dA, dB


# ---------------------------------------------------------------------------
# log probabilities of given tokens (include/qlora_logprobs.h)
class LogitsC(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("N", ctypes.c_int64), ("V", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


MAX_TOP = 32
_LOGITS_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


@dataclass
class TokenLogprobs:
    """What ``token_logprobs`` computes for N rows of logits."""
    logprob: torch.Tensor                       # float32 [N]
    entropy: torch.Tensor                       # float32 [N]
    stats: torch.Tensor                         # float32 [N, 2]: row maximum, log of the sum
    top_logprobs: torch.Tensor | None = None    # float32 [N, top]
    top_ids: torch.Tensor | None = None         # int64 [N, top]

    @staticmethod
    def empty(N: int, top: int = 0, device="cuda") -> "TokenLogprobs":
        f = dict(dtype=torch.float32, device=device)
        out = TokenLogprobs(torch.empty(N, **f), torch.empty(N, **f), torch.empty(N, 2, **f))
        if top:
            out.top_logprobs = torch.empty(N, top, **f)
            out.top_ids = torch.empty(N, top, dtype=torch.int64, device=device)
        return out


def _logits(t: torch.Tensor, name: str) -> LogitsC:
    dtype = _LOGITS_DTYPES.get(t.dtype)
    if t.dim() != 2 or dtype is None or not t.is_cuda:
        raise ValueError(f"{name} must be a two-dimensional bfloat16 or float32 CUDA tensor")
    N, V = t.shape
    ld, step = t.stride()
    if N == 1:
        ld = max(V, ld)
    if (V > 1 and step != 1) or ld < V:
        raise ValueError(f"{name} must have rows of consecutive elements that do not overlap")
    return LogitsC(t.data_ptr(), N, V, ld, dtype, 0)


def logprobs_workspace(logits: torch.Tensor, top: int = 0) -> torch.Tensor | None:
    """Workspace of ``token_logprobs`` for logits of this shape (None: none needed)."""
    b = lib().qlora_token_logprobs_workspace_bytes(logits.shape[0], logits.shape[1],
                                                   _LOGITS_DTYPES.get(logits.dtype, -1), top)
    if b == ctypes.c_size_t(-1).value:
        raise QLoRAError(QLORA_ERR_UNSUPPORTED, "logprobs_workspace")
    return _workspace(int(b), logits.device, None)[0]


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top: int = 0,
                   out: TokenLogprobs | None = None, ws: torch.Tensor | None = None,
                   stream=None) -> TokenLogprobs:
    """Per row of logits (N x V bf16 or float32, rows at any stride, the first of
    them 16-byte aligned; a view that starts elsewhere is refused): the log
    probability of its target (int64; outside [0, V): ignored, 0), the
    entropy, and the ``top`` (0..32) best alternatives by value, then index."""
    c = _logits(logits, "logits")
    N = c.N
    if not 0 <= top <= min(c.V, MAX_TOP):
        raise QLoRAError(QLORA_ERR_UNSUPPORTED, f"token_logprobs(top={top})")
    if out is None or ws is None:
        with _on(stream):
            if out is None:
                out = TokenLogprobs.empty(N, top, logits.device)
            if ws is None:
                ws = logprobs_workspace(logits, top)
    f32 = torch.float32
    checks = ((targets, "targets", torch.int64, (N,)), (out.logprob, "out.logprob", f32, (N,)),
              (out.entropy, "out.entropy", f32, (N,)), (out.stats, "out.stats", f32, (N, 2)))
    if top:
        if out.top_logprobs is None or out.top_ids is None:
            raise ValueError(f"out has no top_logprobs and top_ids for top={top}")
        checks += ((out.top_logprobs, "out.top_logprobs", f32, (N, top)),
                   (out.top_ids, "out.top_ids", torch.int64, (N, top)))
    dev = _device_tensors(*checks)
    _beside(dev, (logits, "logits"))
    if ws is not None:
        _beside(dev, (ws, "ws"))
    _check(lib().qlora_token_logprobs(ctypes.addressof(c), targets.data_ptr(),
                                      out.logprob.data_ptr(), out.stats.data_ptr(),
                                      out.entropy.data_ptr(), top,
                                      out.top_logprobs.data_ptr() if top else None,
                                      out.top_ids.data_ptr() if top else None, _ptr(ws),
                                      0 if ws is None else ws.nbytes, _stream(stream)),
           "qlora_token_logprobs")
    return out


def token_logprobs_bwd(logits: torch.Tensor, targets: torch.Tensor, lp: TokenLogprobs,
                       dlogprob: torch.Tensor, dentropy: torch.Tensor | None = None,
                       dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of the logits for upstream gradients of ``lp.logprob`` and
    (optional) ``lp.entropy``, with ``lp`` as the forward returned it.
    ``dlogits`` may be ``logits`` itself, which is then overwritten."""
    c = _logits(logits, "logits")
    N = c.N
    if dlogits is None:
        with _on(stream):
            dlogits = torch.empty(N, c.V, dtype=logits.dtype, device=logits.device)
    co = _logits(dlogits, "dlogits")
    if (co.N, co.V, co.dtype) != (N, c.V, c.dtype):
        raise ValueError("dlogits must have the shape and type of logits")
    checks = ((targets, "targets", torch.int64, (N,)),
              (lp.stats, "lp.stats", torch.float32, (N, 2)),
              (lp.entropy, "lp.entropy", torch.float32, (N,)),
              (dlogprob, "dlogprob", torch.float32, (N,)))
    if dentropy is not None:
        checks += ((dentropy, "dentropy", torch.float32, (N,)),)
    _beside(_device_tensors(*checks), (logits, "logits"), (dlogits, "dlogits"))
    _check(lib().qlora_token_logprobs_bwd(ctypes.addressof(c), targets.data_ptr(),
                                          lp.stats.data_ptr(), lp.entropy.data_ptr(),
                                          dlogprob.data_ptr(), _ptr(dentropy),
                                          ctypes.addressof(co), _stream(stream)),
           "qlora_token_logprobs_bwd")
    return dlogits


def profile_begin(cap: int = 4096, kernels=None):
    """Start bracketing kernel launches of the timing build with HIP events
    (include/qlora_nf4_timing.h); only calls made inside ``timing_build()``
    are seen;
    ``kernels`` (names from KERNELS) limits the bracketing to those kernels."""
    mask = 0
    for name in kernels or ():
        mask |= 1 << KERNELS.index(name)
    _check(timing_lib().qlora_profile_begin(int(cap), mask), "qlora_profile_begin")


def profile_end():
    _check(timing_lib().qlora_profile_end(), "qlora_profile_end")


def profile_query(kernel: str):
    """(launch count, total milliseconds) of a kernel since profile_begin."""
    cnt = ctypes.c_int32(0)
    ms = ctypes.c_double(0.0)
    _check(timing_lib().qlora_profile_query(KERNELS.index(kernel), ctypes.byref(cnt),
                                     ctypes.byref(ms)), "qlora_profile_query")
    return int(cnt.value), float(ms.value)


__all__ = ["NF4Weight", "QLoRAError", "quantize", "dequantize", "linear_fwd", "linear_bwd",
           "merge", "storage_bytes", "workspace_bytes", "codebook", "lib",
           "OP_QUANTIZE", "OP_FWD", "OP_BWD", "SIGNATURES", "LIB_PATH", "KERNELS",
           "profile_begin", "profile_end", "profile_query", "timing_build", "timing_lib",
           "TIMING_LIB_PATH", "AdapterPlan", "adapter_plan", "adapters_workspace",
           "adapters_workspace_bytes", "linear_fwd_adapters", "linear_bwd_adapters",
           "TokenLogprobs", "token_logprobs", "token_logprobs_bwd", "logprobs_workspace"]
