"""ctypes binding of the C ABI in include/qfp4.h (argument marshalling only).

Every step of the quantizers, GEMMs and linear layer runs in the sm_100a CUDA
library ``libqfp4.so`` built from ``csrc/``; PyTorch provides device memory
and streams. There is no fallback: if the library is missing or the device is
not a B200 the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QFP4_BOUNDS_CHECK=1 selects the bounds-checked build (libqfp4_bc.so): the
# same kernels with every store address checked, reported by qfp4_status
LIB_PATH = os.path.join(_HERE, "libqfp4_bc.so" if os.environ.get("QFP4_BOUNDS_CHECK") == "1" else "libqfp4.so")

NVFP4, MXFP4, MXFP4_RU = 0, 1, 2
RTN, SR, QUARTET2 = 0, 1, 2
HAD_NONE, HAD_DET16, HAD_DET32, HAD_RAND16, HAD_RAND32 = 0, 1, 2, 3, 4
ROW, COL = 0, 1
OUT_BF16, OUT_F32 = 0, 1
PRESETS = {"NVIDIA_NVFP4": 0, "QUARTET2_NVFP4": 1, "AMD_MXFP4_H": 2}
BLOCK = {NVFP4: 16, MXFP4: 32, MXFP4_RU: 32}

OK, ERR_INVALID_ARG, ERR_MISALIGNED, ERR_UNSUPPORTED_ARCH, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6
ERR_TOO_LARGE = -7
ERR_BOUNDS = -8
ERR_OFFSETS = -9
NOALLOC_SCRATCH_BYTES = 32 << 20
ROUND_E2M1_SR, ROUND_E2M1_RN, ROUND_E4M3_SR, ROUND_E4M3_RN, ROUND_E8M0_SR = 0, 1, 2, 3, 4


class Seed(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_uint64), ("sr", ctypes.c_uint64), ("rot_stream", ctypes.c_uint32),
                ("sr_stream", ctypes.c_uint32)]


class TensorDesc(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("fmt", ctypes.c_int32), ("had", ctypes.c_int32),
                ("rot_seed", ctypes.c_uint64), ("rot_stream", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class GemmCfg(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("rnd_a", ctypes.c_int32), ("rnd_b", ctypes.c_int32), ("had", ctypes.c_int32)]


class Recipe(ctypes.Structure):
    _fields_ = [("fprop", GemmCfg), ("dgrad", GemmCfg), ("wgrad", GemmCfg), ("y_dtype", ctypes.c_int32),
                ("dx_dtype", ctypes.c_int32), ("dw_dtype", ctypes.c_int32), ("dw_accumulate", ctypes.c_int32)]


class QFP4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = lib().qfp4_strerror(status).decode()
        if status == ERR_CUDA:
            msg += f" (cudaError {lib().qfp4_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")
        self.status = status


_lib = None
_VOID, _I32, _I64, _U64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t
_F32 = ctypes.c_float

_SIGNATURES = {
    "qfp4_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "qfp4_last_cuda_error": (ctypes.c_int, []),
    "qfp4_codes_bytes": (_SZ, [_I64, _I64]),
    "qfp4_scales_bytes": (_SZ, [_I32, _I64, _I64]),
    "qfp4_scale_offset": (_I64, [_I32, _I64, _I64, _I64, _I64]),
    "qfp4_quantize_workspace_bytes": (_SZ, []),
    "qfp4_amax": (ctypes.c_int, [_VOID, _I64, _I64, _I64, _I32, _I32, ctypes.POINTER(Seed), _VOID, _VOID, _SZ, _VOID]),
    "qfp4_amax_rowcol": (ctypes.c_int, [_VOID, _I64, _I64, _I64, _I32, _I32, ctypes.POINTER(Seed), ctypes.POINTER(Seed),
                                        _VOID, _VOID, _VOID, _SZ, _VOID]),
    "qfp4_quantize": (ctypes.c_int, [_VOID, _I64, _I64, _I64, _I32, _I32, _I32, _I32, ctypes.POINTER(Seed), _VOID,
                                     ctypes.POINTER(TensorDesc), _VOID, _SZ, _VOID]),
    "qfp4_quantize_dual": (ctypes.c_int, [_VOID, _I64, _I64, _I64, _I32, _I32, _I32, _I32, ctypes.POINTER(Seed),
                                          ctypes.POINTER(Seed), _VOID, _VOID, ctypes.POINTER(TensorDesc),
                                          ctypes.POINTER(TensorDesc), _VOID]),
    "qfp4_gemm": (ctypes.c_int, [ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), _VOID, _I64, _I32, _VOID]),
    "qfp4_gemm_quantize": (ctypes.c_int, [ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), _VOID, _I64, _I32,
                                          ctypes.POINTER(Seed), ctypes.POINTER(TensorDesc), _VOID]),
    "qfp4_gemm_accumulate": (ctypes.c_int, [ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), _VOID, _I64,
                                            _VOID]),
    "qfp4_gemm_amax": (ctypes.c_int, [ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), _VOID, _I64, _I32,
                                      ctypes.POINTER(Seed), _VOID, _VOID, _SZ, _VOID]),
    "qfp4_recipe_preset": (ctypes.c_int, [_I32, ctypes.POINTER(Recipe)]),
    "qfp4_linear_workspace_bytes": (_SZ, [_I32, _I64, _I64, _I64, ctypes.POINTER(Recipe)]),
    "qfp4_linear_fwd": (ctypes.c_int, [_VOID, _VOID, _VOID, _I64, _I64, _I64, ctypes.POINTER(Recipe),
                                       ctypes.POINTER(Seed), _VOID, _SZ, _VOID]),
    "qfp4_linear_bwd": (ctypes.c_int, [_VOID, _VOID, _VOID, _VOID, _VOID, _I64, _I64, _I64, ctypes.POINTER(Recipe),
                                       ctypes.POINTER(Seed), _VOID, _SZ, _VOID]),
    "qfp4_linear_fwd_chain": (ctypes.c_int, [_VOID, _VOID, _VOID, _I64, _I64, _I64, ctypes.POINTER(Recipe),
                                             ctypes.POINTER(Seed), _VOID, _I32, ctypes.POINTER(Seed), _VOID, _VOID,
                                             _SZ, _VOID]),
    "qfp4_linear_fwd_noalloc": (ctypes.c_int, [_VOID, _VOID, _VOID, _I64, _I64, _I64, ctypes.POINTER(Recipe),
                                               ctypes.POINTER(Seed), _VOID]),
    "qfp4_rmsnorm_fwd": (ctypes.c_int, [_VOID, _I64, _VOID, _I64, _VOID, _I64, _I64, _F32, _VOID, _I64, _VOID, _I64,
                                        _VOID, _I32, ctypes.POINTER(Seed), _VOID, _VOID, _SZ, _VOID]),
    "qfp4_rmsnorm_quantize": (ctypes.c_int, [_VOID, _I64, _VOID, _I64, _VOID, _I64, _I64, _F32, _VOID, _I64, _VOID,
                                             _I64, _VOID, _I32, _I32, ctypes.POINTER(Seed), ctypes.POINTER(TensorDesc),
                                             _VOID]),
    "qfp4_rmsnorm_bwd_workspace_bytes": (_SZ, [_I64, _I64]),
    "qfp4_rmsnorm_bwd": (ctypes.c_int, [_VOID, _I64, _VOID, _I64, _VOID, _VOID, _VOID, _I64, _I64, _I64, _VOID, _I64,
                                        _VOID, _I32, _VOID, _SZ, _VOID]),
    "qfp4_group_rows": (_I64, [_I64, _I32]),
    "qfp4_quantize_grouped": (ctypes.c_int, [_VOID, _I64, _I64, _I64, _VOID, _I32, _I32, _I32, _I32, _I32,
                                             ctypes.POINTER(Seed), _VOID, ctypes.POINTER(TensorDesc), _VOID, _SZ,
                                             _VOID]),
    "qfp4_gemm_grouped": (ctypes.c_int, [ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), _VOID, _I32, _I64,
                                         _VOID, _I64, _I32, _VOID]),
    "qfp4_gemm_grouped_wgrad": (ctypes.c_int, [ctypes.POINTER(TensorDesc), ctypes.POINTER(TensorDesc), _VOID, _I32,
                                               _I64, _VOID, _I32, _I32, _VOID]),
    "qfp4_linear_grouped_workspace_bytes": (_SZ, [_I32, _I64, _I32, _I64, _I64, ctypes.POINTER(Recipe)]),
    "qfp4_linear_grouped_fwd": (ctypes.c_int, [_VOID, _VOID, _VOID, _VOID, _I32, _I64, _I64, _I64,
                                               ctypes.POINTER(Recipe), ctypes.POINTER(Seed), _VOID, _VOID, _SZ, _VOID]),
    "qfp4_linear_grouped_bwd": (ctypes.c_int, [_VOID, _VOID, _VOID, _VOID, _VOID, _VOID, _I32, _I64, _I64, _I64,
                                               ctypes.POINTER(Recipe), ctypes.POINTER(Seed), _VOID, _SZ, _VOID]),
    "qfp4_status": (ctypes.c_int, [_VOID]),
    "qfp4_selftest_wait_timeout": (ctypes.c_int, [_I64, _VOID]),
    "qfp4_selftest_rounding": (ctypes.c_int, [_I32, _VOID, _VOID, _VOID, _I64, _VOID]),
    "qfp4_launch_count": (_I64, [_I32]),
}


def lib() -> ctypes.CDLL:
    """Load libqfp4.so (built by ``fp4_precision_b200.build``). Raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m fp4_precision_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != OK:
        raise QFP4Error(status, what)


# The current device and its stream without the objects around them, at every
# call; torch's public calls where a version does not have these.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        torch.cuda.init()
        return ctypes.c_void_p(_current_stream(_current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t: torch.Tensor | None) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def make_seed(rot: int = 0, sr: int = 0, rot_stream: int = 0, sr_stream: int = 0) -> Seed:
    return Seed(rot, sr, rot_stream, sr_stream)


# ---------------------------------------------------------------------------
# sizes / layout helpers (host only)

def codes_bytes(rows: int, k: int) -> int:
    return lib().qfp4_codes_bytes(rows, k)


def scales_bytes(fmt: int, rows: int, k: int) -> int:
    return lib().qfp4_scales_bytes(fmt, rows, k)


def scale_offset(fmt: int, rows: int, k: int, r: int, c: int) -> int:
    return lib().qfp4_scale_offset(fmt, rows, k, r, c)


def quantize_workspace_bytes() -> int:
    return lib().qfp4_quantize_workspace_bytes()


def launch_count(reset: bool = False) -> int:
    return lib().qfp4_launch_count(1 if reset else 0)


# ---------------------------------------------------------------------------
@dataclass
class QTensor:
    """A quantized operand in device memory (see qfp4_tensor in include/qfp4.h)."""
    codes: torch.Tensor         # uint8 [rows, k/2]
    scales: torch.Tensor        # uint8 [scales_bytes], MMA atom layout
    tensor_scale: torch.Tensor  # float32 [1]
    desc: TensorDesc

    @property
    def rows(self) -> int:
        return self.desc.rows

    @property
    def k(self) -> int:
        return self.desc.k

    @property
    def fmt(self) -> int:
        return self.desc.fmt


def empty_qtensor(fmt: int, rows: int, k: int, device) -> QTensor:
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=device)
    scales = torch.empty((max(scales_bytes(fmt, rows, k), 16),), dtype=torch.uint8, device=device)
    ts = torch.empty((1,), dtype=torch.float32, device=device)
    desc = TensorDesc(codes.data_ptr(), scales.data_ptr(), ts.data_ptr(), 0, 0, 0, 0, 0, 0, 0)
    return QTensor(codes, scales, ts, desc)


def amax(x: torch.Tensor, had: int = HAD_NONE, axis: int = ROW, seed: Seed | None = None, out=None,
         workspace=None, stream=None) -> torch.Tensor:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    R, C = x.shape
    out = torch.empty((1,), dtype=torch.float32, device=x.device) if out is None else out
    ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=x.device) if workspace is None else workspace
    seed = seed or make_seed()
    _check(lib().qfp4_amax(_ptr(x), R, C, x.stride(0), had, axis, ctypes.byref(seed), _ptr(out), _ptr(ws),
                           ws.numel(), _stream(stream)), "qfp4_amax")
    return out


def amax_rowcol(x: torch.Tensor, had: int, seed_row: Seed | None = None, seed_col: Seed | None = None, out=None,
                workspace=None, stream=None, had_col: int | None = None) -> torch.Tensor:
    """Both orientations' tensor amax in one call: out[0] as amax(x, had, ROW,
    seed_row), out[1] as amax(x, had_col (default had), COL, seed_col)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    R, C = x.shape
    out = torch.empty((2,), dtype=torch.float32, device=x.device) if out is None else out
    ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=x.device) if workspace is None else workspace
    seed_row = seed_row or make_seed()
    seed_col = seed_col or make_seed()
    had_col = had if had_col is None else had_col
    _check(lib().qfp4_amax_rowcol(_ptr(x), R, C, x.stride(0), had, had_col, ctypes.byref(seed_row),
                                  ctypes.byref(seed_col),
                                  _ptr(out), ctypes.c_void_p(out.data_ptr() + 4), _ptr(ws), ws.numel(),
                                  _stream(stream)), "qfp4_amax_rowcol")
    return out


def quantize(x: torch.Tensor, fmt: int, rounding: int, had: int, axis: int, seed: Seed | None = None,
             amax_in: torch.Tensor | None = None, out: QTensor | None = None, workspace=None,
             stream=None) -> QTensor:
    """Quantize a bf16 matrix (row stride x.stride(0)); see qfp4_quantize."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    R, C = x.shape
    rows, k = (R, C) if axis == ROW else (C, R)
    out = empty_qtensor(fmt, rows, k, x.device) if out is None else out
    ws = workspace
    if ws is None:
        ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=x.device)
    seed = seed or make_seed()
    _check(lib().qfp4_quantize(_ptr(x), R, C, x.stride(0), fmt, rounding, had, axis, ctypes.byref(seed),
                               _ptr(amax_in), ctypes.byref(out.desc), _ptr(ws), ws.numel(), _stream(stream)),
           "qfp4_quantize")
    return out


def quantize_dual(x: torch.Tensor, fmt: int, rounding: int, had_row: int, had_col: int, seed_row: Seed,
                  seed_col: Seed, amax_row: torch.Tensor | None = None, amax_col: torch.Tensor | None = None,
                  out_row: QTensor | None = None, out_col: QTensor | None = None, stream=None):
    """Row and column quantization of a bf16 matrix from one read; see qfp4_quantize_dual."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    R, C = x.shape
    out_row = empty_qtensor(fmt, R, C, x.device) if out_row is None else out_row
    out_col = empty_qtensor(fmt, C, R, x.device) if out_col is None else out_col
    _check(lib().qfp4_quantize_dual(_ptr(x), R, C, x.stride(0), fmt, rounding, had_row, had_col,
                                    ctypes.byref(seed_row), ctypes.byref(seed_col), _ptr(amax_row), _ptr(amax_col),
                                    ctypes.byref(out_row.desc), ctypes.byref(out_col.desc), _stream(stream)),
           "qfp4_quantize_dual")
    return out_row, out_col


def gemm(A: QTensor, B: QTensor, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """D = gA gB A . B^T (A.rows x B.rows); see qfp4_gemm."""
    dt = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    if out is None:
        out = torch.empty((A.rows, B.rows), dtype=out_dtype, device=A.codes.device)
    _check(lib().qfp4_gemm(ctypes.byref(A.desc), ctypes.byref(B.desc), _ptr(out), out.stride(0), dt,
                           _stream(stream)), "qfp4_gemm")
    return out


def gemm_quantize(A: QTensor, B: QTensor, had: int, seed: Seed, out: torch.Tensor | None = None,
                  qout: QTensor | None = None, stream=None):
    """bf16 D = gA gB A . B^T and its MXFP4 quantization along N; see qfp4_gemm_quantize."""
    if out is None:
        out = torch.empty((A.rows, B.rows), dtype=torch.bfloat16, device=A.codes.device)
    qout = empty_qtensor(MXFP4, A.rows, B.rows, A.codes.device) if qout is None else qout
    _check(lib().qfp4_gemm_quantize(ctypes.byref(A.desc), ctypes.byref(B.desc), _ptr(out), out.stride(0), had,
                                    ctypes.byref(seed), ctypes.byref(qout.desc), _stream(stream)),
           "qfp4_gemm_quantize")
    return out, qout


def gemm_amax(A: QTensor, B: QTensor, had: int, seed: Seed | None = None, out: torch.Tensor | None = None,
              amax: torch.Tensor | None = None, workspace=None, stream=None):
    """bf16 D = gA gB A . B^T and the NVFP4 tensor amax of D along its rows
    after the rotation `had`; see qfp4_gemm_amax. Returns (D, amax)."""
    if out is None:
        out = torch.empty((A.rows, B.rows), dtype=torch.bfloat16, device=A.codes.device)
    amax = torch.empty((1,), dtype=torch.float32, device=A.codes.device) if amax is None else amax
    ws = workspace
    if ws is None:
        ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=A.codes.device)
    seed = seed or make_seed()
    _check(lib().qfp4_gemm_amax(ctypes.byref(A.desc), ctypes.byref(B.desc), _ptr(out), out.stride(0), had,
                                ctypes.byref(seed), _ptr(amax), _ptr(ws), ws.numel(), _stream(stream)),
           "qfp4_gemm_amax")
    return out, amax


def gemm_accumulate(A: QTensor, B: QTensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    """out += gA gB A . B^T in fp32 (A.rows x B.rows); see qfp4_gemm_accumulate."""
    assert out.dtype == torch.float32 and out.dim() == 2 and out.stride(1) == 1
    _check(lib().qfp4_gemm_accumulate(ctypes.byref(A.desc), ctypes.byref(B.desc), _ptr(out), out.stride(0),
                                      _stream(stream)), "qfp4_gemm_accumulate")
    return out


def recipe(name: str, dw_fp32: bool = True) -> Recipe:
    r = Recipe()
    _check(lib().qfp4_recipe_preset(PRESETS[name], ctypes.byref(r)), "qfp4_recipe_preset")
    r.dw_dtype = OUT_F32 if dw_fp32 else OUT_BF16
    return r


def linear_workspace_bytes(backward: bool, M: int, N: int, K: int, rec: Recipe) -> int:
    return lib().qfp4_linear_workspace_bytes(1 if backward else 0, M, N, K, ctypes.byref(rec))


def _dtype(code: int):
    return torch.float32 if code == OUT_F32 else torch.bfloat16


def linear_fwd(X, W, rec: Recipe, seed: Seed, Y=None, workspace=None, stream=None) -> torch.Tensor:
    M, K = X.shape
    N = W.shape[0]
    Y = torch.empty((M, N), dtype=_dtype(rec.y_dtype), device=X.device) if Y is None else Y
    if workspace is None:
        workspace = torch.empty((linear_workspace_bytes(False, M, N, K, rec),), dtype=torch.uint8, device=X.device)
    _check(lib().qfp4_linear_fwd(_ptr(X), _ptr(W), _ptr(Y), M, N, K, ctypes.byref(rec), ctypes.byref(seed),
                                 _ptr(workspace), workspace.numel(), _stream(stream)), "qfp4_linear_fwd")
    return Y


def linear_fwd_chain(X, W, rec: Recipe, seed: Seed, x_amax=None, next_had: int = HAD_NONE,
                     next_seed: Seed | None = None, want_y_amax: bool = True, Y=None, workspace=None, stream=None):
    """qfp4_linear_fwd_chain: the forward pass taking X's NVFP4 tensor amax
    (x_amax, from the previous layer) and returning Y's for the next layer's
    Fprop rotation (next_had, next_seed). Returns (Y, y_amax or None)."""
    M, K = X.shape
    N = W.shape[0]
    Y = torch.empty((M, N), dtype=_dtype(rec.y_dtype), device=X.device) if Y is None else Y
    if workspace is None:
        workspace = torch.empty((linear_workspace_bytes(False, M, N, K, rec),), dtype=torch.uint8, device=X.device)
    y_amax = torch.empty((1,), dtype=torch.float32, device=X.device) if want_y_amax else None
    ns = ctypes.byref(next_seed) if next_seed is not None else None
    _check(lib().qfp4_linear_fwd_chain(_ptr(X), _ptr(W), _ptr(Y), M, N, K, ctypes.byref(rec), ctypes.byref(seed),
                                       _ptr(x_amax), next_had, ns, _ptr(y_amax), _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "qfp4_linear_fwd_chain")
    return Y, y_amax


def linear_fwd_noalloc(X, W, rec: Recipe, seed: Seed, Y=None, stream=None) -> torch.Tensor:
    """qfp4_linear_fwd_noalloc: the forward pass with the library's fixed
    scratch instead of a workspace (the binding allocates Y only if not given)."""
    M, K = X.shape
    N = W.shape[0]
    Y = torch.empty((M, N), dtype=_dtype(rec.y_dtype), device=X.device) if Y is None else Y
    _check(lib().qfp4_linear_fwd_noalloc(_ptr(X), _ptr(W), _ptr(Y), M, N, K, ctypes.byref(rec), ctypes.byref(seed),
                                         _stream(stream)), "qfp4_linear_fwd_noalloc")
    return Y


def linear_bwd(dY, X, W, rec: Recipe, seed: Seed, dX=None, dW=None, workspace=None, stream=None):
    M, K = X.shape
    N = W.shape[0]
    dX = torch.empty((M, K), dtype=_dtype(rec.dx_dtype), device=X.device) if dX is None else dX
    if rec.dw_accumulate and dW is None:
        raise ValueError("a recipe with dw_accumulate adds into dW: pass the buffer")
    dW = torch.empty((N, K), dtype=_dtype(rec.dw_dtype), device=X.device) if dW is None else dW
    if workspace is None:
        workspace = torch.empty((linear_workspace_bytes(True, M, N, K, rec),), dtype=torch.uint8, device=X.device)
    _check(lib().qfp4_linear_bwd(_ptr(dY), _ptr(X), _ptr(W), _ptr(dX), _ptr(dW), M, N, K, ctypes.byref(rec),
                                 ctypes.byref(seed), _ptr(workspace), workspace.numel(), _stream(stream)),
           "qfp4_linear_bwd")
    return dX, dW


# ---------------------------------------------------------------------------
# The calls below run on the stream that is current on their tensors' device,
# whichever device is current, or on the one given; what they allocate belongs
# to that stream too.

_WS_FLOATS = 1024  # the quantizers' workspace as fp32 words


def _on_stream(f):
    """Adds a keyword `stream`, on which the call then runs."""
    @functools.wraps(f)
    def call(*args, **kwargs):
        if "stream" not in kwargs:
            return f(*args, **kwargs)
        stream = kwargs.pop("stream")
        if stream is None:
            return f(*args, **kwargs)
        t = next(a for a in (*args, *kwargs.values()) if isinstance(a, (torch.Tensor, QTensor)))
        assert stream.device.index == _gpu(t.codes if isinstance(t, QTensor) else t), "a stream of the tensors' GPU"
        with torch.cuda.stream(stream):
            return f(*args, **kwargs)
    return call


def _go(fn, what: str, i: int, *args):
    h = _current_stream(i)
    if i == _current_device():
        status = fn(*args, h)
    else:
        with torch.cuda.device(i):
            status = fn(*args, h)
    if status != OK:
        raise QFP4Error(status, what)


def _gpu(t: torch.Tensor) -> int:
    """Index of the GPU that t is on."""
    i = t.get_device()
    assert i >= 0, "tensors on a GPU"
    return i


def _matrix(t: torch.Tensor, shape, i: int, dtype=torch.bfloat16) -> int:
    """Check a matrix with contiguous rows on GPU i; its row stride (a single row's is not looked at)."""
    assert t.dtype is dtype and t.shape == shape and t.get_device() == i
    if t.is_contiguous():
        return shape[1] or 8
    assert t.stride(1) == 1 or shape[1] == 1
    return t.stride(0) if shape[0] > 1 else max(shape[1], 8)


def _vector(t: torch.Tensor, n: int, dtype, i: int) -> int:
    """Check a contiguous vector of n on GPU i; its address."""
    assert t.dtype is dtype and t.shape == (n,) and t.is_contiguous() and t.get_device() == i
    return t.data_ptr()


def _new_qtensor(like: torch.Tensor, fmt: int, rows: int, k: int) -> QTensor:
    """empty_qtensor on like's device."""
    codes = like.new_empty((rows, k // 2), dtype=torch.uint8)
    scales = like.new_empty((max(scales_bytes(fmt, rows, k), 16),), dtype=torch.uint8)
    ts = like.new_empty((1,), dtype=torch.float32)
    return QTensor(codes, scales, ts, TensorDesc(codes.data_ptr(), scales.data_ptr(), ts.data_ptr()))


def _operand(q: QTensor, fmt: int, rows: int, k: int, i: int) -> QTensor:
    """Check that q's buffers, the ones its descriptor names, hold a rows x k operand on GPU i."""
    parts = (q.codes, codes_bytes(rows, k)), (q.scales, scales_bytes(fmt, rows, k)), (q.tensor_scale, 4)
    for t, nbytes in parts:
        assert t.is_contiguous() and t.get_device() == i, "an operand's buffers on the tensors' GPU"
        assert t.numel() * t.element_size() >= nbytes, f"a buffer of {nbytes} bytes for a {rows} x {k} operand"
    named = (q.desc.codes, q.desc.scales, q.desc.tensor_scale)
    assert all((a or 0) == t.data_ptr() for a, (t, _) in zip(named, parts)), "a descriptor of the operand's buffers"
    return q


def _ref(seed: Seed | None):
    return None if seed is None else ctypes.byref(seed)


def _workspace(given, nbytes: int, like: torch.Tensor):
    """Address and size of a workspace on like's GPU, and the tensor that holds it."""
    if given is None:
        given = like.new_empty((nbytes,), dtype=torch.uint8)
    else:
        assert given.is_contiguous() and given.get_device() == like.get_device(), "a workspace on the tensors' GPU"
    return given.data_ptr(), given.numel() * given.element_size(), given


# ---------------------------------------------------------------------------
# RMSNorm

def _residual(x, res, h, shape, i: int):
    """h (x itself without res and a buffer for it), its address and stride, and res's."""
    if res is None and (h is None or h is x):
        return x, None, 0, None, 0
    h = torch.empty_like(x) if h is None else h
    ldh = _matrix(h, shape, i)
    return (h, h.data_ptr(), ldh, None, 0) if res is None else (h, h.data_ptr(), ldh, res.data_ptr(),
                                                                _matrix(res, shape, i))


@_on_stream
def rmsnorm_fwd(x: torch.Tensor, w: torch.Tensor, eps: float, res: torch.Tensor | None = None, had: int = HAD_NONE,
                seed: Seed | None = None, want_amax: bool = False, y=None, h=None, rstd=None, y_amax=None,
                workspace=None):
    """h = x + res, y = h / rms(h) * w; see qfp4_rmsnorm_fwd. Returns (y, h,
    rstd, y_amax): without res, h is x itself unless a buffer for it is given
    (which the backward pass needs if y goes to x's place); y_amax, y's NVFP4 tensor amax after the rotation `had`, is None unless
    wanted (want_amax or a buffer for it)."""
    shape, i = x.shape, _gpu(x)
    ldx = _matrix(x, shape, i)
    R, C = shape
    y = torch.empty_like(x) if y is None else y
    h, hp, ldh, rp, ldr = _residual(x, res, h, shape, i)
    amax = want_amax or y_amax is not None
    ap, wsp, wsb = None, None, 0
    if amax and rstd is None and y_amax is None and workspace is None:
        # one allocation for the three
        workspace = x.new_empty((_WS_FLOATS + 4 + R,), dtype=torch.float32)
        y_amax = workspace.as_strided((1,), (1,), _WS_FLOATS)
        rstd = workspace.as_strided((R,), (1,), _WS_FLOATS + 4)
        wsp, wsb = workspace.data_ptr(), 4 * _WS_FLOATS
        ap, rsp = wsp + 4 * _WS_FLOATS, wsp + 4 * (_WS_FLOATS + 4)
    else:
        rstd = x.new_empty((R,), dtype=torch.float32) if rstd is None else rstd
        rsp = _vector(rstd, R, torch.float32, i)
        if amax:
            y_amax = x.new_empty((1,), dtype=torch.float32) if y_amax is None else y_amax
            ap = _vector(y_amax, 1, torch.float32, i)
            wsp, wsb, workspace = _workspace(workspace, 4 * _WS_FLOATS, x)
    _go(lib().qfp4_rmsnorm_fwd, "qfp4_rmsnorm_fwd", i, x.data_ptr(), ldx, rp, ldr, _vector(w, C, torch.bfloat16, i), R,
        C, eps, hp, ldh, y.data_ptr(), _matrix(y, shape, i), rsp, had, _ref(seed), ap, wsp, wsb)
    return y, h, rstd, y_amax


@_on_stream
def rmsnorm_quantize(x: torch.Tensor, w: torch.Tensor, eps: float, res: torch.Tensor | None = None, fmt: int = MXFP4,
                     had: int = HAD_NONE, seed: Seed | None = None, want_y: bool = True, y=None, h=None, rstd=None,
                     out: QTensor | None = None):
    """rmsnorm_fwd and y's MXFP4 (or MXFP4_RU) quantization along its rows; see
    qfp4_rmsnorm_quantize. Returns (y, h, rstd, q); y is None unless wanted."""
    shape, i = x.shape, _gpu(x)
    ldx = _matrix(x, shape, i)
    R, C = shape
    if y is None and want_y:
        y = torch.empty_like(x)
    h, hp, ldh, rp, ldr = _residual(x, res, h, shape, i)
    rstd = x.new_empty((R,), dtype=torch.float32) if rstd is None else rstd
    out = _new_qtensor(x, MXFP4, R, C) if out is None else _operand(out, MXFP4, R, C, i)
    _go(lib().qfp4_rmsnorm_quantize, "qfp4_rmsnorm_quantize", i, x.data_ptr(), ldx, rp, ldr,
        _vector(w, C, torch.bfloat16, i), R, C, eps, hp, ldh, None if y is None else y.data_ptr(),
        0 if y is None else _matrix(y, shape, i), _vector(rstd, R, torch.float32, i), fmt, had, _ref(seed),
        ctypes.byref(out.desc))
    return y, h, rstd, out


@_on_stream
def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor, dh: torch.Tensor | None = None,
                dx=None, dw=None, accumulate: bool = False, workspace=None):
    """Gradients (dx, dw) of rmsnorm_fwd from y's gradient and (dh) h's own;
    see qfp4_rmsnorm_bwd. dx is the gradient of x and of res alike; dw is fp32."""
    shape, i = dy.shape, _gpu(dy)
    lddy = _matrix(dy, shape, i)
    R, C = shape
    dx = torch.empty_like(dy) if dx is None else dx
    if accumulate and dw is None:
        raise ValueError("accumulate adds into dw: pass the buffer")
    dw = dy.new_empty((C,), dtype=torch.float32) if dw is None else dw
    wsp, wsb, workspace = _workspace(workspace, lib().qfp4_rmsnorm_bwd_workspace_bytes(R, C), dy)
    _go(lib().qfp4_rmsnorm_bwd, "qfp4_rmsnorm_bwd", i, dy.data_ptr(), lddy, h.data_ptr(), _matrix(h, shape, i),
        _vector(w, C, torch.bfloat16, i), _vector(rstd, R, torch.float32, i), None if dh is None else dh.data_ptr(),
        0 if dh is None else _matrix(dh, shape, i), R, C, dx.data_ptr(), _matrix(dx, shape, i),
        _vector(dw, C, torch.float32, i), 1 if accumulate else 0, wsp, wsb)
    return dx, dw


# ---------------------------------------------------------------------------
# groups of rows: the experts of a mixture

def group_rows(T: int, E: int) -> int:
    """Rows of the padded layout of T rows in E groups."""
    return lib().qfp4_group_rows(T, E)


def _groups(offsets: torch.Tensor, i: int) -> int:
    """Check the group offsets (int32 [E + 1] on GPU i); E."""
    n = offsets.shape[0]
    assert n >= 2
    _vector(offsets, n, torch.int32, i)
    return n - 1


@_on_stream
def quantize_grouped(x: torch.Tensor, offsets: torch.Tensor, fmt: int, rounding: int, had: int, axis: int,
                     seed: Seed | None = None, amax_in: torch.Tensor | None = None, out: QTensor | None = None,
                     workspace=None) -> QTensor:
    """Quantize rows sorted by group, in the padded layout; see qfp4_quantize_grouped."""
    shape, i = x.shape, _gpu(x)
    ldx = _matrix(x, shape, i)
    T, C = shape
    E = _groups(offsets, i)
    Tp = max(group_rows(T, E), 0)
    rows, k = (Tp, C) if axis == ROW else (C, Tp)
    out = _new_qtensor(x, fmt, rows, k) if out is None else _operand(out, fmt, rows, k, i)
    wsp, wsb = None, 0
    if amax_in is None and fmt == NVFP4:
        wsp, wsb, workspace = _workspace(workspace, 4 * _WS_FLOATS, x)
    _go(lib().qfp4_quantize_grouped, "qfp4_quantize_grouped", i, x.data_ptr(), T, C, ldx, offsets.data_ptr(), E, fmt,
        rounding, had, axis, ctypes.byref(seed or make_seed()),
        None if amax_in is None else _vector(amax_in, 1, torch.float32, i), ctypes.byref(out.desc), wsp, wsb)
    return out


@_on_stream
def gemm_grouped(A: QTensor, B: QTensor, offsets: torch.Tensor, T: int, out_dtype=torch.bfloat16,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Each group's rows of A times its part of B, as T rows; see
    qfp4_gemm_grouped. Rows of no group are not written."""
    i = _gpu(A.codes)
    E = _groups(offsets, i)
    a, b = A.desc, B.desc
    N = b.rows // E if b.k == a.k else b.rows
    out = A.codes.new_empty((T, N), dtype=out_dtype) if out is None else out
    f32 = out.dtype is torch.float32
    ldd = _matrix(out, (T, N), i, torch.float32 if f32 else torch.bfloat16)
    assert B.codes.get_device() == i
    _go(lib().qfp4_gemm_grouped, "qfp4_gemm_grouped", i, ctypes.byref(a), ctypes.byref(b), offsets.data_ptr(), E, T,
        out.data_ptr(), ldd, OUT_F32 if f32 else OUT_BF16)
    return out


@_on_stream
def gemm_grouped_wgrad(A: QTensor, B: QTensor, offsets: torch.Tensor, T: int, out_dtype=torch.float32,
                       out: torch.Tensor | None = None, accumulate: bool = False) -> torch.Tensor:
    """Per group, the product over its tokens [E, A.rows, B.rows]; see qfp4_gemm_grouped_wgrad."""
    i = _gpu(A.codes)
    E = _groups(offsets, i)
    if accumulate and out is None:
        raise ValueError("accumulate adds into out: pass the buffer")
    if out is None:
        out = A.codes.new_empty((E, A.rows, B.rows), dtype=out_dtype)
    assert out.shape == (E, A.rows, B.rows) and out.is_contiguous() and out.get_device() == i == B.codes.get_device()
    assert out.dtype in (torch.bfloat16, torch.float32)
    _go(lib().qfp4_gemm_grouped_wgrad, "qfp4_gemm_grouped_wgrad", i, ctypes.byref(A.desc),
        ctypes.byref(B.desc), offsets.data_ptr(), E, T, out.data_ptr(),
        OUT_F32 if out.dtype == torch.float32 else OUT_BF16, 1 if accumulate else 0)
    return out


def linear_grouped_workspace_bytes(backward: bool, T: int, E: int, N: int, K: int, rec: Recipe) -> int:
    return lib().qfp4_linear_grouped_workspace_bytes(1 if backward else 0, T, E, N, K, ctypes.byref(rec))


def _linear_grouped_args(X, W, offsets):
    T, K = X.shape
    E, N, _ = W.shape
    i = _gpu(X)
    assert X.dtype == W.dtype == torch.bfloat16 and W.shape[2] == K and i == W.get_device()
    assert X.is_contiguous() and W.is_contiguous() and _groups(offsets, i) == E
    return T, E, N, K, i


def _linear_output(t, shape, code: int, like: torch.Tensor) -> torch.Tensor:
    if t is None:
        return like.new_empty(shape, dtype=_dtype(code))
    assert t.shape == shape and t.dtype == _dtype(code) and t.is_contiguous() and t.get_device() == like.get_device()
    return t


@_on_stream
def linear_grouped_fwd(X, W, offsets, rec: Recipe, seed: Seed, x_amax=None, Y=None, workspace=None) -> torch.Tensor:
    """Y[t] = X[t] W_e^T for the rows t of group e, W [E, N, K]; see
    qfp4_linear_grouped_fwd. Rows of Y that are no group's are not written."""
    T, E, N, K, i = _linear_grouped_args(X, W, offsets)
    Y = _linear_output(Y, (T, N), rec.y_dtype, X)
    wsp, wsb, workspace = _workspace(workspace, linear_grouped_workspace_bytes(False, T, E, N, K, rec), X)
    _go(lib().qfp4_linear_grouped_fwd, "qfp4_linear_grouped_fwd", i, X.data_ptr(), W.data_ptr(), Y.data_ptr(),
        offsets.data_ptr(), E, T, N, K, ctypes.byref(rec), ctypes.byref(seed),
        None if x_amax is None else _vector(x_amax, 1, torch.float32, i), wsp, wsb)
    return Y


@_on_stream
def linear_grouped_bwd(dY, X, W, offsets, rec: Recipe, seed: Seed, dX=None, dW=None, workspace=None):
    """(dX, dW) of linear_grouped_fwd; see qfp4_linear_grouped_bwd. Rows of dX
    that are no group's are not written; dW of an empty group is zero."""
    T, E, N, K, i = _linear_grouped_args(X, W, offsets)
    assert dY.shape == (T, N) and dY.dtype == torch.bfloat16 and dY.is_contiguous() and dY.get_device() == i
    dX = _linear_output(dX, (T, K), rec.dx_dtype, X)
    if rec.dw_accumulate and dW is None:
        raise ValueError("a recipe with dw_accumulate adds into dW: pass the buffer")
    dW = _linear_output(dW, (E, N, K), rec.dw_dtype, X)
    wsp, wsb, workspace = _workspace(workspace, linear_grouped_workspace_bytes(True, T, E, N, K, rec), X)
    _go(lib().qfp4_linear_grouped_bwd, "qfp4_linear_grouped_bwd", i, dY.data_ptr(), X.data_ptr(),
        W.data_ptr(), dX.data_ptr(), dW.data_ptr(), offsets.data_ptr(), E, T, N, K, ctypes.byref(rec),
        ctypes.byref(seed), wsp, wsb)
    return dX, dW


def status(stream=None):
    """Synchronize and raise if a kernel reported a device-side error."""
    _check(lib().qfp4_status(_stream(stream)), "qfp4_status")


def selftest_rounding(op: int, x: torch.Tensor, w: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The quantizers' rounding step `op` (ROUND_*) applied to each fp32 of x
    with the uint32 random words w (int32 storage): one code byte per value."""
    assert x.dtype == torch.float32 and x.is_contiguous()
    assert w is None or (w.dtype == torch.int32 and w.is_contiguous() and w.numel() == x.numel())
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(lib().qfp4_selftest_rounding(op, _ptr(x), _ptr(w), _ptr(codes), x.numel(), _stream(stream)),
           "qfp4_selftest_rounding")
    return codes


class _FirstOrder(torch.autograd.Function):
    """The tensors that compute() gives, as functions of deps whose own
    gradients are refused."""

    @staticmethod
    def forward(ctx, compute, *deps):
        return compute()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("these kernels have first derivatives only: a gradient made with create_graph=True cannot "
                           "be differentiated again")


def _first_order(compute, *deps):
    """compute(), gradients that depend on deps. With create_graph=True they would count as constants, and a second
    backward pass drop their part without a word; here it raises."""
    return _FirstOrder.apply(compute, *deps) if torch.is_grad_enabled() else compute()


class Fp4Linear(torch.autograd.Function):
    """y = x W^T with FP4 Fprop/Dgrad/Wgrad (bf16 inputs, recipe + seed per
    call). First derivatives only."""

    @staticmethod
    def forward(ctx, X, W, rec: Recipe, seed: Seed):
        ctx.save_for_backward(X, W)
        ctx.rec, ctx.seed = rec, seed
        return linear_fwd(X.contiguous(), W.contiguous(), rec, seed)

    @staticmethod
    def backward(ctx, dY):
        X, W = ctx.saved_tensors

        def gradients():
            dX, dW = linear_bwd(dY.contiguous().to(torch.bfloat16), X.contiguous(), W.contiguous(), ctx.rec, ctx.seed)
            return dX.to(X.dtype), dW.to(W.dtype)

        return *_first_order(gradients, dY, X, W), None, None


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as a matrix of its last dimension's rows; a copy where the kernels do
    not take its strides or its address."""
    m = t.reshape(-1, t.shape[-1])
    if m.is_contiguous():
        return m if m.data_ptr() % 16 == 0 else m.clone()
    taken = m.stride(1) == 1 and m.stride(0) >= m.shape[1] and m.stride(0) % 8 == 0 and m.data_ptr() % 16 == 0
    return m if taken else m.contiguous()


class RmsNorm(torch.autograd.Function):
    """(y, h) = (h / rms(h) * w, x + res) in bf16; res may be None. First derivatives only."""

    @staticmethod
    def forward(ctx, x, res, w, eps: float):
        C = x.shape[-1]
        # tensors of their own, not views: a program may change y in place (h is
        # kept for the backward pass, which refuses a changed one)
        y, h = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for _ in range(2))
        _, _, rstd, _ = rmsnorm_fwd(_rows(x), _rows(w)[0], eps, res=None if res is None else _rows(res),
                                    y=y.view(-1, C), h=h.view(-1, C))
        ctx.save_for_backward(h, w, rstd)
        ctx.has_res = res is not None
        ctx.set_materialize_grads(False)  # an output that nothing uses has no gradient
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, w, rstd = ctx.saved_tensors
        if dy is None:  # h alone was used: it is x + res
            return dh, dh if ctx.has_res else None, None, None

        def gradients():
            C = h.shape[-1]
            dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
            _, dw = rmsnorm_bwd(_rows(dy), h.view(-1, C), _rows(w)[0], rstd, dh=None if dh is None else _rows(dh),
                                dx=dx.view(-1, C))
            return dx, dw.to(w.dtype)

        dx, dw = _first_order(gradients, dy, dh, h, w)
        return dx, dx if ctx.has_res else None, dw, None


class Fp4GroupedLinear(torch.autograd.Function):
    """y[t] = x[t] W_e^T over the rows t of group e, W [E, N, K] (bf16 inputs,
    recipe + seed per call). Rows that are no group's give zeros. First
    derivatives only."""

    @staticmethod
    def forward(ctx, X, W, offsets, rec: Recipe, seed: Seed):
        ctx.save_for_backward(X, W, offsets)
        ctx.rec, ctx.seed = rec, seed
        Y = torch.zeros((X.shape[0], W.shape[1]), dtype=_dtype(rec.y_dtype), device=X.device)
        return linear_grouped_fwd(X.contiguous(), W.contiguous(), offsets, rec, seed, Y=Y)

    @staticmethod
    def backward(ctx, dY):
        X, W, offsets = ctx.saved_tensors

        def gradients():
            dX = torch.zeros(X.shape, dtype=_dtype(ctx.rec.dx_dtype), device=X.device)
            _, dW = linear_grouped_bwd(dY.contiguous().to(torch.bfloat16), X.contiguous(), W.contiguous(), offsets,
                                       ctx.rec, ctx.seed, dX=dX)
            return dX.to(X.dtype), dW.to(W.dtype)

        return *_first_order(gradients, dY, X, W), None, None, None
