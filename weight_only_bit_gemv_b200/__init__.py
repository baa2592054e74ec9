"""Python binding of the sm_100a 4-bit codebook linear-layer library (libq4.so).

Argument marshalling only: every step of pack, dequant and the matmuls runs in
the CUDA kernels of libq4.so, on the tensors' device, on the current torch
stream.  PyTorch supplies device memory and streams.  There is no CPU path:
if the library cannot be loaded, every call raises.

Q4_LIBRARY=debug in the environment loads libq4_debug.so instead: the same
kernels built with -DQ4_DEBUG, in which each global load and store checks its
index range first and a failed check sets a bit of bounds_flags() and skips
the access.  It is slower and meant for tests only.

Tensor conventions (all contiguous, on one CUDA device):
  w        float32            [N, K]
  codebook float16 or uint16  [16]       (binary16 bits)
  codes    uint8              [N, K/2]   low nibble = even k
  scales   float16 or uint16  [N, K/64]  (binary16 bits)
  x        bfloat16 or uint16 [M, K]     (bfloat16 bits)
  y        float32            [M, N]

The microscaled 4-bit calls (q4_pack_mx and the products on it) take blocks of
128 rows x 128 k, padded with zeros, Nb = ceil(N / 128), Kb = ceil(K / 128):
  codes    uint8              [Nb, Kb, 128, 64]   a stack of experts: [E, Nb, Kb, 128, 64]
  scales   uint8              [Nb, Kb, 512]                          [E, Nb, Kb, 512]
They run on the tensors' device whatever the current device is (a stream of
another device is refused), and what they
allocate belongs to the stream that they run on.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import build as _build

GROUP = 64
_HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(os.path.dirname(_HERE), "include", "q4.h")

STATUS = {0: "Q4_OK", 1: "Q4_ERR_NULL", 2: "Q4_ERR_SHAPE", 3: "Q4_ERR_ALIGN", 4: "Q4_ERR_ARCH",
          5: "Q4_ERR_CUDA", 6: "Q4_ERR_TOO_LARGE"}


class Q4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lib = None


class Q4Linear(ctypes.Structure):
    """struct q4_linear of q4.h: one linear of a recorded step."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("codebook", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


def debug_selected() -> bool:
    """True when Q4_LIBRARY=debug selects the bounds-checked build."""
    v = os.environ.get("Q4_LIBRARY", "").strip().lower()
    if v not in ("", "release", "debug"):
        raise RuntimeError(f"Q4_LIBRARY must be 'release' or 'debug', not {v!r}")
    return v == "debug"


def library_path() -> str:
    return _build.DEBUG_LIBRARY if debug_selected() else _build.LIBRARY


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libq4.so, or libq4_debug.so under Q4_LIBRARY=debug (building it
    with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    debug = debug_selected()
    path = library_path()
    if build_if_missing and _build.stale(path):
        _build.build(debug=debug)
    if not os.path.exists(path):
        raise RuntimeError(f"{os.path.basename(path)} not found at {path}; run "
                           "python -m weight_only_bit_gemv_b200.build" + (" --debug" if debug else ""))
    lib = ctypes.CDLL(path)
    P, I64, S = ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p
    lib.q4_pack.argtypes = [P, P, P, P, I64, I64, S]
    lib.q4_dequant.argtypes = [P, P, P, P, I64, I64, S]
    lib.q4_gemv.argtypes = [P, P, P, P, P, I64, I64, I64, S]
    lib.q4_gemm.argtypes = [P, P, P, P, P, I64, I64, I64, S]
    lib.q4_gemm_noalloc.argtypes = [P, P, P, P, P, I64, I64, I64, S]
    lib.q4_embed_rows.argtypes = [P, P, P, P, P, I64, I64, I64, S]
    lib.q4_pack2.argtypes = [P, P, P, P, I64, I64, S]
    lib.q4_dequant2.argtypes = [P, P, P, P, I64, I64, S]
    lib.q4_gemv2.argtypes = [P, P, P, P, P, I64, I64, S]
    for f in ("q4_pack", "q4_dequant", "q4_gemv", "q4_gemm", "q4_gemm_noalloc", "q4_embed_rows",
              "q4_pack2", "q4_dequant2", "q4_gemv2"):
        getattr(lib, f).restype = ctypes.c_int
    lib.q4_status_string.argtypes = [ctypes.c_int]
    lib.q4_status_string.restype = ctypes.c_char_p
    lib.q4_last_cuda_error.argtypes = []
    lib.q4_last_cuda_error.restype = ctypes.c_int
    lib.q4_abi_version.argtypes = []
    lib.q4_abi_version.restype = ctypes.c_int
    lib.q4_timeout_flags.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.q4_timeout_flags.restype = ctypes.c_int
    lib.q4_ring_create.argtypes = [I64, ctypes.POINTER(ctypes.c_void_p)]
    lib.q4_ring_create.restype = ctypes.c_int
    lib.q4_ring_gemm.argtypes = [P, P, P, P, P, P, I64, I64, I64, S]
    lib.q4_ring_gemm.restype = ctypes.c_int
    lib.q4_ring_destroy.argtypes = [P]
    lib.q4_ring_destroy.restype = ctypes.c_int
    lib.q4_step_create.argtypes = [ctypes.POINTER(Q4Linear), I64, ctypes.POINTER(ctypes.c_void_p)]
    lib.q4_step_create.restype = ctypes.c_int
    lib.q4_step_launch.argtypes = [P, S]
    lib.q4_step_launch.restype = ctypes.c_int
    lib.q4_step_destroy.argtypes = [P]
    lib.q4_step_destroy.restype = ctypes.c_int
    lib.q4_wait_selftest.argtypes = [ctypes.c_uint32, ctypes.c_int, ctypes.POINTER(ctypes.c_uint32)]
    lib.q4_wait_selftest.restype = ctypes.c_int
    T, W = ctypes.c_int, ctypes.c_int
    lib.q4_pack_mx.argtypes = [P, T, P, P, I64, I64, I64, S]
    lib.q4_dequant_mx.argtypes = [P, P, P, T, I64, I64, I64, S]
    lib.q4_gemm_mx.argtypes = [P, P, P, P, T, I64, I64, I64, P, I64, S]
    lib.q4_gemm_experts.argtypes = [P, P, P, P, P, P, T, I64, I64, I64, I64, I64, P, I64, S]
    lib.q4_sort_experts.argtypes = [P, W, P, P, P, I64, I64, I64, S]
    lib.q4_dispatch.argtypes = [P, P, P, T, I64, I64, I64, S]
    lib.q4_combine.argtypes = [P, P, P, P, T, I64, I64, I64, S]
    lib.q4_combine_grad.argtypes = [P, P, P, P, P, P, T, I64, I64, I64, S]
    for f in ("q4_pack_mx", "q4_dequant_mx", "q4_gemm_mx", "q4_gemm_experts", "q4_sort_experts",
              "q4_dispatch", "q4_combine", "q4_combine_grad"):
        getattr(lib, f).restype = ctypes.c_int
    lib.q4_gemm_mx_workspace.argtypes = [I64, I64, I64]
    lib.q4_gemm_mx_workspace.restype = I64
    lib.q4_gemm_experts_workspace.argtypes = [I64, I64, I64, I64]
    lib.q4_gemm_experts_workspace.restype = I64
    lib.q4_bounds_flags.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.q4_bounds_flags.restype = ctypes.c_int
    lib.q4_bounds_checked.argtypes = []
    lib.q4_bounds_checked.restype = ctypes.c_int
    _lib = lib
    return lib


def header_functions() -> list:
    """Names of the functions include/q4.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(q4_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return load().q4_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        lib = load()
        msg = f"{what}: {status_string(status)}"
        if status == 5:
            msg += f" (cudaError {lib.q4_last_cuda_error()})"
        raise Q4Error(status, msg)


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtypes, shape=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


_H16 = (torch.float16, torch.uint16, torch.int16)
_BF16 = (torch.bfloat16, torch.uint16, torch.int16)


def _packed_dims(codes: torch.Tensor):
    if codes.dim() != 2:
        raise ValueError("codes must be [N, K/2]")
    return codes.shape[0], codes.shape[1] * 2


def q4_pack(w: torch.Tensor, codebook: torch.Tensor, codes: torch.Tensor = None,
            scales: torch.Tensor = None, stream=None):
    """Quantize w [N, K] fp32 into (codes, scales); allocates them with torch if not given."""
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // GROUP), dtype=torch.float16, device=w.device)
    _need(w, "w", (torch.float32,))
    _need(codebook, "codebook", _H16, (16,))
    _need(codes, "codes", (torch.uint8,), (N, K // 2))
    _need(scales, "scales", _H16, (N, K // GROUP))
    st = load().q4_pack(w.data_ptr(), codebook.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                        N, K, _stream(w, stream))
    _check(st, "q4_pack")
    return codes, scales


def q4_dequant(codes: torch.Tensor, scales: torch.Tensor, codebook: torch.Tensor,
               w_out: torch.Tensor = None, stream=None) -> torch.Tensor:
    N, K = _packed_dims(codes)
    if w_out is None:
        w_out = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _H16, (N, K // GROUP))
    _need(codebook, "codebook", _H16, (16,))
    _need(w_out, "w_out", (torch.float32,), (N, K))
    st = load().q4_dequant(codes.data_ptr(), scales.data_ptr(), codebook.data_ptr(),
                           w_out.data_ptr(), N, K, _stream(codes, stream))
    _check(st, "q4_dequant")
    return w_out


def q4_embed_rows(codes: torch.Tensor, scales: torch.Tensor, codebook: torch.Tensor,
                  ids: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """out [n, K] fp32 = rows ids [n] (int32) of the packed matrix, dequantized
    exactly; ids outside [0, N) give rows of zeros."""
    N, K = _packed_dims(codes)
    if ids.dim() != 1:
        raise ValueError("ids must be [n]")
    n = ids.shape[0]
    if out is None:
        out = torch.empty((n, K), dtype=torch.float32, device=codes.device)
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _H16, (N, K // GROUP))
    _need(codebook, "codebook", _H16, (16,))
    _need(ids, "ids", (torch.int32,))
    _need(out, "out", (torch.float32,), (n, K))
    st = load().q4_embed_rows(codes.data_ptr(), scales.data_ptr(), codebook.data_ptr(),
                              ids.data_ptr(), out.data_ptr(), n, N, K, _stream(codes, stream))
    _check(st, "q4_embed_rows")
    return out


def _matmul(fn: str, codes, scales, codebook, x, y, stream):
    N, K = _packed_dims(codes)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M, {K}]")
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=codes.device)
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _H16, (N, K // GROUP))
    _need(codebook, "codebook", _H16, (16,))
    _need(x, "x", _BF16)
    _need(y, "y", (torch.float32,), (M, N))
    st = getattr(load(), fn)(codes.data_ptr(), scales.data_ptr(), codebook.data_ptr(),
                             x.data_ptr(), y.data_ptr(), M, N, K, _stream(codes, stream))
    _check(st, fn)
    return y


# ---- the two-bit variant: codes [N, K/4], a 4-entry codebook ---------------

def q4_pack2(w: torch.Tensor, codebook4: torch.Tensor, codes: torch.Tensor = None,
             scales: torch.Tensor = None, stream=None):
    """Quantize w [N, K] fp32 into 2-bit (codes [N, K/4], scales [N, K/64])."""
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    N, K = w.shape
    if codes is None:
        codes = torch.empty((N, K // 4), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((N, K // GROUP), dtype=torch.float16, device=w.device)
    _need(w, "w", (torch.float32,))
    _need(codebook4, "codebook4", _H16, (4,))
    _need(codes, "codes", (torch.uint8,), (N, K // 4))
    _need(scales, "scales", _H16, (N, K // GROUP))
    st = load().q4_pack2(w.data_ptr(), codebook4.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                         N, K, _stream(w, stream))
    _check(st, "q4_pack2")
    return codes, scales


def _packed2_dims(codes: torch.Tensor):
    if codes.dim() != 2:
        raise ValueError("codes must be [N, K/4]")
    return codes.shape[0], codes.shape[1] * 4


def q4_dequant2(codes: torch.Tensor, scales: torch.Tensor, codebook4: torch.Tensor,
                w_out: torch.Tensor = None, stream=None) -> torch.Tensor:
    N, K = _packed2_dims(codes)
    if w_out is None:
        w_out = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _H16, (N, K // GROUP))
    _need(codebook4, "codebook4", _H16, (4,))
    _need(w_out, "w_out", (torch.float32,), (N, K))
    st = load().q4_dequant2(codes.data_ptr(), scales.data_ptr(), codebook4.data_ptr(),
                            w_out.data_ptr(), N, K, _stream(codes, stream))
    _check(st, "q4_dequant2")
    return w_out


def q4_gemv2(codes, scales, codebook4, x, y=None, stream=None) -> torch.Tensor:
    """y [1, N] = x [1, K] @ W^T with W rebuilt from the 2-bit codes in the kernel."""
    N, K = _packed2_dims(codes)
    if x.dim() != 2 or tuple(x.shape) != (1, K):
        raise ValueError(f"x must be [1, {K}]")
    if y is None:
        y = torch.empty((1, N), dtype=torch.float32, device=codes.device)
    _need(codes, "codes", (torch.uint8,))
    _need(scales, "scales", _H16, (N, K // GROUP))
    _need(codebook4, "codebook4", _H16, (4,))
    _need(x, "x", _BF16)
    _need(y, "y", (torch.float32,), (1, N))
    st = load().q4_gemv2(codes.data_ptr(), scales.data_ptr(), codebook4.data_ptr(),
                         x.data_ptr(), y.data_ptr(), N, K, _stream(codes, stream))
    _check(st, "q4_gemv2")
    return y


def q4_gemv(codes, scales, codebook, x, y=None, stream=None) -> torch.Tensor:
    """y [1, N] = x [1, K] @ W^T with W rebuilt from codes/scales/codebook in the kernel."""
    return _matmul("q4_gemv", codes, scales, codebook, x, y, stream)


def q4_gemm(codes, scales, codebook, x, y=None, stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] @ W^T for any M (M <= 24: verify batches and short
    chunks on the CUDA-core decode kernels; M > 24: prefill on tensor cores)."""
    return _matmul("q4_gemm", codes, scales, codebook, x, y, stream)


def q4_gemm_noalloc(codes, scales, codebook, x, y, stream=None) -> torch.Tensor:
    """q4_gemm without any device allocation by the library: for M > 16 the
    binary16 copy of x lives in the library's fixed 8 MiB device array, so
    2 * M * K must fit in it (else Q4Error Q4_ERR_TOO_LARGE), and calls that
    overlap on the GPU race on that array.  y must be passed in."""
    if y is None:
        raise ValueError("q4_gemm_noalloc writes into a caller-provided y")
    return _matmul("q4_gemm_noalloc", codes, scales, codebook, x, y, stream)


# ---- microscaled 4-bit matrices and layers routed by expert -----------------

MX_BLOCK = 128
MX_GROUP = 32
_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class _Foreign:
    """The context of a call on another stream or device than the current one:
    makes the tensors' device current, and what the call allocates belong to
    the stream that it runs on, so that it can be freed before the call has run."""

    __slots__ = ("_guards",)

    def __init__(self, index: int, stream):
        self._guards = [torch.cuda.device(index)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", index))
            elif stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{index}")
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)


def _elsewhere(t: torch.Tensor, stream) -> bool:
    """Whether a call on ``t``'s device and ``stream`` has to enter _Foreign."""
    return stream is not None or t.get_device() != torch._C._cuda_getDevice()


def _operand(t, name: str, dtypes, shape, on: torch.Tensor) -> None:
    """One tensor of a call: its type, shape, layout and device."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.is_cuda
            and t.get_device() == on.get_device() and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, not on {on.device}")


def _dims(t, name: str, dims, form: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() not in dims:
        raise ValueError(f"{name} must be {form}")


_BYTES = (torch.uint8,)
_I32 = (torch.int32,)
_IDS = (torch.int32, torch.int64)
_F32 = (torch.float32,)
_FLOATS = tuple(_TYPE)
_OUT = (torch.float32, torch.bfloat16)


def _type(dtype, allowed, name: str) -> int:
    if dtype not in allowed:
        raise TypeError(f"{name}: dtype {dtype} not in {allowed}")
    return _TYPE[dtype]


def _mx_sizes(codes, scales, N, K):
    """(E or None, N, K) of a packed matrix or stack, checked against its blocks."""
    _dims(codes, "codes", (4, 5), "[Nb, Kb, 128, 64] or [E, Nb, Kb, 128, 64]")
    shape = codes.shape
    nb, kb = shape[-4], shape[-3]
    if shape[-2] != MX_BLOCK or shape[-1] != MX_BLOCK // 2:
        raise ValueError("codes must be [..., Nb, Kb, 128, 64]")
    N = nb * MX_BLOCK if N is None else int(N)
    K = kb * MX_BLOCK if K is None else int(K)
    if -(-N // MX_BLOCK) != nb or -(-K // MX_BLOCK) != kb or N < 0:
        raise ValueError(f"N = {N}, K = {K} do not have {nb} x {kb} blocks of {MX_BLOCK}")
    _operand(codes, "codes", _BYTES, shape, codes)
    if len(shape) == 4:
        _operand(scales, "scales", _BYTES, (nb, kb, 512), codes)
        return None, N, K
    _operand(scales, "scales", _BYTES, (shape[0], nb, kb, 512), codes)
    return shape[0], N, K


def q4_pack_mx(w: torch.Tensor, codes: torch.Tensor = None, scales: torch.Tensor = None, stream=None):
    """Quantize w [N, K] or [E, N, K] (float32, bfloat16 or float16) into
    microscaled 4-bit (codes, scales) blocks; allocates them if not given."""
    _dims(w, "w", (2, 3), "[N, K] or [E, N, K]")
    N, K = w.shape[-2:]
    lead = tuple(w.shape[:-2])
    nb, kb = -(-N // MX_BLOCK), -(-K // MX_BLOCK)
    _operand(w, "w", _FLOATS, w.shape, w)
    if _elsewhere(w, stream):
        with _Foreign(w.get_device(), stream):
            return q4_pack_mx(w, codes, scales)
    handle = torch._C._cuda_getCurrentRawStream(w.get_device())
    if codes is None:
        codes = torch.empty(*lead, nb, kb, MX_BLOCK, MX_BLOCK // 2, dtype=torch.uint8, device=w.device)
    else:
        _operand(codes, "codes", _BYTES, (*lead, nb, kb, MX_BLOCK, MX_BLOCK // 2), w)
    if scales is None:
        scales = torch.empty(*lead, nb, kb, 512, dtype=torch.uint8, device=w.device)
    else:
        _operand(scales, "scales", _BYTES, (*lead, nb, kb, 512), w)
    st = load().q4_pack_mx(w.data_ptr(), _TYPE[w.dtype], codes.data_ptr(), scales.data_ptr(),
                           lead[0] if lead else 1, N, K, handle)
    _check(st, "q4_pack_mx")
    return codes, scales


def q4_dequant_mx(codes: torch.Tensor, scales: torch.Tensor, w_out: torch.Tensor = None, N: int = None,
                  K: int = None, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """W [N, K] or [E, N, K] from its microscaled blocks, as w_out's type or
    ``dtype``.  N and K default to whole blocks."""
    E, N, K = _mx_sizes(codes, scales, N, K)
    shape = (N, K) if E is None else (E, N, K)
    if _elsewhere(codes, stream):
        with _Foreign(codes.get_device(), stream):
            return q4_dequant_mx(codes, scales, w_out, N, K, dtype)
    handle = torch._C._cuda_getCurrentRawStream(codes.get_device())
    if w_out is None:
        _type(dtype, _FLOATS, "dtype")
        w_out = torch.empty(*shape, dtype=dtype, device=codes.device)
    else:
        _operand(w_out, "w_out", _FLOATS, shape, codes)
    st = load().q4_dequant_mx(codes.data_ptr(), scales.data_ptr(), w_out.data_ptr(),
                              _TYPE[w_out.dtype], 1 if E is None else E, N, K, handle)
    _check(st, "q4_dequant_mx")
    return w_out


def _scratch(workspace, need: int, of: torch.Tensor, what: str):
    """(address, bytes) of a call's workspace and the tensor that holds it: the
    caller's, or one of the call's own."""
    if need < 0:
        _check(2, what)
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=of.device)
        return workspace.data_ptr(), need, workspace
    _dims(workspace, "workspace", (1,), "[bytes]")
    _operand(workspace, "workspace", _BYTES, workspace.shape, of)
    return workspace.data_ptr(), workspace.numel(), workspace


def q4_gemm_mx_workspace(M: int, N: int, K: int) -> int:
    """Bytes of workspace that q4_gemm_mx needs for M tokens or fewer (0: none,
    -1: it refuses the sizes)."""
    return int(load().q4_gemm_mx_workspace(int(M), int(N), int(K)))


def q4_gemm_experts_workspace(T: int, E: int, N: int, K: int) -> int:
    """Bytes of workspace that q4_gemm_experts needs for T rows or fewer (0: none,
    -1: it refuses the sizes)."""
    return int(load().q4_gemm_experts_workspace(int(T), int(E), int(N), int(K)))


def q4_gemm_mx(codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, y: torch.Tensor = None,
               N: int = None, dtype: torch.dtype = torch.float32, workspace: torch.Tensor = None,
               stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] @ W^T for any M, W a microscaled matrix, x bfloat16,
    y float32 or bfloat16 (y's type, or ``dtype``).  N defaults to whole
    blocks.  ``workspace`` (uint8, at least q4_gemm_mx_workspace bytes) is
    allocated if not given; one that is given must not be shared by calls
    that may overlap.

    x is held to 2^-22 of the largest |x| of each 32 k of a row, exactly where
    it is at least 2^-14 of that (the bound on y is in include/q4.h): rows in
    which a few x are more than 2^14 times their neighbours are better passed as
    two, the large x and the rest, and their results added."""
    _dims(x, "x", (2,), "[M, K]")
    M, K = x.shape
    E, N, K = _mx_sizes(codes, scales, N, K)
    if E is not None:
        raise ValueError("codes is a stack of matrices: use q4_gemm_experts")
    _operand(x, "x", _BF16, x.shape, codes)
    lib = load()
    if _elsewhere(codes, stream):
        with _Foreign(codes.get_device(), stream):
            return q4_gemm_mx(codes, scales, x, y, N, dtype, workspace)
    handle = torch._C._cuda_getCurrentRawStream(codes.get_device())
    if y is None:
        _type(dtype, _OUT, "dtype")
        y = torch.empty(M, N, dtype=dtype, device=codes.device)
    else:
        _operand(y, "y", _OUT, (M, N), codes)
    at, size, _hold = _scratch(workspace, lib.q4_gemm_mx_workspace(M, N, K), codes, "q4_gemm_mx")
    st = lib.q4_gemm_mx(codes.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(), _TYPE[y.dtype],
                        M, N, K, at, size, handle)
    _check(st, "q4_gemm_mx")
    return y


def q4_gemm_experts(codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                    rows: torch.Tensor = None, y: torch.Tensor = None, N: int = None,
                    dtype: torch.dtype = torch.float32, workspace: torch.Tensor = None,
                    stream=None) -> torch.Tensor:
    """y [T, N]: row p is x[rows[p]] @ W[e]^T for offsets[e] <= p <
    offsets[e + 1], with W [E] a stack of microscaled matrices, offsets
    [E + 1] and rows [T] int32 as q4_sort_experts makes them; zero for p >=
    offsets[E].  Without rows, x [T, K] is taken in order.  Other arguments as
    q4_gemm_mx."""
    _dims(x, "x", (2,), "[rows of x, K]")
    Mx, K = x.shape
    E, N, K = _mx_sizes(codes, scales, N, K)
    if E is None:
        raise ValueError("codes is one matrix: use q4_gemm_mx, or codes[None] and scales[None]")
    _operand(x, "x", _BF16, x.shape, codes)
    _operand(offsets, "offsets", _I32, (E + 1,), codes)
    T = Mx
    if rows is not None:
        _dims(rows, "rows", (1,), "[T]")
        _operand(rows, "rows", _I32, rows.shape, codes)
        T = rows.shape[0]
    lib = load()
    if _elsewhere(codes, stream):
        with _Foreign(codes.get_device(), stream):
            return q4_gemm_experts(codes, scales, x, offsets, rows, y, N, dtype, workspace)
    handle = torch._C._cuda_getCurrentRawStream(codes.get_device())
    if y is None:
        _type(dtype, _OUT, "dtype")
        y = torch.empty(T, N, dtype=dtype, device=codes.device)
    else:
        _operand(y, "y", _OUT, (T, N), codes)
    at, size, _hold = _scratch(workspace, lib.q4_gemm_experts_workspace(T, E, N, K), codes, "q4_gemm_experts")
    st = lib.q4_gemm_experts(codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                             None if rows is None else rows.data_ptr(), offsets.data_ptr(),
                             y.data_ptr(), _TYPE[y.dtype], Mx, T, E, N, K, at, size, handle)
    _check(st, "q4_gemm_experts")
    return y


def q4_sort_experts(ids: torch.Tensor, E: int, offsets: torch.Tensor = None, rows: torch.Tensor = None,
                    places: torch.Tensor = None, stream=None):
    """(offsets [E + 1], rows [T], places [M, top]), all int32: the stable order
    by expert of the choices ids [M, top] (int32 or int64), T = M * top.  Ids
    outside 0 .. E - 1 drop their choice: rows -1, places -1 - position."""
    _dims(ids, "ids", (2,), "[M, top]")
    M, top = ids.shape
    E = int(E)
    _operand(ids, "ids", _IDS, ids.shape, ids)
    if E < 1 or top < 1:
        raise ValueError(f"E = {E} and top = {top} must be at least 1")
    if _elsewhere(ids, stream):
        with _Foreign(ids.get_device(), stream):
            return q4_sort_experts(ids, E, offsets, rows, places)
    handle = torch._C._cuda_getCurrentRawStream(ids.get_device())
    if offsets is None:
        offsets = torch.empty(E + 1, dtype=torch.int32, device=ids.device)
    else:
        _operand(offsets, "offsets", _I32, (E + 1,), ids)
    if rows is None:
        rows = torch.empty(M * top, dtype=torch.int32, device=ids.device)
    else:
        _operand(rows, "rows", _I32, (M * top,), ids)
    if places is None:
        places = torch.empty(M, top, dtype=torch.int32, device=ids.device)
    else:
        _operand(places, "places", _I32, (M, top), ids)
    st = load().q4_sort_experts(ids.data_ptr(), int(ids.dtype == torch.int64), offsets.data_ptr(),
                                rows.data_ptr(), places.data_ptr(), M, top, E, handle)
    _check(st, "q4_sort_experts")
    return offsets, rows, places


def _row_sizes(t, name, places, rows_of_tokens: bool):
    """(M, top, K) of a row array and its places; the array has M rows, or M * top."""
    _dims(places, "places", (2,), "[M, top]")
    M, top = places.shape
    _dims(t, name, (2,), "[M, K]" if rows_of_tokens else "[M * top, K]")
    K = t.shape[1]
    _operand(t, name, _FLOATS, (M if rows_of_tokens else M * top, K), t)
    _operand(places, "places", _I32, places.shape, t)
    return M, top, K


def q4_dispatch(x: torch.Tensor, places: torch.Tensor, xs: torch.Tensor = None, stream=None) -> torch.Tensor:
    """xs [M * top, K]: the rows of x [M, K] at their choices' places, zeros at
    dropped ones.  The gradient is q4_combine(dxs, places)."""
    M, top, K = _row_sizes(x, "x", places, True)
    if _elsewhere(x, stream):
        with _Foreign(x.get_device(), stream):
            return q4_dispatch(x, places, xs)
    handle = torch._C._cuda_getCurrentRawStream(x.get_device())
    if xs is None:
        xs = torch.empty(M * top, K, dtype=x.dtype, device=x.device)
    else:
        _operand(xs, "xs", (x.dtype,), (M * top, K), x)
    st = load().q4_dispatch(x.data_ptr(), places.data_ptr(), xs.data_ptr(), _TYPE[x.dtype], M, top, K,
                            handle)
    _check(st, "q4_dispatch")
    return xs


def q4_combine(ys: torch.Tensor, places: torch.Tensor, weights: torch.Tensor = None,
               out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """out [M, K] = sum over a token's kept choices of weights[m, j] (float32;
    1 if None) * ys[places[m, j]], summed in float32.  The gradient is
    q4_combine_grad, without weights q4_dispatch(dout, places)."""
    M, top, K = _row_sizes(ys, "ys", places, False)
    if weights is not None:
        _operand(weights, "weights", _F32, (M, top), ys)
    if _elsewhere(ys, stream):
        with _Foreign(ys.get_device(), stream):
            return q4_combine(ys, places, weights, out)
    handle = torch._C._cuda_getCurrentRawStream(ys.get_device())
    if out is None:
        out = torch.empty(M, K, dtype=ys.dtype, device=ys.device)
    else:
        _operand(out, "out", (ys.dtype,), (M, K), ys)
    st = load().q4_combine(ys.data_ptr(), places.data_ptr(), None if weights is None else weights.data_ptr(),
                           out.data_ptr(), _TYPE[ys.dtype], M, top, K, handle)
    _check(st, "q4_combine")
    return out


def q4_combine_grad(dout: torch.Tensor, ys: torch.Tensor, places: torch.Tensor, weights: torch.Tensor,
                    dys: torch.Tensor = None, dweights: torch.Tensor = None, stream=None):
    """(dys [M * top, K], dweights [M, top] float32): the gradients of
    q4_combine(ys, places, weights) for dout [M, K]; zeros for dropped choices."""
    M, top, K = _row_sizes(ys, "ys", places, False)
    _operand(dout, "dout", (ys.dtype,), (M, K), ys)
    _operand(weights, "weights", _F32, (M, top), ys)
    if _elsewhere(ys, stream):
        with _Foreign(ys.get_device(), stream):
            return q4_combine_grad(dout, ys, places, weights, dys, dweights)
    handle = torch._C._cuda_getCurrentRawStream(ys.get_device())
    if dys is None:
        dys = torch.empty(M * top, K, dtype=ys.dtype, device=ys.device)
    else:
        _operand(dys, "dys", (ys.dtype,), (M * top, K), ys)
    if dweights is None:
        dweights = torch.empty(M, top, dtype=torch.float32, device=ys.device)
    else:
        _operand(dweights, "dweights", _F32, (M, top), ys)
    st = load().q4_combine_grad(dout.data_ptr(), ys.data_ptr(), places.data_ptr(), weights.data_ptr(),
                                dys.data_ptr(), dweights.data_ptr(), _TYPE[ys.dtype], M, top, K, handle)
    _check(st, "q4_combine_grad")
    return dys, dweights


def ring_slot_bytes(N: int, K: int) -> int:
    """Bytes a CopyRing slot needs for one [N, K] matrix (codes padded to 256
    bytes, then scales)."""
    return (N * (K // 2) + 255) // 256 * 256 + N * (K // GROUP) * 2


class Ring:
    """Two device slots fed from host memory ("CopyRing"): ``gemm`` copies a
    matrix's packed codes and scales from (pinned) host tensors into the next
    slot on the ring's copy stream and runs q4_gemm on it, so that the copy of
    one call overlaps the matmul of the previous one."""

    def __init__(self, slot_bytes: int):
        self._h = ctypes.c_void_p()
        _check(load().q4_ring_create(int(slot_bytes), ctypes.byref(self._h)), "q4_ring_create")

    def gemm(self, codes_host: torch.Tensor, scales_host: torch.Tensor, codebook: torch.Tensor,
             x: torch.Tensor, y: torch.Tensor = None, stream=None) -> torch.Tensor:
        if self._h.value is None:
            raise RuntimeError("ring is closed")
        if codes_host.dim() != 2:
            raise ValueError("codes must be [N, K/2]")
        N, K = codes_host.shape[0], codes_host.shape[1] * 2
        for t, name in ((codes_host, "codes_host"), (scales_host, "scales_host")):
            if t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous host tensor")
        if codes_host.dtype != torch.uint8 or scales_host.dtype not in _H16 or \
                tuple(scales_host.shape) != (N, K // GROUP):
            raise TypeError("codes_host uint8 [N, K/2], scales_host binary16 [N, K/64]")
        if x.dim() != 2 or x.shape[1] != K:
            raise ValueError(f"x must be [M, {K}]")
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, N), dtype=torch.float32, device=x.device)
        _need(codebook, "codebook", _H16, (16,))
        _need(x, "x", _BF16)
        _need(y, "y", (torch.float32,), (M, N))
        st = load().q4_ring_gemm(self._h, codes_host.data_ptr(), scales_host.data_ptr(),
                                 codebook.data_ptr(), x.data_ptr(), y.data_ptr(), M, N, K,
                                 _stream(x, stream))
        _check(st, "q4_ring_gemm")
        return y

    def close(self) -> None:
        if self._h.value is not None:
            _check(load().q4_ring_destroy(self._h), "q4_ring_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Step:
    """A decode step recorded once as a CUDA graph (q4_step_create) and
    replayed per token (``launch``).  ``linears`` is a sequence of
    (codes, scales, codebook, x, y) device tensors with the q4_gemm
    conventions; the graph keeps their addresses, so the caller keeps the
    tensors alive and writes each token's activations into the same x."""

    def __init__(self, linears):
        self._keep = []
        arr = (Q4Linear * len(linears))()
        for i, (codes, scales, codebook, x, y) in enumerate(linears):
            N, K = _packed_dims(codes)
            if x.dim() != 2 or x.shape[1] != K:
                raise ValueError(f"linear {i}: x must be [M, {K}]")
            M = x.shape[0]
            _need(codes, "codes", (torch.uint8,))
            _need(scales, "scales", _H16, (N, K // GROUP))
            _need(codebook, "codebook", _H16, (16,))
            _need(x, "x", _BF16)
            _need(y, "y", (torch.float32,), (M, N))
            arr[i] = Q4Linear(codes.data_ptr(), scales.data_ptr(), codebook.data_ptr(),
                              x.data_ptr(), y.data_ptr(), M, N, K)
            self._keep.append((codes, scales, codebook, x, y))
        self._device = self._keep[0][0].device if self._keep else None
        self._h = ctypes.c_void_p()
        _check(load().q4_step_create(arr, len(linears), ctypes.byref(self._h)), "q4_step_create")

    def launch(self, stream=None) -> None:
        if self._h.value is None:
            raise RuntimeError("step is closed")
        if stream is None:
            stream = torch.cuda.current_stream(self._device)
        s = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
        _check(load().q4_step_launch(self._h, s), "q4_step_launch")

    def close(self) -> None:
        if self._h.value is not None:
            _check(load().q4_step_destroy(self._h), "q4_step_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def wait_selftest(limit_us: int, arrive: bool) -> int:
    """Run the bounded-wait self-test kernel (synchronizes the device); returns
    the microseconds the wait took.  Without ``arrive`` the wait runs out and
    sets bit 7 of timeout_flags()."""
    out = ctypes.c_uint32(0)
    _check(load().q4_wait_selftest(int(limit_us), 1 if arrive else 0, ctypes.byref(out)),
           "q4_wait_selftest")
    return int(out.value)


def timeout_flags() -> int:
    """Synchronize the current device; return and clear the kernels' bounded-wait timeout bits."""
    out = ctypes.c_uint32(0)
    _check(load().q4_timeout_flags(ctypes.byref(out)), "q4_timeout_flags")
    return int(out.value)


def bounds_flags() -> int:
    """Synchronize the current device; return and clear the bits of the
    kernels' failed index checks (always 0 from the release build)."""
    out = ctypes.c_uint32(0)
    _check(load().q4_bounds_flags(ctypes.byref(out)), "q4_bounds_flags")
    return int(out.value)


def bounds_checked() -> bool:
    """True when the loaded library is the bounds-checked build."""
    return bool(load().q4_bounds_checked())


def abi_version() -> int:
    return load().q4_abi_version()


# ---- the C names, one Python function per entry point of include/q4.h ------

def q4_status_string(status: int) -> str:
    return status_string(status)


def q4_last_cuda_error() -> int:
    """The CUDA error code behind the calling thread's last Q4_ERR_CUDA."""
    return int(load().q4_last_cuda_error())


def q4_abi_version() -> int:
    return abi_version()


def q4_timeout_flags() -> int:
    return timeout_flags()


def q4_ring_create(slot_bytes: int) -> Ring:
    return Ring(slot_bytes)


def q4_ring_gemm(ring: Ring, codes_host, scales_host, codebook, x, y=None, stream=None):
    return ring.gemm(codes_host, scales_host, codebook, x, y, stream)


def q4_ring_destroy(ring: Ring) -> None:
    ring.close()


def q4_step_create(linears) -> Step:
    return Step(linears)


def q4_step_launch(step: Step, stream=None) -> None:
    step.launch(stream)


def q4_step_destroy(step: Step) -> None:
    step.close()


def q4_wait_selftest(limit_us: int, arrive: bool) -> int:
    return wait_selftest(limit_us, arrive)


def q4_bounds_flags() -> int:
    return bounds_flags()


def q4_bounds_checked() -> bool:
    return bounds_checked()
