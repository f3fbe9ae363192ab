"""ctypes binding of libexl3 (include/exl3.h).

Argument marshalling only: every step of the product runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  If the
shared library is missing this module raises on import -- there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# EXL3_LIBRARY selects another build of the library, e.g. the debug-bounds
# build libexl3_debug.so next to this file.
LIB_PATH = os.environ.get("EXL3_LIBRARY") or os.path.join(_HERE, "libexl3.so")

EXL3_OK = 0
EXL3_ERR_INVALID_ARG = 1
EXL3_ERR_UNSUPPORTED = 2
EXL3_ERR_MISALIGNED = 3
EXL3_ERR_WORKSPACE = 4
EXL3_ERR_ARCH = 5
EXL3_ERR_CUDA = 6
EXL3_ERR_TIMEOUT = 7
EXL3_ERR_BOUNDS = 8
EXL3_ERR_CACHE_FULL = 9
EXL3_ERR_INDEX = 10

# every entry point include/exl3.h declares
EXPORTS = ("exl3_status_string", "exl3_last_cuda_error", "exl3_version", "exl3_workspace_bytes",
           "exl3_workspace_status", "exl3_kernel_launches", "exl3_decode_tiles", "exl3_hadamard128", "exl3_gemv",
           "exl3_gemm_small_m", "exl3_gemm_siblings", "exl3_large_m_workspace_bytes", "exl3_gemm_large_m",
           "exl3_gemv_noalloc", "exl3_grouped_workspace_bytes", "exl3_gemm_grouped", "exl3_q4_workspace_bytes",
           "exl3_q4_gemm", "exl3_q4_pack", "exl3_kv_scratch_bytes", "exl3_kv_reset", "exl3_kv_status",
           "exl3_kv_extend", "exl3_kv_write", "exl3_kv_truncate", "exl3_kv_fork", "exl3_kv_compact",
           "exl3_paged_attention_workspace_bytes", "exl3_paged_attention_launches",
           "exl3_paged_attention")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libexl3.so not built ({LIB_PATH}); run `python -m gemm_exl3_gemv_b200.build`")

lib = ctypes.CDLL(LIB_PATH)
_P, _I, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
lib.exl3_status_string.argtypes = [_I]
lib.exl3_status_string.restype = ctypes.c_char_p
lib.exl3_last_cuda_error.argtypes = []
lib.exl3_last_cuda_error.restype = _I
lib.exl3_version.argtypes = []
lib.exl3_version.restype = _I
lib.exl3_workspace_bytes.argtypes = [_I, _I, _I, _I]
lib.exl3_workspace_bytes.restype = _Z
lib.exl3_kernel_launches.argtypes = [_I, _I, _I, _I]
lib.exl3_kernel_launches.restype = _I
lib.exl3_workspace_status.argtypes = [_P, _P]
lib.exl3_workspace_status.restype = _I
lib.exl3_decode_tiles.argtypes = [_P, _I, _I, _I, _P, _P]
lib.exl3_decode_tiles.restype = _I
lib.exl3_hadamard128.argtypes = [_P, _P, _P, _I, _I, _I, _P]
lib.exl3_hadamard128.restype = _I
lib.exl3_gemv.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P]
lib.exl3_gemv.restype = _I
lib.exl3_gemm_small_m.argtypes = [_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P]
lib.exl3_gemm_small_m.restype = _I
lib.exl3_gemv_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]


class Matrix(ctypes.Structure):
    """exl3_matrix_t: one member of a sibling group (device pointers)."""
    _fields_ = [("packed", _P), ("scale", _P), ("sv", _P), ("y", _P), ("n_out", _I)]


lib.exl3_gemm_siblings.argtypes = [_I, _P, _P, ctypes.POINTER(Matrix), _I, _I, _I, _I, _P, _Z, _P]
lib.exl3_gemm_siblings.restype = _I
lib.exl3_large_m_workspace_bytes.argtypes = [_I, _I, _I, _I]
lib.exl3_large_m_workspace_bytes.restype = _Z
lib.exl3_gemm_large_m.argtypes = [_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P]
lib.exl3_gemm_large_m.restype = _I
lib.exl3_gemv_noalloc.restype = _I


class Problem(ctypes.Structure):
    """exl3_problem_t: one member of a grouped call (device pointers)."""
    _fields_ = [("x", _P), ("su", _P), ("packed", _P), ("scale", _P), ("sv", _P), ("y", _P),
                ("k_in", _I), ("n_out", _I)]


lib.exl3_grouped_workspace_bytes.argtypes = [_I, ctypes.POINTER(Problem), _I, _I]
lib.exl3_grouped_workspace_bytes.restype = _Z
lib.exl3_gemm_grouped.argtypes = [_I, ctypes.POINTER(Problem), _I, _I, _I, _P, _Z, _P]
lib.exl3_gemm_grouped.restype = _I

_L, _F = ctypes.c_longlong, ctypes.c_float
lib.exl3_q4_workspace_bytes.argtypes = [_I, _I, _I]
lib.exl3_q4_workspace_bytes.restype = _Z
lib.exl3_q4_gemm.argtypes = [_I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _Z, _P]
lib.exl3_q4_gemm.restype = _I
lib.exl3_q4_pack.argtypes = [_P, _I, _I, _P, _P]
lib.exl3_q4_pack.restype = _I


class Cache(ctypes.Structure):
    """exl3_kv_cache_t: a paged key-value cache (device pointers and sizes)."""
    _fields_ = [("k", _P), ("v", _P), ("table", _P), ("lens", _P), ("refs", _P), ("free", _P), ("scratch", _P),
                ("n_layers", _I), ("n_pages", _I), ("n_heads", _I), ("page_size", _I), ("head_dim", _I),
                ("n_seqs", _I), ("max_pages", _I)]


# the cache argument is a pointer to a Cache (ctypes.byref)
lib.exl3_kv_scratch_bytes.argtypes = [_I]
lib.exl3_kv_scratch_bytes.restype = _Z
lib.exl3_kv_reset.argtypes = [_P, _P]
lib.exl3_kv_status.argtypes = [_P, _P]
lib.exl3_kv_extend.argtypes = [_P, _I, _I, _P, _P, _P]
lib.exl3_kv_write.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _L, _L, _P]
lib.exl3_kv_truncate.argtypes = [_P, _I, _P, _P, _P]
lib.exl3_kv_fork.argtypes = [_P, _I, _P, _P, _P]
lib.exl3_kv_compact.argtypes = [_P, _P]
lib.exl3_paged_attention_workspace_bytes.argtypes = [_I, _I, _I, _I]
lib.exl3_paged_attention_workspace_bytes.restype = _Z
lib.exl3_paged_attention.argtypes = [_P, _I, _I, _I, _P, _P, _P, _L, _L, _I, _F, _I, _I, _P, _L, _L, _P, _P, _Z, _P]
for _name in ("reset", "status", "extend", "write", "truncate", "fork", "compact"):
    getattr(lib, "exl3_kv_" + _name).restype = _I
lib.exl3_paged_attention.restype = _I
lib.exl3_paged_attention_launches.argtypes = [_P, _I, _I, _I]
lib.exl3_paged_attention_launches.restype = _I


class _CtypesBinding:
    """The calls of csrc/binding.c through ctypes, with its checks of the
    arguments' number and types: 1 to 3 us slower a call, and needs no compiler."""
    NAMES = ("exl3_q4_gemm", "exl3_kv_extend", "exl3_kv_write", "exl3_kv_truncate", "exl3_kv_fork", "exl3_kv_compact",
             "exl3_paged_attention")

    def __init__(self):
        for name in self.NAMES:
            setattr(self, name[len("exl3_"):], self._checked(name))

    @staticmethod
    def _checked(name):
        call = getattr(lib, name)
        types = tuple(call.argtypes)

        def checked(*args):
            if len(args) != len(types):
                raise TypeError(f"{name}: takes {len(types)} arguments, got {len(args)}")
            values = [a if a is None and t is _P else float(a) if t is _F else operator.index(a) for a, t in zip(args, types)]
            for a, t in zip(values, types):
                if t is _I and not -1 << 31 <= a < 1 << 31:
                    raise OverflowError("argument does not fit a C int")       # ctypes would cut it off
            return call(*values)
        return checked


# The same entry points of the same library without ctypes' conversions, which
# cost a small call up to a quarter of its time (csrc/binding.c).  It is built
# for one Python; without it the calls go through ctypes.
try:
    from . import _binding
    _binding.bind([ctypes.cast(getattr(lib, _name), _P).value for _name in _binding.NAMES])
except ImportError:
    _binding = _CtypesBinding()


class Exl3Error(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = lib.exl3_status_string(status).decode()
        if status == EXL3_ERR_CUDA:
            msg += f" (cudaError {lib.exl3_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")
        self.status = status


def _check(status: int, what: str):
    if status != EXL3_OK:
        raise Exl3Error(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object around it: 0.1 us a call
# instead of 3.3 us, of a small call's 10.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
# the same for the current device (CUDA is initialised: there is a tensor on a GPU)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream=None):
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def workspace_bytes(m: int, k_in: int, n_out: int, bits: int) -> int:
    return int(lib.exl3_workspace_bytes(m, k_in, n_out, bits))


def kernel_launches(m: int, k_in: int, n_out: int, bits: int) -> int:
    return int(lib.exl3_kernel_launches(m, k_in, n_out, bits))


def alloc_workspace(m: int, k_in: int, n_out: int, bits: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) for problems up to this size."""
    n = workspace_bytes(m, k_in, n_out, bits)
    if n == 0:
        raise Exl3Error(EXL3_ERR_UNSUPPORTED, "workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    return int(lib.exl3_workspace_status(_ptr(ws), _stream(stream)))


def decode_tiles(packed: torch.Tensor, k_in: int, n_out: int, bits: int,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decoded weights, k_in x n_out fp16."""
    if out is None:
        out = torch.empty((k_in, n_out), dtype=torch.float16, device=packed.device)
    _check(lib.exl3_decode_tiles(_ptr(packed), k_in, n_out, bits, _ptr(out), _stream(stream)),
           "exl3_decode_tiles")
    return out


def hadamard128(x: torch.Tensor, signs: torch.Tensor, mode: int = 0,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """mode 0: H(signs*x); mode 1: signs*H(x); x is rows x n fp16."""
    x2 = x if x.dim() == 2 else x.reshape(1, -1)
    if out is None:
        out = torch.empty_like(x2)
    _check(lib.exl3_hadamard128(_ptr(x2), _ptr(out), _ptr(signs), x2.shape[0], x2.shape[1], mode,
                                _stream(stream)), "exl3_hadamard128")
    return out if x.dim() == 2 else out.reshape(x.shape)


def gemm(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, su: torch.Tensor,
         sv: torch.Tensor, bits: int, out: Optional[torch.Tensor] = None, fp32: bool = False,
         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = sv*H(scale*(H(su*x) W)) for x of shape (m, k_in) (m <= 32) or (k_in,)."""
    squeeze = x.dim() == 1
    x2 = x.reshape(1, -1) if squeeze else x
    m, k_in = x2.shape
    n_out = scale.shape[0]
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.float32 if fp32 else torch.float16, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(m, k_in, n_out, bits, device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if m == 1:
        st = lib.exl3_gemv(_ptr(x2), _ptr(packed), _ptr(scale), _ptr(su), _ptr(sv), _ptr(out),
                           int(fp32), k_in, n_out, bits, _ptr(workspace), ws_bytes, _stream(stream))
        _check(st, "exl3_gemv")
    else:
        st = lib.exl3_gemm_small_m(m, _ptr(x2), _ptr(packed), _ptr(scale), _ptr(su), _ptr(sv),
                                   _ptr(out), int(fp32), k_in, n_out, bits, _ptr(workspace),
                                   ws_bytes, _stream(stream))
        _check(st, "exl3_gemm_small_m")
    return out.reshape(-1) if squeeze else out


def gemm_siblings(x: torch.Tensor, su: torch.Tensor, mats, bits: int, outs=None, fp32: bool = False,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Products of one input with a group of matrices in one pass.  `mats` is a
    list of (packed, scale, sv); returns the list of outputs (m, n_out_i)."""
    squeeze = x.dim() == 1
    x2 = x.reshape(1, -1) if squeeze else x
    m, k_in = x2.shape
    if outs is None:
        outs = [torch.empty((m, sc.shape[0]), dtype=torch.float32 if fp32 else torch.float16, device=x.device)
                for (_, sc, _) in mats]
    n_total = sum(int(sc.shape[0]) for (_, sc, _) in mats)
    if workspace is None:
        workspace = alloc_workspace(m, k_in, n_total, bits, device=x.device)
    arr = (Matrix * len(mats))()
    for i, ((packed, scale, sv), y) in enumerate(zip(mats, outs)):
        arr[i] = Matrix(packed.data_ptr(), scale.data_ptr(), sv.data_ptr(), y.data_ptr(), int(scale.shape[0]))
    st = lib.exl3_gemm_siblings(m, _ptr(x2), _ptr(su), arr, len(mats), int(fp32), k_in, bits, _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "exl3_gemm_siblings")
    return [o.reshape(-1) for o in outs] if squeeze else outs


def gemm_large(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, su: torch.Tensor, sv: torch.Tensor,
               bits: int, out: Optional[torch.Tensor] = None, fp32: bool = False,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The product for many rows (x: m x k_in), decoding W once per call."""
    m, k_in = x.shape
    n_out = scale.shape[0]
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.float32 if fp32 else torch.float16, device=x.device)
    if workspace is None:
        n = int(lib.exl3_large_m_workspace_bytes(m, k_in, n_out, bits))
        if n == 0:
            raise Exl3Error(EXL3_ERR_UNSUPPORTED, "exl3_large_m_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=x.device)
    st = lib.exl3_gemm_large_m(m, _ptr(x), _ptr(packed), _ptr(scale), _ptr(su), _ptr(sv), _ptr(out), int(fp32),
                               k_in, n_out, bits, _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    _check(st, "exl3_gemm_large_m")
    return out



def grouped_workspace_bytes(m: int, shapes, bits: int) -> int:
    """Workspace of a grouped call for members of shapes [(k_in, n_out), ...]."""
    arr = (Problem * len(shapes))()
    for i, (k, n) in enumerate(shapes):
        arr[i] = Problem(None, None, None, None, None, None, int(k), int(n))
    return int(lib.exl3_grouped_workspace_bytes(m, arr, len(shapes), bits))


def grouped_kernel_launches(m: int) -> int:
    """Kernel launches of one grouped call: the product (m = 1), or the
    rotation pre-pass and the product (m >= 2)."""
    return 1 if m == 1 else 2


def gemm_grouped(problems, bits: int, fp32: bool = False, workspace: Optional[torch.Tensor] = None,
                 stream=None):
    """Products of independent problems in one pass.  `problems` is a list of
    (x, packed, scale, su, sv, y) device tensors, x of shape (m, k_in) (or
    (k_in,) for m = 1) and y of shape (m, n_out); returns the list of y."""
    arr = (Problem * len(problems))()
    m = None
    shapes = []
    for i, (x, packed, scale, su, sv, y) in enumerate(problems):
        x2 = x.reshape(1, -1) if x.dim() == 1 else x
        if m is None:
            m = x2.shape[0]
        k_in, n_out = x2.shape[1], scale.shape[0]
        shapes.append((k_in, n_out))
        arr[i] = Problem(x2.data_ptr(), su.data_ptr(), packed.data_ptr(), scale.data_ptr(), sv.data_ptr(),
                         y.data_ptr(), int(k_in), int(n_out))
    if workspace is None:
        n = grouped_workspace_bytes(m, shapes, bits)
        if n == 0:
            raise Exl3Error(EXL3_ERR_UNSUPPORTED, "exl3_grouped_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=problems[0][0].device)
    st = lib.exl3_gemm_grouped(m, arr, len(problems), int(fp32), bits, _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "exl3_gemm_grouped")
    return [p[5] for p in problems]


# ------------------------------------------------- plain 4-bit weights ---

_F16, _I32, _U8 = torch.float16, torch.int32, torch.uint8
_q4_gemm = _binding.q4_gemm


def _dense(t: torch.Tensor, dtype, shape, device: int) -> bool:
    """Whether t is a contiguous tensor of this type and shape on that GPU."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device


def _expect(t: torch.Tensor, what: str, dtype, shape, device: Optional[int] = None):
    """ValueError unless t is a contiguous tensor of this type and shape on the
    given GPU (default: the current one)."""
    device = torch.cuda.current_device() if device is None and t.is_cuda else device
    if device is None or not _dense(t, dtype, shape, device):
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{'the current CUDA device' if device is None else f'cuda:{device}'}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ' (not contiguous)'}")


def _room(ws: torch.Tensor, device: int) -> int:
    """Bytes of a workspace tensor."""
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{device}")
    return ws.nbytes


def q4_workspace_bytes(m: int, k_in: int, n_out: int) -> int:
    return int(lib.exl3_q4_workspace_bytes(m, k_in, n_out))


def q4_alloc_workspace(m: int, k_in: int, n_out: int, device=None) -> torch.Tensor:
    """Zero-filled workspace (uint8) for a 4-bit product of this size."""
    n = q4_workspace_bytes(m, k_in, n_out)
    if n == 0:
        raise Exl3Error(EXL3_ERR_UNSUPPORTED, "q4_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def q4_pack(q: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """4-bit values (k_in, n_out) uint8 in the layout of ``q4_gemm``:
    (n_out/16, k_in/64, 32, 4) int32.  Once per matrix, when it is loaded."""
    if stream is not None and out is None:
        with torch.cuda.stream(stream):                 # what is allocated here belongs to the stream that uses it
            return q4_pack(q)
    if q.dim() != 2:
        raise ValueError("q: expected (k_in, n_out)")
    k_in, n_out = q.shape
    _expect(q, "q", torch.uint8, (k_in, n_out))
    if out is None:
        out = torch.empty((n_out // 16, k_in // 64, 32, 4), dtype=torch.int32, device=q.device)
    else:
        _expect(out, "out", torch.int32, (n_out // 16, k_in // 64, 32, 4))
    _check(lib.exl3_q4_pack(_ptr(q), k_in, n_out, _ptr(out), _stream(stream)), "exl3_q4_pack")
    return out


def q4_gemm(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor] = None,
            group: int = 128, out: Optional[torch.Tensor] = None, fp32: bool = False,
            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[i, n] = sum_k x[i, k] (q[k, n] - zero[k // group, n]) scale[k // group, n]
    for x of shape (m, k_in), m <= 32, or (k_in,).  packed: from ``q4_pack``;
    scale: (k_in / group, n_out) fp16; zero: the same in uint8 (0..15), None
    for 8 everywhere.  Inference only: there is no backward pass."""
    if stream is not None and (out is None or workspace is None):
        with torch.cuda.stream(stream):                 # what is allocated here belongs to the stream that uses it
            return q4_gemm(x, packed, scale, zero, group, out, fp32, workspace)
    squeeze = x.dim() == 1
    x2 = x.reshape(1, -1) if squeeze else x
    device = x.get_device()
    if x2.dim() != 2 or packed.dim() != 4 or device < 0 or device != _current_device():
        raise ValueError("expected x of (m, k_in) or (k_in,) on the current CUDA device and packed of "
                         "(n_out/16, k_in/64, 32, 4)")
    (m, k_in), tiles = x2.shape, packed.shape[0]
    n_out = 16 * tiles
    if group not in (32, 64, 128) or k_in % group or k_in % 64 or not 1 <= m <= 32:
        raise Exl3Error(EXL3_ERR_UNSUPPORTED, f"q4_gemm of {m} rows, k_in {k_in}, group {group}")
    groups = (k_in // group, n_out)
    # one condition on the usual path: a call of a small product is bound by the host
    if not (x2.dtype is _F16 and packed.dtype is _I32 and scale.dtype is _F16 and x2.is_contiguous() and
            packed.is_contiguous() and scale.is_contiguous() and packed.shape == (tiles, k_in // 64, 32, 4) and
            scale.shape == groups and packed.get_device() == device and scale.get_device() == device and
            (zero is None or zero.dtype is _U8 and zero.shape == groups and zero.is_contiguous() and
             zero.get_device() == device)):
        _expect(x2, "x", torch.float16, (m, k_in), device)
        _expect(packed, "packed", torch.int32, (tiles, k_in // 64, 32, 4), device)
        _expect(scale, "scale", torch.float16, groups, device)
        _expect(zero, "zero", torch.uint8, groups, device)
    if out is None:
        out = x2.new_empty((m, n_out), dtype=torch.float32) if fp32 else x2.new_empty((m, n_out))
    else:
        if squeeze and out.dim() == 1:
            out = out.view(1, -1)
        _expect(out, "out", torch.float32 if fp32 else torch.float16, (m, n_out), device)
    if workspace is None:
        workspace = q4_alloc_workspace(m, k_in, n_out, device=x.device)
    st = _q4_gemm(m, x2.data_ptr(), packed.data_ptr(), scale.data_ptr(),
                          None if zero is None else zero.data_ptr(), out.data_ptr(), 1 if fp32 else 0, k_in, n_out, group,
                          workspace.data_ptr(), _room(workspace, device),
                          _raw_stream(device) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "exl3_q4_gemm")
    return out.reshape(-1) if squeeze else out
