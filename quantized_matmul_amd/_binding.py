"""ctypes binding of libqlin (argument marshalling only).

Pages followed for the user-facing defaults:
  "Emily.QuantizedWeight" from_dense options: group_size 64, bits 4,
      transpose true, mode "affine"; Microscaled modes table for the
      (group_size, bits) each microscaled mode pins.
  "EMLX.Quantization" gather_quantized_matmul: lhs_indices None takes the
      activation rows in order; sorted_indices lets the kernel skip its sort.
"""
import ctypes
import dataclasses
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libqlin.so")

# (group_size, bits) each microscaled mode pins ("Emily.QuantizedWeight")
MODE_DEFAULTS = {"affine": (64, 4), "mxfp4": (32, 4), "mxfp8": (32, 8), "nvfp4": (16, 4)}

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.uint8: 3}
_FLOATS = (torch.float32, torch.float16, torch.bfloat16)
_STATUS = {1: "invalid argument", 2: "unsupported", 3: "device error"}

_lib = None


class _CacheStruct(ctypes.Structure):
    """qlin_kv_cache."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "k_biases", "v_codes", "v_scales", "v_biases")]
                + [("mode", ctypes.c_char_p)]
                + [(n, ctypes.c_int64) for n in ("pages", "heads", "page_size", "head_dim")]
                + [(n, ctypes.c_int) for n in ("group_size", "bits", "dtype")])


class QlinError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"qlin {_STATUS.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libqlin.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, cs, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t
    lib.qlin_quantize.argtypes = [vp, i32, i64, i64, i32, i32, cs, vp, vp, vp, vp]
    lib.qlin_dequantize.argtypes = [vp, vp, vp, i32, i64, i64, i32, i32, cs, vp, i32, vp]
    lib.qlin_quantized_matmul.argtypes = [vp, i32, i64, i64, vp, vp, vp, i32, i64, i32, i32, i32,
                                          cs, vp, vp]
    lib.qlin_quantized_dense.argtypes = [vp, i32, i64, i64, vp, vp, vp, i32, i64, i32, i32, i32,
                                         cs, vp, i32, ctypes.c_double, vp, vp]
    lib.qlin_gather_qmm.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, i32, i64, i64, vp, vp,
                                    i64, i32, i32, i32, cs, i32, vp, sz, vp, vp]
    lib.qlin_quantized_matmul_ws.argtypes = [vp, i32, i64, i64, vp, vp, vp, i32, i64, i32, i32,
                                             i32, cs, vp, sz, vp, vp]
    lib.qlin_quantized_matmul_ws.restype = i32
    lib.qlin_quantized_matmul_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32, cs]
    lib.qlin_quantized_matmul_workspace_bytes.restype = sz
    lib.qlin_qqmm.argtypes = [vp, i32, i64, i64, vp, vp, i64, i32, i32, i32, cs, vp, sz, vp, vp]
    lib.qlin_qqmm.restype = i32
    lib.qlin_qqmm_workspace_bytes.argtypes = [i64, i64]
    lib.qlin_qqmm_workspace_bytes.restype = sz
    lib.qlin_gather_qmm_workspace_bytes.argtypes = [i64, i64]
    lib.qlin_gather_qmm_workspace_bytes.restype = sz
    lib.qlin_gather_qmm_noalloc.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, i32, i64, i64,
                                            vp, vp, i64, i32, i32, i32, cs, i32, vp, vp]
    lib.qlin_gather_qmm_noalloc.restype = i32
    lib.qlin_gather_qmm_noalloc_max_rows.restype = sz
    lib.qlin_gather_qmm_noalloc_max_experts.restype = sz
    f64 = ctypes.c_double
    lib.qlin_moe_route.argtypes = [vp, i32, i64, i64, i64, vp, cs, i32, f64, i64, i64, i32, vp, vp, vp]
    lib.qlin_moe_route_grad.argtypes = [vp, i32, i64, i64, i64, vp, vp, cs, i32, f64, vp, vp]
    lib.qlin_mxfp4_matmul.argtypes = [vp, i32, vp, cs, i64, i64, vp, vp, i64, vp, sz, vp, i32, vp]
    lib.qlin_mxfp4_matmul_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.qlin_mxfp4_matmul_workspace_bytes.restype = sz
    lib.qlin_gather_mxfp4_matmul.argtypes = [vp, i32, vp, cs, i64, i64, vp, vp, i64, i64, vp, i64, vp,
                                             sz, vp, i32, vp]
    lib.qlin_gather_mxfp4_matmul_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32]
    lib.qlin_gather_mxfp4_matmul_workspace_bytes.restype = sz
    lib.qlin_moe_combine.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp]
    lib.qlin_moe_combine_grad.argtypes = [vp, vp, i32, i64, i64, i64, vp, vp, vp, vp, vp]
    cache = vp
    lib.qlin_rotary.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, vp, i32, f64, vp, i64, vp]
    lib.qlin_rotary_grad.argtypes = lib.qlin_rotary.argtypes
    lib.qlin_kv_cache_write.argtypes = [cache, vp, vp, i32, i64, i64, i64, vp, vp]
    lib.qlin_kv_cache_read.argtypes = [cache, vp, i64, vp, vp, i32, vp]
    lib.qlin_kv_cache_attention.argtypes = [cache, vp, i32, i64, i64, i64, vp, i64, i64, vp, vp, f64, i32, i64,
                                            vp, sz, vp, vp]
    lib.qlin_kv_cache_attention_workspace_bytes.argtypes = [cache, i32, i64, i64, i64, i64, i32, i64]
    lib.qlin_kv_cache_attention_workspace_bytes.restype = sz
    lib.qlin_last_error.restype = ctypes.c_char_p
    lib.qlin_last_path.restype = ctypes.c_char_p
    for f in ("qlin_quantize", "qlin_dequantize", "qlin_quantized_matmul", "qlin_quantized_dense",
              "qlin_gather_qmm", "qlin_moe_route", "qlin_moe_route_grad", "qlin_mxfp4_matmul",
              "qlin_gather_mxfp4_matmul", "qlin_moe_combine", "qlin_moe_combine_grad", "qlin_rotary",
              "qlin_rotary_grad", "qlin_kv_cache_write", "qlin_kv_cache_read", "qlin_kv_cache_attention"):
        getattr(lib, f).restype = i32
    _lib = lib
    return lib


def last_path() -> str:
    """Kernel path of this thread's last matmul-type call (qlin_last_path)."""
    return (load_library().qlin_last_path() or b"").decode()


def _check(rc: int):
    if rc != 0:
        raise QlinError(rc, (_lib.qlin_last_error() or b"").decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> int:
    """The device's current HIP stream (hipStream_t as an integer)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _dev(t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError("qlin tensors live in GPU memory (got a CPU tensor)")
    if not t.is_contiguous():
        raise ValueError("qlin tensors must be contiguous")
    return t.device


@dataclasses.dataclass
class QuantizedWeight:
    """Packed weight plus metadata ("Emily.QuantizedWeight", t() type)."""
    value: torch.Tensor            # uint32 codes, stored as torch.int32
    scales: torch.Tensor
    biases: Optional[torch.Tensor]
    group_size: int
    bits: int
    transpose: bool = True
    mode: str = "affine"

    @property
    def shape(self):
        """Logical (dense) shape."""
        return tuple(self.value.shape[:-1]) + (self.value.shape[-1] * 32 // self.bits,)


def quantize(w: torch.Tensor, group_size: Optional[int] = None, bits: Optional[int] = None,
             mode: str = "affine", transpose: bool = True) -> QuantizedWeight:
    """qlin_quantize on a rank >= 2 tensor, along its last axis."""
    lib = load_library()
    dev = _dev(w)
    if w.dim() < 2:
        raise ValueError("quantize needs a tensor of rank >= 2")
    g0, b0 = MODE_DEFAULTS.get(mode, (64, 4))
    group_size = g0 if group_size is None else group_size
    bits = b0 if bits is None else bits
    if w.dtype not in (torch.float32, torch.float16, torch.bfloat16):
        raise ValueError("w must be float32, float16 or bfloat16")
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    lead = tuple(w.shape[:-1])
    wq = torch.empty(lead + (max(cols * bits // 32, 0),), dtype=torch.int32, device=dev)
    G = cols // group_size if group_size > 0 else 0
    if mode == "affine":
        scales = torch.empty(lead + (G,), dtype=w.dtype, device=dev)
        biases = torch.empty_like(scales)
    else:
        scales = torch.empty(lead + (G,), dtype=torch.uint8, device=dev)
        biases = None
    rc = lib.qlin_quantize(_ptr(w), _DTYPE[w.dtype], rows, cols, group_size, bits, mode.encode(),
                           _ptr(wq), _ptr(scales), _ptr(biases), _stream(dev))
    _check(rc)
    return QuantizedWeight(wq, scales, biases, group_size, bits, transpose, mode)


def dequantize(qw: QuantizedWeight, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """qlin_dequantize: dense weight of the logical shape (default dtype: the
    scales dtype for affine, float32 for microscaled)."""
    lib = load_library()
    dev = _dev(qw.value)
    if dtype is None:
        dtype = qw.scales.dtype if qw.mode == "affine" else torch.float32
    cols = qw.value.shape[-1] * 32 // qw.bits
    rows = qw.value.numel() // qw.value.shape[-1] if qw.value.shape[-1] else 0
    out = torch.empty(tuple(qw.value.shape[:-1]) + (cols,), dtype=dtype, device=dev)
    rc = lib.qlin_dequantize(_ptr(qw.value), _ptr(qw.scales), _ptr(qw.biases),
                             _DTYPE[qw.scales.dtype], rows, cols, qw.group_size, qw.bits,
                             qw.mode.encode(), _ptr(out), _DTYPE[dtype], _stream(dev))
    _check(rc)
    return out


def _out(out, shape, dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or not out.is_contiguous() \
            or out.device != dev:
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")
    return out


def quantized_matmul_workspace_bytes(M: int, K: int, N: int, transpose: bool, group_size: int,
                                     bits: int, mode: str = "affine") -> int:
    """qlin_quantized_matmul_workspace_bytes (0: the shape takes none)."""
    return int(load_library().qlin_quantized_matmul_workspace_bytes(
        M, K, N, int(transpose), group_size, bits, mode.encode()))


# Zeroed workspaces for the K-split [in, out] calls, one per (device,
# stream): the library keeps completion counters at the start of the
# workspace, which must be zero before the first call and which every call
# leaves zero, so a workspace is zeroed once (on its stream) and then reused
# by the calls of that stream, which never overlap.
_SPLIT_WS = {}


def _split_workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    stream = torch.cuda.current_stream(dev)
    key = (dev.index, stream.cuda_stream)
    ws = _SPLIT_WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        _SPLIT_WS[key] = ws
    return ws


def quantized_matmul(x: torch.Tensor, qw: QuantizedWeight,
                     out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_quantized_matmul: x [..., K] -> y [..., N] in x's dtype.

    W is 2-D: [N, K] packed along K when qw.transpose, else [K, N] packed
    along N ("Emily.Quantization.Layers", quantized_dense). Shapes that take
    a workspace (the [in, out] layout at few bf16 rows, where K is split over
    workgroups) use one zeroed workspace per device and stream, kept for
    later calls, unless `workspace` (a uint8 device tensor whose first 4096
    bytes are zero before its first use) is given; the call then goes to
    qlin_quantized_matmul_ws.
    """
    lib = load_library()
    dev = _dev(x)
    _dev(qw.value)
    if qw.value.dim() != 2:
        raise ValueError("quantized_matmul takes a 2-D quantized weight")
    per = 32 // qw.bits
    if qw.transpose:
        N, K = qw.value.shape[0], qw.value.shape[1] * per
    else:
        K, N = qw.value.shape[0], qw.value.shape[1] * per
    if x.shape[-1] != K:
        raise ValueError(f"x's last dim {x.shape[-1]} does not match the weight's K={K}")
    M = x.numel() // K if K else 0
    y = _out(out, tuple(x.shape[:-1]) + (N,), x.dtype, dev)
    ws_bytes = 0
    if workspace is not None:
        _dev(workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    elif not qw.transpose and x.dtype == torch.bfloat16 and 1 <= M <= 8:
        ws_bytes = quantized_matmul_workspace_bytes(M, K, N, False, qw.group_size, qw.bits, qw.mode)
        if ws_bytes:
            workspace = _split_workspace(dev, ws_bytes)
            ws_bytes = workspace.numel()
    if ws_bytes:
        rc = lib.qlin_quantized_matmul_ws(_ptr(x), _DTYPE[x.dtype], M, K, _ptr(qw.value),
                                          _ptr(qw.scales), _ptr(qw.biases),
                                          _DTYPE[qw.scales.dtype], N, int(qw.transpose),
                                          qw.group_size, qw.bits, qw.mode.encode(),
                                          _ptr(workspace), ws_bytes, _ptr(y), _stream(dev))
    else:
        rc = lib.qlin_quantized_matmul(_ptr(x), _DTYPE[x.dtype], M, K, _ptr(qw.value),
                                       _ptr(qw.scales), _ptr(qw.biases), _DTYPE[qw.scales.dtype],
                                       N, int(qw.transpose), qw.group_size, qw.bits,
                                       qw.mode.encode(), _ptr(y), _stream(dev))
    _check(rc)
    return y


def quantized_dense(x: torch.Tensor, qw: QuantizedWeight, bias=0,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_quantized_dense: x @ W (+ bias) ("Emily.Quantization.Layers",
    quantized_dense). bias is a number, or a float tensor of N values (one
    per output column) on x's device; it is added in fp32 before the output's
    one rounding.
    """
    lib = load_library()
    dev = _dev(x)
    _dev(qw.value)
    if qw.value.dim() != 2:
        raise ValueError("quantized_dense takes a 2-D quantized weight")
    per = 32 // qw.bits
    if qw.transpose:
        N, K = qw.value.shape[0], qw.value.shape[1] * per
    else:
        K, N = qw.value.shape[0], qw.value.shape[1] * per
    if x.shape[-1] != K:
        raise ValueError(f"x's last dim {x.shape[-1]} does not match the weight's K={K}")
    bias_t, bias_value, bias_dt = None, 0.0, _DTYPE[torch.float32]
    if isinstance(bias, torch.Tensor):
        _dev(bias)
        if bias.device != dev:
            raise ValueError("bias must be on x's device")
        if bias.numel() != N or bias.dim() < 1 or bias.shape[-1] != N:
            raise ValueError(f"a tensor bias holds one value per output column ({N})")
        if bias.dtype not in (torch.float32, torch.bfloat16, torch.float16):
            raise ValueError("bias must be float32, bfloat16 or float16")
        bias_t = bias.contiguous()
        bias_dt = _DTYPE[bias_t.dtype]
    else:
        bias_value = float(bias)
    M = x.numel() // K if K else 0
    y = _out(out, tuple(x.shape[:-1]) + (N,), x.dtype, dev)
    rc = lib.qlin_quantized_dense(_ptr(x), _DTYPE[x.dtype], M, K, _ptr(qw.value),
                                  _ptr(qw.scales), _ptr(qw.biases), _DTYPE[qw.scales.dtype], N,
                                  int(qw.transpose), qw.group_size, qw.bits, qw.mode.encode(),
                                  _ptr(bias_t), bias_dt, bias_value, _ptr(y), _stream(dev))
    _check(rc)
    return y


def qqmm_workspace_bytes(M: int, K: int) -> int:
    return int(load_library().qlin_qqmm_workspace_bytes(M, K))


def qqmm(x: torch.Tensor, qw: QuantizedWeight, workspace: Optional[torch.Tensor] = None,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_qqmm (mlx-rs qqmm): bf16 x quantized on the fly with qw's mode
    (nvfp4 or mxfp8), times the quantized weight. x [..., K] -> y [..., N]."""
    lib = load_library()
    dev = _dev(x)
    _dev(qw.value)
    if qw.value.dim() != 2:
        raise ValueError("qqmm takes a 2-D quantized weight")
    per = 32 // qw.bits
    if qw.transpose:
        N, K = qw.value.shape[0], qw.value.shape[1] * per
    else:
        K, N = qw.value.shape[0], qw.value.shape[1] * per
    if x.shape[-1] != K:
        raise ValueError(f"x's last dim {x.shape[-1]} does not match the weight's K={K}")
    M = x.numel() // K if K else 0
    need = qqmm_workspace_bytes(M, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    y = _out(out, tuple(x.shape[:-1]) + (N,), x.dtype, dev)
    rc = lib.qlin_qqmm(_ptr(x), _DTYPE[x.dtype], M, K, _ptr(qw.value), _ptr(qw.scales), N,
                       int(qw.transpose), qw.group_size, qw.bits, qw.mode.encode(),
                       _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(y),
                       _stream(dev))
    _check(rc)
    return y


def gather_qmm_workspace_bytes(R: int, E: int) -> int:
    return int(load_library().qlin_gather_qmm_workspace_bytes(R, E))


def _gather_prep(x, qw, rhs_indices, lhs_indices):
    """Shapes and flattened int32 index arrays of a gather call (no copy
    when the indices are already contiguous int32 tensors on x's device and
    lhs, if given, has rhs's shape)."""
    dev = _dev(x)
    if x.dim() != 3 or qw.value.dim() != 3:
        raise ValueError("gather_qmm takes x [B, M, K] and a stacked weight [E, ., .]")
    B, M, K = x.shape
    E = qw.value.shape[0]
    per = 32 // qw.bits
    N = qw.value.shape[1] if qw.transpose else qw.value.shape[2] * per
    Kw = qw.value.shape[2] * per if qw.transpose else qw.value.shape[1]
    if Kw != K:
        raise ValueError(f"x's last dim {K} does not match the weight's K={Kw}")
    rhs = rhs_indices.to(device=dev, dtype=torch.int32)
    shape = tuple(rhs.shape)
    lhs = None
    if lhs_indices is not None:
        lhs_b, rhs_b = torch.broadcast_tensors(lhs_indices.to(device=dev, dtype=torch.int32), rhs)
        shape = tuple(rhs_b.shape)
        lhs = lhs_b.contiguous().reshape(-1)
        rhs = rhs_b.contiguous().reshape(-1)
    else:
        rhs = rhs.contiguous().reshape(-1)
    return dev, B, M, K, E, N, shape, lhs, rhs


def gather_qmm(x: torch.Tensor, qw: QuantizedWeight, rhs_indices: torch.Tensor,
               lhs_indices: Optional[torch.Tensor] = None, sorted_indices: bool = False,
               workspace: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_gather_qmm: y[r] = x[lhs[r]] . W[rhs[r]]^T (or . W[rhs[r]]).

    x [B, M, K]; qw.value stacks experts on its leading axis; rhs_indices
    (and lhs_indices, broadcast against it) of any shape S. Returns
    y of shape S + (M, N). ("EMLX.Quantization", gather_quantized_matmul.)
    """
    lib = load_library()
    dev, B, M, K, E, N, shape, lhs, rhs = _gather_prep(x, qw, rhs_indices, lhs_indices)
    R = rhs.numel()
    need = int(lib.qlin_gather_qmm_workspace_bytes(R, E))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    y = _out(out, shape + (M, N), x.dtype, dev)
    rc = lib.qlin_gather_qmm(_ptr(x), _DTYPE[x.dtype], B, M, K, _ptr(qw.value), _ptr(qw.scales),
                             _ptr(qw.biases), _DTYPE[qw.scales.dtype], E, N, _ptr(lhs), _ptr(rhs),
                             R, int(qw.transpose), qw.group_size, qw.bits, qw.mode.encode(),
                             int(bool(sorted_indices)), _ptr(workspace), workspace.numel(),
                             _ptr(y), _stream(dev))
    _check(rc)
    return y


def gather_qmm_noalloc(x: torch.Tensor, qw: QuantizedWeight, rhs_indices: torch.Tensor,
                       lhs_indices: Optional[torch.Tensor] = None, sorted_indices: bool = False,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_gather_qmm_noalloc: gather_qmm with the library's own fixed
    scratch instead of a workspace (at most 65536 index rows and 4096
    experts). The C call allocates nothing; this wrapper allocates only y
    when `out` is not given and index copies when the indices are not
    contiguous int32 tensors of one shape on x's device."""
    lib = load_library()
    dev, B, M, K, E, N, shape, lhs, rhs = _gather_prep(x, qw, rhs_indices, lhs_indices)
    R = rhs.numel()
    y = _out(out, shape + (M, N), x.dtype, dev)
    rc = lib.qlin_gather_qmm_noalloc(_ptr(x), _DTYPE[x.dtype], B, M, K, _ptr(qw.value),
                                     _ptr(qw.scales), _ptr(qw.biases), _DTYPE[qw.scales.dtype], E,
                                     N, _ptr(lhs), _ptr(rhs), R, int(qw.transpose), qw.group_size,
                                     qw.bits, qw.mode.encode(), int(bool(sorted_indices)), _ptr(y),
                                     _stream(dev))
    _check(rc)
    return y


def _check_tensor(name, t, dev, dtype):
    """t is a contiguous tensor of dtype on dev."""
    if t.dtype is dtype and t.is_contiguous() and t.device == dev:
        return
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev} (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _float_code(name, t):
    code = _DTYPE.get(t.dtype, 3)
    if code == 3:
        raise ValueError(f"{name} must be float32, float16 or bfloat16")
    return code


def moe_route(logits: torch.Tensor, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              renormalize: bool = True, scale: float = 1.0, groups: int = 1, groups_kept: int = 1,
              group_top: int = 1):
    """qlin_moe_route: the k experts of each token and their weights.

    logits [..., E]; bias float32 [E] (for the choice only). Returns
    (weights float32 [..., k], experts int32 [..., k]), best first, equal
    ones by ascending index; a place no expert can take holds -1 and 0.
    """
    lib = _lib or load_library()
    dev = _dev(logits)
    code = _float_code("logits", logits)
    shape = logits.shape
    if not shape:
        raise ValueError("logits has a last axis of experts")
    E = shape[-1]
    if bias is not None:
        _check_tensor("bias", bias, dev, torch.float32)
        if bias.shape != (E,):
            raise ValueError(f"bias must hold one value per expert ({E})")
    T = logits.numel() // E if E else 0
    shape = (*shape[:-1], max(k, 0))
    weights = torch.empty(*shape, dtype=torch.float32, device=dev)
    experts = torch.empty(*shape, dtype=torch.int32, device=dev)
    _check(lib.qlin_moe_route(logits.data_ptr(), code, T, E, k, None if bias is None else bias.data_ptr(),
                              score.encode(), renormalize, scale, groups, groups_kept, group_top,
                              weights.data_ptr(), experts.data_ptr(), _stream(dev)))
    return weights, experts


def moe_route_grad(logits: torch.Tensor, experts: torch.Tensor, grad_weights: torch.Tensor,
                   score: str = "softmax", renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """qlin_moe_route_grad: gradient of moe_route's weights with respect to
    logits, in logits' dtype; experts is moe_route's output for them."""
    lib = _lib or load_library()
    dev = _dev(logits)
    code = _float_code("logits", logits)
    _check_tensor("experts", experts, dev, torch.int32)
    _check_tensor("grad_weights", grad_weights, dev, torch.float32)
    if not logits.shape or experts.shape != grad_weights.shape or experts.shape[:-1] != logits.shape[:-1]:
        raise ValueError("experts and grad_weights are [..., k] for logits [..., E]")
    E = logits.shape[-1]
    out = torch.empty_like(logits)
    _check(lib.qlin_moe_route_grad(logits.data_ptr(), code, logits.numel() // E if E else 0, E,
                                   experts.shape[-1], experts.data_ptr(), grad_weights.data_ptr(),
                                   score.encode(), renormalize, scale, out.data_ptr(), _stream(dev)))
    return out


def _mxfp4_operands(x, qw, activation, dim):
    """Device, x's tensor, scales and type code, y's default dtype, K and N of an mxfp4 product."""
    value, wscales = qw.value, qw.scales
    shape = value.shape
    if qw.mode != "mxfp4" or not qw.transpose or len(shape) != dim:
        raise ValueError(f"the weight must be a {dim}-D mxfp4 weight in the [out, in] layout")
    K, N = shape[-1] * 8, shape[-2]
    if isinstance(x, QuantizedWeight):
        if x.mode != "mxfp4":
            raise ValueError("a quantized x must be mxfp4")
        t, scales, code, dtype, wide = x.value, x.scales, 3, torch.bfloat16, K // 8
        dev = _dev(t)
        _check_tensor("x's words", t, dev, torch.int32)
        _check_tensor("x's scales", scales, dev, torch.uint8)
        if scales.numel() * 4 != t.numel():
            raise ValueError("x's scales do not fit its words")
    else:
        t, scales, code, dtype = x, None, _float_code("x", x), x.dtype
        dev = _dev(t)
        wide = 2 * K if activation == "swiglu" else K
    _check_tensor("the weight's words", value, dev, torch.int32)
    _check_tensor("the weight's scales", wscales, dev, torch.uint8)
    if not K or not t.shape or t.shape[-1] != wide:
        raise ValueError(f"x's last dim {t.shape[-1] if t.shape else None} does not match the weight's K={K}"
                         + (" (twice K with swiglu)" if activation == "swiglu" else ""))
    if wscales.numel() * 4 != value.numel():
        raise ValueError("the weight's scales do not fit its words")
    return dev, t, scales, code, dtype, K, N


def _workspace(workspace, need, dev):
    """(tensor, address, bytes) of the given workspace, or of a new one; the tensor keeps it alive."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace, workspace.data_ptr(), need
    if _dev(workspace) != dev:
        raise ValueError(f"workspace must be on {dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def mxfp4_matmul_workspace_bytes(M: int, K: int, N: int, x_dtype: torch.dtype = torch.bfloat16) -> int:
    """qlin_mxfp4_matmul_workspace_bytes; torch.uint8 stands for an x given as codes."""
    return int(load_library().qlin_mxfp4_matmul_workspace_bytes(M, K, N, _DTYPE[x_dtype]))


def mxfp4_matmul(x, qw: QuantizedWeight, activation: Optional[str] = None,
                 out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_mxfp4_matmul: x [..., K] times an mxfp4 weight [N, K], both as
    4-bit codes on the scaled MFMA.

    x is a float tensor, quantized to mxfp4 on the way (with activation
    "swiglu": x [..., 2K], silu of its first half times its second), or an
    mxfp4 QuantizedWeight that holds the activation's codes. y takes
    out_dtype, by default x's (bfloat16 for codes).
    """
    lib = _lib or load_library()
    dev, t, scales, code, dtype, K, N = _mxfp4_operands(x, qw, activation, 2)
    M = t.numel() // t.shape[-1]
    if out_dtype is not None:
        dtype = out_dtype
    y = torch.empty(*t.shape[:-1], N, dtype=dtype, device=dev) if out is None else _out(out, (*t.shape[:-1], N), dtype, dev)
    keep, ws, ws_bytes = _workspace(workspace, lib.qlin_mxfp4_matmul_workspace_bytes(M, K, N, code), dev)
    _check(lib.qlin_mxfp4_matmul(t.data_ptr(), code, None if scales is None else scales.data_ptr(),
                                 activation.encode() if activation else None, M, K, qw.value.data_ptr(),
                                 qw.scales.data_ptr(), N, ws, ws_bytes, y.data_ptr(), _DTYPE[dtype],
                                 _stream(dev)))
    return y


def gather_mxfp4_matmul_workspace_bytes(B: int, R: int, K: int, E: int, N: int,
                                        x_dtype: torch.dtype = torch.bfloat16) -> int:
    """qlin_gather_mxfp4_matmul_workspace_bytes; torch.uint8 stands for codes."""
    return int(load_library().qlin_gather_mxfp4_matmul_workspace_bytes(B, R, K, E, N, _DTYPE[x_dtype]))


def gather_mxfp4_matmul(x, qw: QuantizedWeight, experts: torch.Tensor, activation: Optional[str] = None,
                        out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_gather_mxfp4_matmul: y[r] = x[r // (R / B)] . W[experts[r]]^T.

    x [B, K] (or [B, 2K] with "swiglu", or mxfp4 codes) as for mxfp4_matmul;
    qw stacks experts [E, N, K]; experts int32 [B, ...], the experts of each
    row of x. Returns y of shape experts.shape + (N,); a row whose expert is
    outside [0, E) is zeros.
    """
    lib = _lib or load_library()
    dev, t, scales, code, dtype, K, N = _mxfp4_operands(x, qw, activation, 3)
    _check_tensor("experts", experts, dev, torch.int32)
    if t.dim() != 2 or not experts.shape or experts.shape[0] != t.shape[0]:
        raise ValueError("gather_mxfp4_matmul takes x [B, K] and experts [B, ...]")
    B, R, E = t.shape[0], experts.numel(), qw.value.shape[0]
    if out_dtype is not None:
        dtype = out_dtype
    y = torch.empty(*experts.shape, N, dtype=dtype, device=dev) if out is None else _out(out, (*experts.shape, N), dtype, dev)
    keep, ws, ws_bytes = _workspace(
        workspace, lib.qlin_gather_mxfp4_matmul_workspace_bytes(B, R, K, E, N, code), dev)
    _check(lib.qlin_gather_mxfp4_matmul(t.data_ptr(), code, None if scales is None else scales.data_ptr(),
                                        activation.encode() if activation else None, B, K,
                                        qw.value.data_ptr(), qw.scales.data_ptr(), E, N, experts.data_ptr(),
                                        R, ws, ws_bytes, y.data_ptr(), _DTYPE[dtype], _stream(dev)))
    return y


def _combine_operands(h, weights, experts):
    dev = _dev(h)
    code = _float_code("h", h)
    shape = h.shape
    if len(shape) < 2 or weights.shape != shape[:-1] or (experts is not None and experts.shape != shape[:-1]):
        raise ValueError("moe_combine takes h [..., k, D] with weights (and experts) [..., k]")
    _check_tensor("weights", weights, dev, torch.float32)
    if experts is not None:
        _check_tensor("experts", experts, dev, torch.int32)
        experts = experts.data_ptr()
    k = shape[-2]
    return dev, code, (weights.numel() // k if k else 0), k, shape[-1], experts


def moe_combine(h: torch.Tensor, weights: torch.Tensor, experts: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_moe_combine: y[..., :] = sum over j of weights[..., j] * h[..., j, :],
    places with a negative expert left out."""
    lib = _lib or load_library()
    dev, code, T, k, D, ids = _combine_operands(h, weights, experts)
    y = torch.empty(*h.shape[:-2], D, dtype=h.dtype, device=dev) if out is None else _out(out, (*h.shape[:-2], D), h.dtype, dev)
    _check(lib.qlin_moe_combine(h.data_ptr(), code, T, k, D, weights.data_ptr(), ids, y.data_ptr(),
                                _stream(dev)))
    return y


def moe_combine_grad(grad_y: torch.Tensor, h: torch.Tensor, weights: torch.Tensor,
                     experts: Optional[torch.Tensor] = None):
    """qlin_moe_combine_grad: (grad_h in h's dtype, grad_weights float32)."""
    lib = _lib or load_library()
    dev, code, T, k, D, ids = _combine_operands(h, weights, experts)
    _check_tensor("grad_y", grad_y, dev, h.dtype)
    if grad_y.shape != (*h.shape[:-2], D):
        raise ValueError(f"grad_y must have the shape {(*h.shape[:-2], D)}")
    grad_h = torch.empty_like(h)
    grad_w = torch.empty_like(weights)
    _check(lib.qlin_moe_combine_grad(grad_y.data_ptr(), h.data_ptr(), code, T, k, D, weights.data_ptr(), ids,
                                     grad_h.data_ptr(), grad_w.data_ptr(), _stream(dev)))
    return grad_h, grad_w


_current_device = torch._C._cuda_getDevice


def _elsewhere(dev, f, args):
    """f(*args, stream) with dev, which is not the current device, made it for the call."""
    with torch.cuda.device(dev):
        return f(*args, _stream(dev))


def _token_rows(name, t, dev, dtype, heads, dim, tokens):
    """Elements between the tokens of t [tokens, heads, dim], whose heads and values are dense (None: any size)."""
    shape, strides = t.shape, t.stride()
    if (t.dtype is dtype and len(shape) == 3 and t.device == dev and strides[2] == 1 and strides[1] == shape[2]
            and (heads is None or shape[1] == heads) and (dim is None or shape[2] == dim)
            and (tokens is None or shape[0] == tokens)):
        return strides[0] if shape[0] > 1 else shape[1] * shape[2]
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev} (got {t.device})")
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (dim is not None and shape[2] != dim) \
            or (tokens is not None and shape[0] != tokens):
        raise ValueError(f"{name} must be [{'T' if tokens is None else tokens}, {'heads' if heads is None else heads}, "
                         f"{'head_dim' if dim is None else dim}] (got {tuple(shape)})")
    if (strides[2] != 1 and shape[2] > 1) or (strides[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"the heads and values of {name} must be dense (only its tokens may lie apart)")
    return strides[0] if shape[0] > 1 else shape[1] * shape[2]


def _index_rows(name, t, dev, n):
    if t.dtype is torch.int32 and t.device == dev and t.is_contiguous() and len(t.shape) == 1 \
            and (n is None or t.shape[0] == n):
        return
    _check_tensor(name, t, dev, torch.int32)
    raise ValueError(f"{name} must be one-dimensional" + ("" if n is None else f" with {n} entries"))


def rotary_frequencies(dim: int, base: float = 10000.0, factor: float = 1.0, method: str = "linear",
                       trained: int = 4096, slow: float = 1.0, fast: float = 32.0, device="cuda") -> torch.Tensor:
    """Angles of a step for rotary, float32 [dim / 2]: base ** (-2 i / dim), scaled for contexts `factor` times the
    trained one.

    method "linear" divides all of them by factor; "base" raises the base to base * factor ** (dim / (dim - 2)), which
    leaves the first and divides the last by factor; "parts" divides those that turn at most `slow` times in `trained`
    tokens, leaves those that turn `fast` times or more, and mixes the two in between, evenly in the turns.
    """
    if dim < 2 or dim % 2:
        raise ValueError("dim must be even and positive")
    if not factor > 0 or not base > 0:
        raise ValueError("base and factor must be positive")
    i = torch.arange(0, dim, 2, dtype=torch.float64)
    if method == "base":
        if dim < 4:
            raise ValueError('method "base" needs dim of 4 or more')
        base = base * factor ** (dim / (dim - 2))
    freqs = base ** (-i / dim)
    if method == "linear":
        freqs = freqs / factor
    elif method == "parts":
        if not fast > slow:
            raise ValueError("fast must be above slow")
        keep = ((trained * freqs / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        freqs = freqs * keep + freqs / factor * (1 - keep)
    elif method != "base":
        raise ValueError(f'unknown method "{method}" (linear, base, parts)')
    return freqs.float().to(device)


def _rotary(call, name, x, positions, freqs, interleaved, scale, out):
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("qlin tensors live in GPU memory (got a CPU tensor)")
    code = _float_code(name, x)
    stride = _token_rows(name, x, dev, x.dtype, None, None, None)
    T, heads, D = x.shape
    _index_rows("positions", positions, dev, T)
    _check_tensor("freqs", freqs, dev, torch.float32)
    if len(freqs.shape) != 1:
        raise ValueError("freqs must be one-dimensional")
    if out is None:
        out = torch.empty((T, heads, D), dtype=x.dtype, device=dev)
        out_stride = heads * D
    else:
        out_stride = _token_rows("out", out, dev, x.dtype, heads, D, T)
    args = (x.data_ptr(), code, T, stride, heads, D, 2 * freqs.shape[0], positions.data_ptr(), freqs.data_ptr(),
            interleaved, scale, out.data_ptr(), out_stride)
    rc = call(*args, _stream(dev)) if dev.index == _current_device() else _elsewhere(dev, call, args)
    if rc:
        _check(rc)
    return out


def rotary(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool = False,
           scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_rotary: the first 2 * len(freqs) values of each head of x [T, heads, D] turned in pairs by
    positions[t] * freqs[i] (pairs (i, i + len(freqs)), or neighbours where interleaved) and multiplied by scale, the
    rest copied.

    positions int32 [T], freqs float32 (rotary_frequencies). x's tokens may lie apart, as the heads of a projection's
    rows do; so may out's, and out may be x.
    """
    return _rotary((_lib or load_library()).qlin_rotary, "x", x, positions, freqs, interleaved, scale, out)


def rotary_grad(grad_y: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool = False,
                scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_rotary_grad: gradient of rotary with respect to x."""
    return _rotary((_lib or load_library()).qlin_rotary_grad, "grad_y", grad_y, positions, freqs, interleaved, scale, out)


class KVCache:
    """Attention keys and values held in 4 bits (qlin_kv_cache): two pools [pages, heads, page_size, head_dim],
    quantized along head_dim as `quantize` does it ("affine" with 4 bits, "mxfp4" or "nvfp4").

    key and value are their QuantizedWeights (`dequantize` takes them). Slot p * page_size + o is place o of page p.
    """

    def __init__(self, key: QuantizedWeight, value: QuantizedWeight):
        if (key.mode, key.group_size, key.bits) != (value.mode, value.group_size, value.bits):
            raise ValueError("keys and values must be quantized alike")
        dev = _dev(key.value)
        dtype = key.scales.dtype
        lead = tuple(key.value.shape)
        if len(lead) != 4:
            raise ValueError("a cache's words are [pages, heads, page_size, head_dim / 8]")
        if key.group_size < 1 or lead[3] * 8 % key.group_size:
            raise ValueError("head_dim must be a multiple of group_size")
        groups = lead[:3] + (lead[3] * 8 // key.group_size,)
        affine = key.mode == "affine"
        if affine and dtype not in _FLOATS:
            raise ValueError("an affine cache's scales must be float32, float16 or bfloat16")
        for side, w in (("key", key), ("value", value)):
            _check_tensor(f"the {side} words", w.value, dev, torch.int32)
            _check_tensor(f"the {side} scales", w.scales, dev, dtype if affine else torch.uint8)
            if tuple(w.value.shape) != lead or tuple(w.scales.shape) != groups:
                raise ValueError(f"the {side} words and scales must be {lead} and {groups}")
            if (w.biases is not None) != affine:
                raise ValueError("affine caches have biases, others have none")
            if affine:
                _check_tensor(f"the {side} biases", w.biases, dev, dtype)
                if tuple(w.biases.shape) != groups:
                    raise ValueError(f"the {side} biases must be {groups}")
        self.pages, self.heads, self.page_size = lead[:3]
        self.head_dim = lead[3] * 8
        self.group_size, self.bits, self.mode, self.device = key.group_size, key.bits, key.mode, dev
        self.dtype = dtype if affine else None      # of an affine cache's scales, and so of its rows
        # the tensors themselves are kept, so that the addresses below stay theirs
        self._parts = tuple(t for w in (key, value) for t in (w.value, w.scales, w.biases))
        self._struct = _CacheStruct(*[None if t is None else t.data_ptr() for t in self._parts], self.mode.encode(),
                                    self.pages, self.heads, self.page_size, self.head_dim, self.group_size, self.bits,
                                    _DTYPE[dtype])
        self._address = ctypes.addressof(self._struct)

    @property
    def key(self) -> QuantizedWeight:
        return QuantizedWeight(*self._parts[:3], self.group_size, self.bits, True, self.mode)

    @property
    def value(self) -> QuantizedWeight:
        return QuantizedWeight(*self._parts[3:], self.group_size, self.bits, True, self.mode)


def kv_cache(pages: int, heads: int, page_size: int, head_dim: int, group_size: Optional[int] = None,
             mode: str = "affine", dtype: torch.dtype = torch.bfloat16, device="cuda") -> KVCache:
    """An empty KVCache; dtype is that of an affine cache's scales and rows."""
    group_size = MODE_DEFAULTS.get(mode, (64, 4))[0] if group_size is None else group_size
    if group_size < 1 or head_dim < 1 or head_dim % group_size:
        raise ValueError("head_dim must be a multiple of group_size")
    lead = (pages, heads, page_size)
    groups = lead + (head_dim // group_size,)

    def pool():
        scales = torch.zeros(groups, dtype=dtype if mode == "affine" else torch.uint8, device=device)
        return QuantizedWeight(torch.zeros(lead + (head_dim // 8,), dtype=torch.int32, device=device), scales,
                               torch.zeros_like(scales) if mode == "affine" else None, group_size, 4, True, mode)

    return KVCache(pool(), pool())


def kv_cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """qlin_kv_cache_write: k and v [T, heads, head_dim] quantized into the cache, token t into slot slots[t].

    slots int32 [T]; one outside the pool (-1) is left out, and none may come twice. The tokens of k and v may lie
    apart, as in a projection's rows.
    """
    lib = _lib or load_library()
    dev = cache.device
    code = _float_code("k", k)
    k_stride = _token_rows("k", k, dev, cache.dtype or k.dtype, cache.heads, cache.head_dim, None)
    T = k.shape[0]
    v_stride = _token_rows("v", v, dev, k.dtype, cache.heads, cache.head_dim, T)
    _index_rows("slots", slots, dev, T)
    args = (cache._address, k.data_ptr(), v.data_ptr(), code, T, k_stride, v_stride, slots.data_ptr())
    call = lib.qlin_kv_cache_write
    rc = call(*args, _stream(dev)) if dev.index == _current_device() else _elsewhere(dev, call, args)
    if rc:
        _check(rc)


def kv_cache_read(cache: KVCache, slots: torch.Tensor, dtype: Optional[torch.dtype] = None):
    """qlin_kv_cache_read: (k, v) [T, heads, head_dim] of the rows at slots (int32 [T]), zeros for slots outside the
    pool; dtype by default the scales' for affine, float32 otherwise, as for dequantize."""
    lib = _lib or load_library()
    dev = cache.device
    _index_rows("slots", slots, dev, None)
    dtype = dtype or cache.dtype or torch.float32
    if dtype not in _FLOATS:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    shape = (slots.shape[0], cache.heads, cache.head_dim)
    k = torch.empty(shape, dtype=dtype, device=dev)
    v = torch.empty(shape, dtype=dtype, device=dev)
    args = (cache._address, slots.data_ptr(), shape[0], k.data_ptr(), v.data_ptr(), _DTYPE[dtype])
    call = lib.qlin_kv_cache_read
    rc = call(*args, _stream(dev)) if dev.index == _current_device() else _elsewhere(dev, call, args)
    if rc:
        _check(rc)
    return k, v


def kv_cache_attention_workspace_bytes(cache: KVCache, T: int, q_heads: int, B: int, width: int, has_offsets: bool,
                                       window: int = 0, dtype: Optional[torch.dtype] = None) -> int:
    """qlin_kv_cache_attention_workspace_bytes for q [T, q_heads, head_dim] of dtype (an affine cache's own, else bfloat16,
    by default)."""
    return int(load_library().qlin_kv_cache_attention_workspace_bytes(
        cache._address, _DTYPE[dtype or cache.dtype or torch.bfloat16], T, q_heads, B, width, int(has_offsets), window))


def kv_cache_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lengths: torch.Tensor,
                       offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = True,
                       window: int = 0, workspace: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qlin_kv_cache_attention: attention of q [T, q_heads, head_dim] to the keys of its sequences in the cache.

    Sequence b has lengths[b] keys (int32 [B]), in the pages table[b] (int32 [B, width]) names; its rows of q are
    offsets[b] to offsets[b + 1] (int32 [B + 1]), the last of them at its last key, or row b alone without offsets.
    causal hides the keys behind a row's place, window > 0 those that many or more before it. scale is
    head_dim ** -0.5 by default. Rows of no sequence are left as they are in out (zeros without out); rows that see no
    key become zeros. Prompts take a workspace by the table's width, not the lengths (up to 8 GiB; qlin.h): a table no
    wider than the longest sequence keeps it small.
    """
    lib = _lib or load_library()
    dev = cache.device
    code = _float_code("q", q)
    q_stride = _token_rows("q", q, dev, cache.dtype or q.dtype, None, cache.head_dim, None)
    T, heads, D = q.shape
    _check_tensor("table", table, dev, torch.int32)
    if len(table.shape) != 2:
        raise ValueError("table must be [B, width]")
    B, width = table.shape
    _index_rows("lengths", lengths, dev, B)
    if offsets is not None:
        _index_rows("offsets", offsets, dev, B + 1)
    if out is None:
        # with offsets there may be rows of no sequence
        out = (torch.empty if offsets is None else torch.zeros)((T, heads, D), dtype=q.dtype, device=dev)
    else:
        out = _out(out, (T, heads, D), q.dtype, dev)
    keep, ws, ws_bytes = _workspace(workspace, lib.qlin_kv_cache_attention_workspace_bytes(
        cache._address, code, T, heads, B, width, offsets is not None, window), dev)
    args = (cache._address, q.data_ptr(), code, T, q_stride, heads, table.data_ptr(), B, width, lengths.data_ptr(),
            None if offsets is None else offsets.data_ptr(), D ** -0.5 if scale is None else scale, causal, window, ws,
            ws_bytes, out.data_ptr())
    call = lib.qlin_kv_cache_attention
    rc = call(*args, _stream(dev)) if dev.index == _current_device() else _elsewhere(dev, call, args)
    if rc:
        _check(rc)
    return out
