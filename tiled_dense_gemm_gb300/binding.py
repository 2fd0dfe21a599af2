"""ctypes binding to libgemmrelu.so (argument marshalling only).

Every step of the computation runs in the CUDA library; this module checks
tensor properties, passes raw pointers, sizes and the current CUDA stream,
and turns status codes into exceptions.  There is no CPU fallback: if the
library is missing or the device is not a GB300 (sm_103a), calls raise.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

from .build import INCLUDE, LIB_PATH

GEMM_OK = 0
STATUS_NAMES = {
    0: "GEMM_OK", 1: "GEMM_ERR_INVALID_ARG", 2: "GEMM_ERR_ALIGNMENT",
    3: "GEMM_ERR_UNSUPPORTED_DEVICE", 4: "GEMM_ERR_OUT_OF_MEMORY", 5: "GEMM_ERR_LAUNCH",
    6: "GEMM_ERR_TIMEOUT", 7: "GEMM_ERR_CUDA", 8: "GEMM_ERR_TOO_LARGE", 9: "GEMM_ERR_INDEX",
}


class GemmReluError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}" if what else
                         STATUS_NAMES.get(status, str(status)))


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "path", "mma_m", "mma_n", "tile_m", "tile_n", "tiles_m", "tiles_n", "num_tiles",
        "num_kb", "block_k", "group_m", "grid", "cluster", "dp_tiles", "sk_tiles", "sk_q", "sk_r",
        "splits", "max_slots", "num_stages", "stage_bytes", "smem_bytes", "tmem_cols", "pack_a")] + [
        ("workspace_bytes", ctypes.c_int64), ("counter_count", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {n: getattr(self, n) for n, _ in self._fields_}


_lock = threading.Lock()
_lib = None


class Boxes(ctypes.Structure):
    """gemm_relu_boxes_t: the TMA boxes of one ring stage's copies."""
    _fields_ = [("a_3d", ctypes.c_int32), ("a_box", ctypes.c_uint32 * 3), ("b_3d", ctypes.c_int32),
                ("b_box", ctypes.c_uint32 * 3), ("b2_box", ctypes.c_uint32 * 2), ("b_view_inner", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {"a_3d": self.a_3d, "a_box": list(self.a_box), "b_3d": self.b_3d, "b_box": list(self.b_box),
                "b2_box": list(self.b2_box), "b_view_inner": self.b_view_inner}


def declared_functions() -> list[str]:
    """Names of the functions include/gemm_relu.h declares."""
    text = open(os.path.join(INCLUDE, "gemm_relu.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gemm_relu\w*)\s*\(", text)))


def lib():
    """Load libgemmrelu.so (built by ``__graft_entry__.build()`` or
    ``python -m tiled_dense_gemm_gb300.build``).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it first "
                               "(python -m tiled_dense_gemm_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.gemm_relu.restype = i32
        L.gemm_relu.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
        L.gemm_relu_ex.restype = i32
        L.gemm_relu_ex.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, i32, vp]
        L.gemm_relu_host.restype = i32
        L.gemm_relu_host.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
        L.gemm_relu_noalloc.restype = i32
        L.gemm_relu_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
        L.gemm_relu_noalloc_check_device_error.restype = i32
        L.gemm_relu_noalloc_check_device_error.argtypes = [vp]
        L.gemm_relu_check_device_error.restype = i32
        L.gemm_relu_check_device_error.argtypes = [vp]
        L.gemm_relu_status_string.restype = ctypes.c_char_p
        L.gemm_relu_status_string.argtypes = [i32]
        L.gemm_relu_shutdown.restype = None
        L.gemm_relu_shutdown.argtypes = []
        L.gemm_relu_grouped.restype = i32
        L.gemm_relu_grouped.argtypes = [vp] * 4 + [i64] * 6 + [i32] * 3 + [vp]
        L.gemm_relu_grouped_dx.restype = i32
        L.gemm_relu_grouped_dx.argtypes = [vp] * 5 + [i64] * 7 + [i32] * 2 + [vp]
        L.gemm_relu_grouped_dw.restype = i32
        L.gemm_relu_grouped_dw.argtypes = [vp] * 4 + [i64] * 6 + [i32] * 2 + [vp]
        L.gemm_relu_adapters.restype = i32
        L.gemm_relu_adapters.argtypes = [vp] * 7 + [i64] * 7 + [i32] * 3 + [vp]
        f32 = ctypes.c_float
        L.gemm_relu_loss_workspace.restype = i64
        L.gemm_relu_loss_workspace.argtypes = [i64] * 4 + [i32]
        L.gemm_relu_xent.restype = i32
        L.gemm_relu_xent.argtypes = [vp] * 5 + [i64] * 4 + [i32] * 2 + [vp, i64, vp]
        L.gemm_relu_xent_grad.restype = i32
        L.gemm_relu_xent_grad.argtypes = [vp] * 5 + [i64, vp, vp] + [i64] * 5 + [i32] * 2 + [vp, i64, vp]
        L.gemm_relu_distill.restype = i32
        L.gemm_relu_distill.argtypes = [vp] * 4 + [f32, vp, vp] + [i64] * 7 + [i32] * 3 + [vp, i64, vp]
        L.gemm_relu_distill_grad.restype = i32
        L.gemm_relu_distill_grad.argtypes = [vp] * 4 + [f32, vp, vp, i64, vp, vp] + [i64] * 8 + [i32] * 3 + [vp, i64, vp]
        L.gemm_relu_plan.restype = i32
        L.gemm_relu_plan.argtypes = [i64, i64, i64, i32, ctypes.POINTER(Plan)]
        p32 = ctypes.POINTER(ctypes.c_int32)
        L.gemm_relu_plan_boxes.restype = i32
        L.gemm_relu_plan_boxes.argtypes = [ctypes.POINTER(Plan), i64, i64, i64, i32, ctypes.POINTER(Boxes)]
        L.gemm_relu_plan_work_item.restype = i32
        L.gemm_relu_plan_work_item.argtypes = [ctypes.POINTER(Plan), i32, i32] + [p32] * 7
        _lib = L
        return L


def status_string(status: int) -> str:
    return lib().gemm_relu_status_string(int(status)).decode()


def plan(M: int, N: int, K: int, num_sms: int) -> Plan:
    p = Plan()
    rc = lib().gemm_relu_plan(M, N, K, num_sms, ctypes.byref(p))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "gemm_relu_plan")
    return p


def plan_work_items(p: Plan, cta: int) -> list[dict]:
    """Work items of one CTA, as the kernel walks them."""
    out = []
    vals = [ctypes.c_int32() for _ in range(7)]
    idx = 0
    while True:
        rc = lib().gemm_relu_plan_work_item(ctypes.byref(p), cta, idx,
                                            *[ctypes.byref(v) for v in vals])
        if rc < 0:
            raise GemmReluError(GEMM_OK + 1, "gemm_relu_plan_work_item")
        if rc == 0:
            return out
        out.append(dict(zip(("tile", "tm", "tn", "kb0", "kb1", "slot", "nslots"),
                            (v.value for v in vals))))
        idx += 1


def plan_boxes(p: Plan, M: int, N: int, K: int, b_layout: str = "kn") -> Boxes:
    """The TMA boxes the kernel's copies use for one ring stage under plan ``p``."""
    out = Boxes()
    rc = lib().gemm_relu_plan_boxes(ctypes.byref(p), M, N, K, B_LAYOUTS[b_layout], ctypes.byref(out))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "gemm_relu_plan_boxes")
    return out


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on_device(device, fn, *args):
    """Call fn(*args) with `device` current (no device switch when it
    already is: the switch costs more host time than the call itself)."""
    import torch
    if device.index is None or device.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def gemm_relu(a, b, c=None, apply_relu: bool = True, stream=None):
    """C = ReLU(a @ b) (or a @ b) for CUDA fp16 tensors a (M, K), b (K, N).

    ``c`` (M, N) fp16 is written in place when given, else allocated.  Runs
    asynchronously on ``stream`` (default: torch's current stream)."""
    import torch
    if not (isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor)):
        raise TypeError("a and b must be torch tensors")
    if a.dtype != torch.float16 or b.dtype != torch.float16:
        raise TypeError("a and b must be float16")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError(f"bad shapes {tuple(a.shape)} @ {tuple(b.shape)}")
    if not (a.is_cuda and b.is_cuda) or a.device != b.device:
        raise ValueError("a and b must be CUDA tensors on the same device")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous row-major (call .contiguous())")
    M, K = a.shape
    N = b.shape[1]
    if c is None:
        c = torch.empty((M, N), dtype=torch.float16, device=a.device)
    elif (c.dtype != torch.float16 or tuple(c.shape) != (M, N) or c.device != a.device
          or not c.is_contiguous()):
        raise ValueError("c must be a contiguous float16 (M, N) tensor on a's device")
    rc = _on_device(a.device, lib().gemm_relu, a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K,
                    int(bool(apply_relu)), _stream_handle(stream, a.device))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "gemm_relu")
    return c


B_LAYOUTS = {"kn": 0, "nk": 1}  # gemm_b_layout_t


def gemm_relu_ex(a, b, c=None, apply_relu: bool = True, b_layout: str = "kn", stream=None):
    """C = ReLU(a @ b) for b_layout "kn" (b is (K, N)) or ReLU(a @ b.T) for
    "nk" (b is (N, K)); a, b and c are CUDA tensors of one element type,
    float16 or bfloat16.  ``c`` (M, N) is written in place when given."""
    import torch
    if not (isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor)):
        raise TypeError("a and b must be torch tensors")
    dtypes = {torch.float16: 0, torch.bfloat16: 1}
    if a.dtype not in dtypes or b.dtype != a.dtype:
        raise TypeError("a and b must both be float16 or both bfloat16")
    if b_layout not in B_LAYOUTS:
        raise ValueError(f"b_layout must be 'kn' or 'nk', not {b_layout!r}")
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be 2-D")
    M, K = a.shape
    N, Kb = (b.shape[1], b.shape[0]) if b_layout == "kn" else (b.shape[0], b.shape[1])
    if Kb != K:
        raise ValueError(f"bad shapes {tuple(a.shape)} and {tuple(b.shape)} ({b_layout})")
    if not (a.is_cuda and b.is_cuda) or a.device != b.device:
        raise ValueError("a and b must be CUDA tensors on the same device")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous row-major (call .contiguous())")
    if c is None:
        c = torch.empty((M, N), dtype=a.dtype, device=a.device)
    elif (c.dtype != a.dtype or tuple(c.shape) != (M, N) or c.device != a.device
          or not c.is_contiguous()):
        raise ValueError("c must be a contiguous (M, N) tensor of a's type on a's device")
    rc = _on_device(a.device, lib().gemm_relu_ex, a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K,
                    int(bool(apply_relu)), B_LAYOUTS[b_layout], dtypes[a.dtype],
                    _stream_handle(stream, a.device))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "gemm_relu_ex")
    return c


def gemm_relu_host(a, b, c=None, apply_relu: bool = True, stream=None, device=None):
    """Same operation on CPU fp16 tensors (pinned memory is fastest): the
    library copies them to the GPU, computes, and copies C back before
    returning."""
    import torch
    if a.dtype != torch.float16 or b.dtype != torch.float16 or a.is_cuda or b.is_cuda:
        raise TypeError("a and b must be CPU float16 tensors")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError(f"bad shapes {tuple(a.shape)} @ {tuple(b.shape)}")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    M, K = a.shape
    N = b.shape[1]
    if c is None:
        c = torch.empty((M, N), dtype=torch.float16, pin_memory=a.is_pinned())
    cur = torch.cuda.current_device()
    dev = torch.device("cuda", cur) if device is None else torch.device(device)
    args = (a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, int(bool(apply_relu)), _stream_handle(stream, dev))
    if dev.index is None or dev.index == cur:
        rc = lib().gemm_relu_host(*args)
    else:
        with torch.cuda.device(dev):
            rc = lib().gemm_relu_host(*args)
    if rc != GEMM_OK:
        raise GemmReluError(rc, "gemm_relu_host")
    return c


def check_device_error(stream=None, device=None):
    """Synchronize ``stream`` and raise if a kernel of this library reported
    a timed-out wait, or offsets or ids outside their range, since the last
    check (of both, the timeout first)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        rc = lib().gemm_relu_check_device_error(_stream_handle(stream, dev))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "device")


def gemm_relu_noalloc(a, b, c, apply_relu: bool = True, stream=None):
    """gemm_relu through the entry point that allocates no device memory
    (small M only; its split-K scratch is a fixed device array of the
    library).  ``c`` must be given: this call allocates nothing."""
    import torch
    if a.dtype != torch.float16 or b.dtype != torch.float16 or c.dtype != torch.float16:
        raise TypeError("a, b and c must be float16")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0] or tuple(c.shape) != (a.shape[0], b.shape[1]):
        raise ValueError(f"bad shapes {tuple(a.shape)} @ {tuple(b.shape)} -> {tuple(c.shape)}")
    if not (a.is_cuda and b.is_cuda and c.is_cuda) or a.device != b.device or c.device != a.device:
        raise ValueError("a, b and c must be CUDA tensors on one device")
    if not (a.is_contiguous() and b.is_contiguous() and c.is_contiguous()):
        raise ValueError("a, b and c must be contiguous row-major")
    M, K = a.shape
    N = b.shape[1]
    rc = _on_device(a.device, lib().gemm_relu_noalloc, a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K,
                    int(bool(apply_relu)), _stream_handle(stream, a.device))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "gemm_relu_noalloc")
    return c


def noalloc_check_device_error(stream=None, device=None):
    """Synchronize ``stream`` and raise if a gemm_relu_noalloc kernel
    reported a timed-out wait since the last check."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        rc = lib().gemm_relu_noalloc_check_device_error(_stream_handle(stream, dev))
    if rc != GEMM_OK:
        raise GemmReluError(rc, "device (noalloc)")


# ---- Ragged products.  A small call's GPU time is a few microseconds, so the
# checks below read each tensor property once and compare plain integers.

_torch = None
_CODES = {}  # {torch type: gemm_dtype_t}


def _load_torch():
    """torch, imported on first use."""
    global _torch
    if _torch is None:
        import torch
        _CODES.update({torch.float16: 0, torch.bfloat16: 1})
        _torch = torch
    return _torch


def _dtype_code(*tensors):
    """gemm_dtype_t of tensors that all have one of the library's types."""
    _load_torch()
    try:
        dtype = tensors[0].dtype
        code = _CODES.get(dtype)
        for t in tensors:
            if t.dtype is not dtype:
                code = None
    except AttributeError:
        raise TypeError("expected torch tensors") from None
    if code is None:
        raise TypeError("the matrices must all be float16 or all bfloat16")
    return code


def _layout_code(b_layout):
    try:
        return B_LAYOUTS[b_layout]
    except (KeyError, TypeError):
        raise ValueError(f"b_layout must be 'kn' or 'nk', not {b_layout!r}") from None


def _device_of(t):
    """Index of the tensor's CUDA device."""
    index = t.get_device()
    if index < 0:
        raise ValueError("the operands must be CUDA tensors")
    return index


def _rows(name, t, rows, width, device):
    """Row pitch of a (rows, width) matrix whose rows are contiguous."""
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be ({rows}, {width}), not {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on CUDA device {device}")
    if t.is_contiguous():
        return width
    row, col = t.stride()
    if col != 1 or row < width:
        raise ValueError(f"{name} must have contiguous rows that do not overlap (call .contiguous())")
    return row


def _stack(name, t, shape, device):
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape}, not {tuple(t.shape)}")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on CUDA device {device}")


def _index(name, t, count, device):
    try:
        if t.dtype is not _torch.int32:
            raise TypeError(f"{name} must be an int32 tensor")
    except AttributeError:
        raise TypeError(f"{name} must be an int32 tensor") from None
    if t.dim() != 1 or (count is not None and t.shape[0] != count):
        raise ValueError(f"{name} must hold {count} values" if count is not None else f"{name} must be 1-D")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on CUDA device {device}")


def _output(name, t, like, rows, width, device):
    """(matrix, row pitch) of an output: the caller's, or a new one."""
    if t is None:
        return _torch.empty((rows, width), dtype=like.dtype, device=like.device), width
    if getattr(t, "dtype", None) is not like.dtype:
        raise TypeError(f"{name} must be a tensor of the operands' type")
    return t, _rows(name, t, rows, width, device)


def _enqueue(fn, device, stream, *args):
    """fn(*args, stream) on that CUDA device; raises what it reports."""
    if stream is None:
        stream = _torch._C._cuda_getCurrentRawStream(device)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if device == _torch._C._cuda_getDevice():
        rc = fn(*args, stream)
    else:
        with _torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != GEMM_OK:
        raise GemmReluError(rc, fn.__name__)


def _grouped_sizes(rows, w, offsets, layout, forward):
    """(T, G, N, K, device) of a grouped product from its row matrix and weights."""
    if rows.dim() != 2 or w.dim() != 3:
        raise ValueError("the rows must be 2-D and the weights 3-D")
    device = _device_of(rows)
    G, K, N = w.shape
    if layout:
        K, N = N, K
    T, width = rows.shape
    if width != (K if forward else N):
        raise ValueError(f"bad shapes {tuple(rows.shape)} and {tuple(w.shape)}")
    if w.get_device() != device or not w.is_contiguous():
        raise ValueError(f"w must be contiguous and on CUDA device {device}")
    _index("offsets", offsets, G + 1, device)
    return T, G, N, K, device


def gemm_relu_grouped(x, w, offsets, y=None, apply_relu: bool = True, b_layout: str = "kn", stream=None):
    """y[t] = ReLU(x[t] @ w[g]) for the rows offsets[g] <= t < offsets[g + 1].

    ``x`` (T, K) and ``y`` (T, N) have contiguous rows (any row pitch that is
    a multiple of 8), ``w`` is (G, K, N), or (G, N, K) for ``b_layout="nk"``;
    float16 or bfloat16 CUDA tensors.  ``offsets`` is a CUDA int32 tensor of
    G + 1 values that the host does not read.  Rows of no group get zeros."""
    dtype, layout = _dtype_code(x, w), _layout_code(b_layout)
    T, G, N, K, device = _grouped_sizes(x, w, offsets, layout, True)
    ldx = _rows("x", x, T, K, device)
    y, ldy = _output("y", y, x, T, N, device)
    _enqueue(lib().gemm_relu_grouped, device, stream, x.data_ptr(), w.data_ptr(), y.data_ptr(), offsets.data_ptr(),
             T, G, N, K, ldx, ldy, 1 if apply_relu else 0, layout, dtype)
    return y


def gemm_relu_grouped_dx(dy, w, offsets, act=None, dx=None, b_layout: str = "kn", stream=None):
    """dx[t] = dy[t] @ w[g].T, and zero where ``act`` is given and not positive.

    ``act`` (T, K) is the activation that went into the product (its x): where
    that came out of a ReLU, dx is the gradient before that ReLU.  Shapes,
    types and ``offsets`` as ``gemm_relu_grouped``."""
    dtype, layout = _dtype_code(dy, w) if act is None else _dtype_code(dy, w, act), _layout_code(b_layout)
    T, G, N, K, device = _grouped_sizes(dy, w, offsets, layout, False)
    ld_dy = _rows("dy", dy, T, N, device)
    dx, ld_dx = _output("dx", dx, dy, T, K, device)
    ld_act = 0 if act is None else _rows("act", act, T, K, device)
    _enqueue(lib().gemm_relu_grouped_dx, device, stream, dy.data_ptr(), w.data_ptr(), dx.data_ptr(),
             offsets.data_ptr(), None if act is None else act.data_ptr(), T, G, N, K, ld_dy, ld_dx, ld_act, layout,
             dtype)
    return dx


def gemm_relu_grouped_dw(x, dy, offsets, dw=None, b_layout: str = "kn", stream=None):
    """dw[g] = x[rows of g].T @ dy[rows of g], (G, K, N), or its transpose
    (G, N, K) for ``b_layout="nk"``; zero for an empty group."""
    dtype, layout = _dtype_code(x, dy), _layout_code(b_layout)
    if x.dim() != 2 or dy.dim() != 2 or x.shape[0] != dy.shape[0]:
        raise ValueError(f"bad shapes {tuple(x.shape)} and {tuple(dy.shape)}")
    device = _device_of(x)
    _index("offsets", offsets, None, device)
    (T, K), N, G = x.shape, dy.shape[1], offsets.shape[0] - 1
    if G < 0:
        raise ValueError("offsets must hold at least one value")
    ldx, ld_dy = _rows("x", x, T, K, device), _rows("dy", dy, T, N, device)
    shape = (G, N, K) if layout else (G, K, N)
    if dw is None:
        dw = _torch.empty(shape, dtype=x.dtype, device=x.device)
    elif getattr(dw, "dtype", None) is not x.dtype:
        raise TypeError("dw must be a tensor of the operands' type")
    else:
        _stack("dw", dw, shape, device)
    _enqueue(lib().gemm_relu_grouped_dw, device, stream, x.data_ptr(), dy.data_ptr(), dw.data_ptr(),
             offsets.data_ptr(), T, G, N, K, ldx, ld_dy, layout, dtype)
    return dw


def gemm_relu_adapters(x, w, a, b, ids, scale=None, y=None, apply_relu: bool = True, b_layout: str = "kn",
                       stream=None):
    """y[t] = ReLU(x[t] @ w + scale[i] * (x[t] @ a[i].T) @ b[i]), i = ids[t].

    ``x`` (T, K), ``w`` (K, N) or (N, K) for ``b_layout="nk"``, ``a``
    (R, rank, K), ``b`` (R, rank, N): float16 or bfloat16 CUDA tensors;
    ``ids`` CUDA int32 (T,), -1 for a row without adapter; ``scale`` CUDA
    float32 (R,) or None for 1."""
    dtype, layout = _dtype_code(x, w, a, b), _layout_code(b_layout)
    if x.dim() != 2 or w.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x and w must be 2-D, a and b 3-D")
    device = _device_of(x)
    T, K = x.shape
    Kw, N = w.shape
    if layout:
        Kw, N = N, Kw
    if Kw != K:
        raise ValueError(f"bad shapes {tuple(x.shape)} and {tuple(w.shape)} ({b_layout})")
    R, rank = a.shape[0], a.shape[1]
    _stack("w", w, w.shape, device)
    _stack("a", a, (R, rank, K), device)
    _stack("b", b, (R, rank, N), device)
    _index("ids", ids, T, device)
    if scale is not None:
        if getattr(scale, "dtype", None) is not _torch.float32:
            raise TypeError("scale must be a float32 tensor")
        _stack("scale", scale, (R,), device)
    ldx = _rows("x", x, T, K, device)
    y, ldy = _output("y", y, x, T, N, device)
    _enqueue(lib().gemm_relu_adapters, device, stream, x.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(),
             ids.data_ptr(), None if scale is None else scale.data_ptr(), y.data_ptr(), T, N, K, R, rank, ldx, ldy,
             1 if apply_relu else 0, layout, dtype)
    return y


# ---- Losses over a vocabulary.  The workspace is a tensor of the caching
# allocator's, taken and given back on the call's stream: calls on two streams,
# or captured in two graphs, never share one.

_LOGIT_CODES = {}  # {torch type: gemm_logits_t}


def _head_sizes(x, w, layout):
    """(T, V, D, row pitch of x, device) of rows and a vocabulary's weights."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be 2-D")
    device = _device_of(x)
    T, D = x.shape
    V, Dw = w.shape
    if not layout:
        V, Dw = Dw, V
    if Dw != D:
        raise ValueError(f"bad shapes {tuple(x.shape)} and {tuple(w.shape)}")
    if w.get_device() != device or not w.is_contiguous():
        raise ValueError(f"w must be contiguous and on CUDA device {device}")
    return T, V, D, _rows("x", x, T, D, device), device


def _floats(name, t, T, device):
    if getattr(t, "dtype", None) is not _torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    _stack(name, t, (T,), device)


def _dloss(t, T, device):
    """Stride of the losses' gradient: 1, or 0 where all rows share one value."""
    if getattr(t, "dtype", None) is not _torch.float32:
        raise TypeError("dloss must be a float32 tensor")
    if t.get_device() != device:
        raise ValueError(f"dloss must be on CUDA device {device}")
    if t.dim() <= 1 and t.numel() == 1:
        return 0
    if t.shape != (T,) or (T > 1 and t.stride(0) not in (0, 1)):
        raise ValueError(f"dloss must hold one value, or {T} contiguous ones")
    return t.stride(0) if T > 1 else 1


def _teacher(ids, logits, T, device):
    """(k, pitch of ids, pitch of logits, type of logits)"""
    if not _LOGIT_CODES:
        _LOGIT_CODES.update({_torch.float16: 0, _torch.bfloat16: 1, _torch.float32: 2})
    if getattr(ids, "dtype", None) is not _torch.int32:
        raise TypeError("ids must be an int32 tensor")
    code = _LOGIT_CODES.get(getattr(logits, "dtype", None))
    if code is None:
        raise TypeError("logits must be a float16, bfloat16 or float32 tensor")
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D")
    k = ids.shape[1]
    return k, _rows("ids", ids, T, k, device), _rows("logits", logits, T, k, device), code


_loss_space = {}  # {(T, V, D, k, gradient): workspace bytes}


def _workspace(what, x, *sizes):
    need = _loss_space.get(sizes)
    if need is None:
        need = lib().gemm_relu_loss_workspace(*sizes)
        if need < 0:
            raise GemmReluError(-need, what)
        if len(_loss_space) >= 4096:
            _loss_space.clear()
        _loss_space[sizes] = need
    return _torch.empty(need, dtype=_torch.uint8, device=x.device)


def _on_stream(stream, device):
    """The context of a call's stream: what the call allocates belongs to it."""
    if not hasattr(stream, "cuda_stream"):
        stream = _torch.cuda.ExternalStream(stream, device=device)
    return _torch.cuda.stream(stream)


def _row_floats(name, t, T, x, device):
    """A loss's output: the caller's, or a new one."""
    if t is None:
        return _torch.empty(T, dtype=_torch.float32, device=x.device)
    _floats(name, t, T, device)
    return t


def _gradients(dx, dw, x, w, T, D, device, want_dx, want_dw):
    """(dx, its pitch, dw), the caller's or new ones; None for one that is not wanted."""
    ld = D
    if not want_dx:
        dx = None
    else:
        dx, ld = _output("dx", dx, x, T, D, device)
    if not want_dw:
        dw = None
    elif dw is None:
        dw = _torch.empty_like(w)
    else:
        if getattr(dw, "dtype", None) is not x.dtype:
            raise TypeError("dw must be a tensor of the operands' type")
        _stack("dw", dw, w.shape, device)
    return dx, ld, dw


def _pointer(t):
    return None if t is None else t.data_ptr()


def gemm_relu_xent(x, w, targets, loss=None, lse=None, b_layout: str = "kn", stream=None):
    """(loss, lse) of a cross entropy over a vocabulary, without its logits:
    lse[t] = log sum_v exp z[t, v], loss[t] = lse[t] - z[t, targets[t]], z = x @ w.

    ``x`` (T, D) has contiguous rows, ``w`` is (D, V), or (V, D) for
    ``b_layout="nk"``; float16 or bfloat16 CUDA tensors.  ``targets``: CUDA
    int32 (T,), negative for a row without one, whose loss and lse are 0.
    ``loss`` and ``lse`` are float32 (T,), written in place when given."""
    dtype, layout = _dtype_code(x, w), _layout_code(b_layout)
    T, V, D, ldx, device = _head_sizes(x, w, layout)
    if stream is not None:
        with _on_stream(stream, device):
            return gemm_relu_xent(x, w, targets, loss, lse, b_layout)
    _index("targets", targets, T, device)
    loss, lse = _row_floats("loss", loss, T, x, device), _row_floats("lse", lse, T, x, device)
    space = _workspace("gemm_relu_xent", x, T, V, D, 0, 0)
    _enqueue(lib().gemm_relu_xent, device, None, x.data_ptr(), w.data_ptr(), targets.data_ptr(), loss.data_ptr(),
             lse.data_ptr(), T, V, D, ldx, layout, dtype, space.data_ptr(), space.shape[0])
    return loss, lse


def gemm_relu_xent_grad(x, w, targets, lse, dloss, dx=None, dw=None, want_dx: bool = True, want_dw: bool = True,
                        b_layout: str = "kn", stream=None):
    """(dx, dw) of ``gemm_relu_xent``, from its ``lse`` and the gradient of its
    losses, ``dloss``: float32 (T,), or one value for all rows (a mean's).

    ``want_dx=False`` or ``want_dw=False`` leaves that one out (None)."""
    dtype, layout = _dtype_code(x, w), _layout_code(b_layout)
    T, V, D, ldx, device = _head_sizes(x, w, layout)
    if stream is not None:
        with _on_stream(stream, device):
            return gemm_relu_xent_grad(x, w, targets, lse, dloss, dx, dw, want_dx, want_dw, b_layout)
    _index("targets", targets, T, device)
    _floats("lse", lse, T, device)
    step = _dloss(dloss, T, device)
    dx, ld_dx, dw = _gradients(dx, dw, x, w, T, D, device, want_dx, want_dw)
    space = _workspace("gemm_relu_xent_grad", x, T, V, D, 0, 1)
    _enqueue(lib().gemm_relu_xent_grad, device, None, x.data_ptr(), w.data_ptr(), targets.data_ptr(), lse.data_ptr(),
             dloss.data_ptr(), step, _pointer(dx), _pointer(dw), T, V, D, ldx, ld_dx, layout, dtype, space.data_ptr(),
             space.shape[0])
    return dx, dw


def gemm_relu_distill(x, w, ids, logits, temperature: float = 1.0, loss=None, lse=None, b_layout: str = "kn",
                      stream=None):
    """(loss, lse) of a distillation from a teacher's k best words of each row,
    ``ids`` (T, k) int32, negative for none, and their ``logits`` (T, k) of a
    16- or 32-bit floating type:

    q = softmax(logits / tau), lse[t] = log sum_v exp(z[t, v] / tau),
    loss[t] = tau^2 sum_j q_j (log q_j - z[t, ids_j] / tau + lse[t]), z = x @ w.

    The rest as ``gemm_relu_xent``."""
    dtype, layout = _dtype_code(x, w), _layout_code(b_layout)
    T, V, D, ldx, device = _head_sizes(x, w, layout)
    if stream is not None:
        with _on_stream(stream, device):
            return gemm_relu_distill(x, w, ids, logits, temperature, loss, lse, b_layout)
    k, ld_ids, ld_logits, code = _teacher(ids, logits, T, device)
    loss, lse = _row_floats("loss", loss, T, x, device), _row_floats("lse", lse, T, x, device)
    space = _workspace("gemm_relu_distill", x, T, V, D, k, 0)
    _enqueue(lib().gemm_relu_distill, device, None, x.data_ptr(), w.data_ptr(), ids.data_ptr(), logits.data_ptr(),
             temperature, loss.data_ptr(), lse.data_ptr(), T, V, D, k, ldx, ld_ids, ld_logits, layout, dtype, code,
             space.data_ptr(), space.shape[0])
    return loss, lse


def gemm_relu_distill_grad(x, w, ids, logits, lse, dloss, temperature: float = 1.0, dx=None, dw=None,
                           want_dx: bool = True, want_dw: bool = True, b_layout: str = "kn", stream=None):
    """(dx, dw) of ``gemm_relu_distill``, as ``gemm_relu_xent_grad``."""
    dtype, layout = _dtype_code(x, w), _layout_code(b_layout)
    T, V, D, ldx, device = _head_sizes(x, w, layout)
    if stream is not None:
        with _on_stream(stream, device):
            return gemm_relu_distill_grad(x, w, ids, logits, lse, dloss, temperature, dx, dw, want_dx, want_dw,
                                          b_layout)
    k, ld_ids, ld_logits, code = _teacher(ids, logits, T, device)
    _floats("lse", lse, T, device)
    step = _dloss(dloss, T, device)
    dx, ld_dx, dw = _gradients(dx, dw, x, w, T, D, device, want_dx, want_dw)
    space = _workspace("gemm_relu_distill_grad", x, T, V, D, k, 1)
    _enqueue(lib().gemm_relu_distill_grad, device, None, x.data_ptr(), w.data_ptr(), ids.data_ptr(), logits.data_ptr(),
             temperature, lse.data_ptr(), dloss.data_ptr(), step, _pointer(dx), _pointer(dw), T, V, D, k, ldx, ld_ids,
             ld_logits, ld_dx, layout, dtype, code, space.data_ptr(), space.shape[0])
    return dx, dw


def shutdown():
    lib().gemm_relu_shutdown()
