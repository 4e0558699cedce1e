"""ctypes binding of libmuon_mi355x.so: argument marshalling only.

Every step of the computation runs in the HIP library.  torch is used for
device memory (tensors, the workspace) and for the current HIP stream.  If the
library is missing the calls raise; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from array import array
from typing import List, NamedTuple, Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmuon_mi355x.so")
LISTS_PATH = os.path.join(_PKG, "lib", "tensor_lists.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "muon_mi355x.h")

MUON_BF16, MUON_FP32 = 0, 1
MUON_OK, MUON_ERR_INVALID_ARG, MUON_ERR_UNSUPPORTED, MUON_ERR_WORKSPACE, MUON_ERR_HIP = range(5)
MAX_DIM = 65536
NOALLOC_MAX_WORKSPACE = 256 << 20  # MUON_NOALLOC_MAX_WORKSPACE
SIZE_MAX = ctypes.c_size_t(-1).value

QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)

EXPORTED = ("muon_workspace_bytes", "muon_workspace_bytes_ex", "muon_ns_batched",
            "muon_ns_batched_noalloc",
            "muon_step_batched",
            "muon_adamw_workspace_bytes", "muon_adamw_batched",
            "muon_status_string", "muon_last_error_detail", "muon_timing_enable",
            "muon_timing_read", "muon_timing_reset", "muon_hbm_stream",
            "muon_grad_workspace_bytes", "muon_grad_norm_batched", "muon_grad_scale_batched",
            "muon_grad_clip_batched", "muon_step_batched_scaled", "muon_adamw_batched_scaled",
            "muon_f8_workspace_bytes", "muon_f8_quantize_batched", "muon_f8_matmul_batched")
KERNELS = ("prepare", "norm", "gram", "poly", "prod", "finish", "adamw", "prod_finish", "prod_first",
           "quant8", "gram8", "poly8", "prod8", "mom_in", "mom_out",
           "grad_norm", "grad_scale", "f8_quantize", "f8_prod")


class MuonError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}: {detail}")


class NsParams(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float), ("cu_budget", ctypes.c_int32),
                ("fp8_steps", ctypes.c_int32)]


class StepParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("ns", NsParams), ("momentum_host", ctypes.c_int32)]


class AdamWParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int32)]


class GradNormParams(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("clip", ctypes.c_int32), ("max_norm", ctypes.c_float),
                ("eps", ctypes.c_float)]


_lib_handle: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the HIP library first "
            "(python -m newton_schulz_03_amd.build, or __graft_entry__.build())")
    # torch brings its own copy of the HIP runtime.  Loaded first, it serves
    # this library too (one runtime per process); loaded after this library,
    # the library's runtime reported no device (hipErrorNoDevice) on MI355X.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    i32, i64p, vpp, vp, sz = (ctypes.c_int32, ctypes.POINTER(ctypes.c_int64),
                              ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p, ctypes.c_size_t)
    lib.muon_workspace_bytes.argtypes = [i32, i64p, i64p, i32]
    lib.muon_workspace_bytes.restype = sz
    lib.muon_workspace_bytes_ex.argtypes = [i32, i64p, i64p, i32, ctypes.c_uint32]
    lib.muon_workspace_bytes_ex.restype = sz
    lib.muon_ns_batched.argtypes = [i32, i64p, i64p, vpp, vpp, i32, ctypes.POINTER(NsParams), vp,
                                    sz, vp]
    lib.muon_ns_batched.restype = i32
    lib.muon_ns_batched_noalloc.argtypes = [i32, i64p, i64p, vpp, vpp, i32,
                                            ctypes.POINTER(NsParams), vp]
    lib.muon_ns_batched_noalloc.restype = i32
    lib.muon_step_batched.argtypes = [i32, i64p, i64p, vpp, vpp, vpp, i32,
                                      ctypes.POINTER(StepParams), vp, sz, vp]
    lib.muon_step_batched.restype = i32
    lib.muon_adamw_workspace_bytes.argtypes = [i32, vp]
    lib.muon_adamw_workspace_bytes.restype = sz
    lib.muon_adamw_batched.argtypes = [i32, vp, vp, vp, vp, vp, i32,
                                       ctypes.POINTER(AdamWParams), vp, sz, vp]
    lib.muon_adamw_batched.restype = i32
    lib.muon_status_string.argtypes = [i32]
    lib.muon_status_string.restype = ctypes.c_char_p
    lib.muon_last_error_detail.argtypes = []
    lib.muon_last_error_detail.restype = ctypes.c_char_p
    lib.muon_timing_enable.argtypes = [i32]
    lib.muon_timing_enable.restype = i32
    lib.muon_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int64)]
    lib.muon_timing_read.restype = i32
    lib.muon_timing_reset.argtypes = []
    lib.muon_timing_reset.restype = i32
    lib.muon_hbm_stream.argtypes = [i32, vpp, i32, vpp, sz, i32, vp]
    lib.muon_hbm_stream.restype = i32
    # The calls below take their host arrays as bytes objects or ctypes arrays.
    lib.muon_grad_workspace_bytes.argtypes = [i32, vp]
    lib.muon_grad_workspace_bytes.restype = sz
    lib.muon_grad_norm_batched.argtypes = [i32, vp, vp, vp, ctypes.POINTER(GradNormParams), vp, vp,
                                           sz, vp]
    lib.muon_grad_norm_batched.restype = i32
    lib.muon_grad_scale_batched.argtypes = [i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.muon_grad_scale_batched.restype = i32
    lib.muon_grad_clip_batched.argtypes = [i32, vp, vp, vp, vp, vp, ctypes.POINTER(GradNormParams),
                                           vp, vp, sz, vp]
    lib.muon_grad_clip_batched.restype = i32
    lib.muon_step_batched_scaled.argtypes = [i32, i64p, i64p, vpp, vpp, vpp, i32,
                                             ctypes.POINTER(StepParams), vp, vp, sz, vp]
    lib.muon_step_batched_scaled.restype = i32
    lib.muon_adamw_batched_scaled.argtypes = [i32, vp, vp, vp, vp, vp, i32,
                                              ctypes.POINTER(AdamWParams), vp, vp, sz, vp]
    lib.muon_adamw_batched_scaled.restype = i32
    lib.muon_f8_workspace_bytes.argtypes = [i32]
    lib.muon_f8_workspace_bytes.restype = sz
    lib.muon_f8_quantize_batched.argtypes = [i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.muon_f8_quantize_batched.restype = i32
    lib.muon_f8_matmul_batched.argtypes = [i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, sz, vp]
    lib.muon_f8_matmul_batched.restype = i32
    _lib_handle = lib
    return lib


@functools.lru_cache(maxsize=None)
def _lists():
    """The extension that reads lists of tensors (csrc/tensor_lists.cpp)."""
    import importlib.machinery
    import importlib.util

    import torch  # noqa: F401  the extension links against it

    if not os.path.exists(LISTS_PATH):
        raise RuntimeError(f"{LISTS_PATH} is missing: build the library first "
                           "(python -m newton_schulz_03_amd.build, or __graft_entry__.build())")
    loader = importlib.machinery.ExtensionFileLoader("tensor_lists", LISTS_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("tensor_lists", loader))
    loader.exec_module(module)
    return module


def status_string(status: int) -> str:
    return load_library().muon_status_string(status).decode()


def last_error_detail() -> str:
    return load_library().muon_last_error_detail().decode()


def _check(status: int, where: str) -> None:
    if status != MUON_OK:
        raise MuonError(status, where, last_error_detail())


def _i64_array(vals: Sequence[int]):
    return (ctypes.c_int64 * max(1, len(vals)))(*vals)


def _ptr_array(vals: Sequence[int]):
    return (ctypes.c_void_p * max(1, len(vals)))(*vals)


def _dtype_code(dtype) -> int:
    import torch

    if dtype == torch.bfloat16:
        return MUON_BF16
    if dtype == torch.float32:
        return MUON_FP32
    raise TypeError(f"unsupported dtype {dtype}: use torch.bfloat16 or torch.float32")


MUON_WS_FP8, MUON_WS_MOMENTUM_HOST = 1, 2


def workspace_bytes(shapes: Sequence[Tuple[int, int]], dtype, fp8: bool = False,
                    momentum_host: bool = False) -> int:
    """Device workspace bytes for a batch of (rows, cols) shapes (fp8: for a bf16
    call with e4m3 steps; momentum_host: for a step with the momentum in host memory)."""
    lib = load_library()
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    rows = _i64_array([int(r) for r, _ in shapes])
    cols = _i64_array([int(c) for _, c in shapes])
    flags = (MUON_WS_FP8 if fp8 else 0) | (MUON_WS_MOMENTUM_HOST if momentum_host else 0)
    if flags:
        n = lib.muon_workspace_bytes_ex(len(shapes), rows, cols, code, flags)
    else:
        n = lib.muon_workspace_bytes(len(shapes), rows, cols, code)
    if n == SIZE_MAX:
        raise MuonError(MUON_ERR_INVALID_ARG, "muon_workspace_bytes", last_error_detail())
    return int(n)


def allocate_workspace(shapes, dtype, device, fp8: bool = False, momentum_host: bool = False):
    """A uint8 device tensor usable as the workspace of a call over `shapes`
    (fp8: with e4m3 steps; momentum_host: a step with the momentum in host memory)."""
    import torch

    n = workspace_bytes(shapes, dtype, fp8, momentum_host)
    ws = torch.empty(max(n, 1) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + max(n, 1)]


def _check_workspace(workspace, dev) -> None:
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the device of the other tensors")


def _stream_handle(device) -> int:
    import torch

    # the handle itself: a torch.cuda.Stream object around it takes 2 us to build
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check_tensors(ts, name):
    import torch

    dev = ts[0].device
    if dev.type != "cuda":
        raise ValueError(f"{name}: tensors must live on a HIP device, got {dev}")
    for t in ts:
        if t.device != dev or t.dtype != ts[0].dtype:
            raise ValueError(f"{name}: every tensor must share one device and dtype")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name}: tensors must be contiguous 2-D matrices")
    return dev


def ns_batched(xs: Sequence, steps: int = 5, coeffs=QUINTIC, eps: float = 1e-7,
               out: Optional[Sequence] = None, workspace=None, cu_budget: int = 0,
               fp8_steps: int = 0) -> List:
    """Newton-Schulz orthogonalization of a ragged batch of matrices on the GPU.

    Returns the outputs (new tensors, or `out` when given; out[i] may be xs[i]).
    Runs on the current HIP stream of the tensors' device.  cu_budget > 0 keeps
    the matrix-core launches to that many CUs (the rest stay free for other
    streams).  fp8_steps > 0 (bf16, fewer than steps): the first fp8_steps
    iterations take block-scaled e4m3 operands.
    """
    import torch

    lib = load_library()
    xs = list(xs)
    if not xs:
        return []
    dev = _check_tensors(xs, "xs")
    if out is None:
        out = [torch.empty_like(x) for x in xs]
    out = list(out)
    if len(out) != len(xs):
        raise ValueError("out must have one tensor per input")
    _check_tensors(out + xs, "out")
    shapes = [tuple(x.shape) for x in xs]
    if any(tuple(o.shape) != s for o, s in zip(out, shapes)):
        raise ValueError("out shapes must match the inputs")
    code = _dtype_code(xs[0].dtype)
    if workspace is None:
        workspace = allocate_workspace(shapes, xs[0].dtype, dev, fp8=fp8_steps > 0)
    _check_workspace(workspace, dev)
    a, b, c = (float(v) for v in coeffs)
    p = NsParams(int(steps), a, b, c, float(eps), int(cu_budget), int(fp8_steps))
    with torch.cuda.device(dev):
        st = lib.muon_ns_batched(len(xs), _i64_array([s[0] for s in shapes]),
                                 _i64_array([s[1] for s in shapes]),
                                 _ptr_array([x.data_ptr() for x in xs]),
                                 _ptr_array([o.data_ptr() for o in out]), code, ctypes.byref(p),
                                 ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                 ctypes.c_void_p(_stream_handle(dev)))
    _check(st, "muon_ns_batched")
    return out


def ns_batched_noalloc(xs: Sequence, out: Sequence, steps: int = 5, coeffs=QUINTIC,
                       eps: float = 1e-7, cu_budget: int = 0, fp8_steps: int = 0) -> List:
    """ns_batched through the allocation-free entry point: no workspace (the
    library's own array of NOALLOC_MAX_WORKSPACE bytes per GPU serves), and the
    caller passes the outputs.  Calls that overlap on one GPU race."""
    import torch

    lib = load_library()
    xs, out = list(xs), list(out)
    if not xs:
        return out
    if len(out) != len(xs):
        raise ValueError("out must have one tensor per input")
    dev = _check_tensors(out + xs, "xs/out")
    shapes = [tuple(x.shape) for x in xs]
    if any(tuple(o.shape) != s for o, s in zip(out, shapes)):
        raise ValueError("out shapes must match the inputs")
    a, b, c = (float(v) for v in coeffs)
    p = NsParams(int(steps), a, b, c, float(eps), int(cu_budget), int(fp8_steps))
    with torch.cuda.device(dev):
        st = lib.muon_ns_batched_noalloc(len(xs), _i64_array([s[0] for s in shapes]),
                                         _i64_array([s[1] for s in shapes]),
                                         _ptr_array([x.data_ptr() for x in xs]),
                                         _ptr_array([o.data_ptr() for o in out]),
                                         _dtype_code(xs[0].dtype), ctypes.byref(p),
                                         ctypes.c_void_p(_stream_handle(dev)))
    _check(st, "muon_ns_batched_noalloc")
    return out


def step_batched(ws: Sequence, gs: Sequence, ms: Sequence, lr: float = 0.02, beta: float = 0.95,
                 nesterov: bool = False, steps: int = 5, coeffs=QUINTIC, eps: float = 1e-7,
                 workspace=None, momentum_host: bool = False, cu_budget: int = 0,
                 fp8_steps: int = 0, grad_scale=None) -> None:
    """One Muon step over a ragged batch, in place on ws (weights) and ms (momentum).

    grad_scale: a one-element float32 tensor on the weights' device (the clip
    factor of grad_norm_batched); every gradient is multiplied by it in fp32 as
    it is read.

    momentum_host: the momenta are pinned host tensors (pin_memory), updated in
    place: the step copies them to the device and back in chunks, overlapped
    with the Newton-Schulz work.
    """
    import torch

    lib = load_library()
    ws, gs, ms = list(ws), list(gs), list(ms)
    if not (len(ws) == len(gs) == len(ms)):
        raise ValueError("ws, gs and ms must have the same length")
    if not ws:
        return
    if momentum_host:
        dev = _check_tensors(ws + gs, "ws/gs")
        for m in ms:
            if m.device.type != "cpu" or not m.is_pinned() or m.dtype != ws[0].dtype or \
                    m.dim() != 2 or not m.is_contiguous():
                raise ValueError("ms: with momentum_host, every momentum must be a pinned, "
                                 "contiguous 2-D host tensor of the weights' dtype")
    else:
        dev = _check_tensors(ws + gs + ms, "ws/gs/ms")
    shapes = [tuple(w.shape) for w in ws]
    if any(tuple(g.shape) != s or tuple(m.shape) != s for g, m, s in zip(gs, ms, shapes)):
        raise ValueError("w, g and m of one matrix must share a shape")
    code = _dtype_code(ws[0].dtype)
    if workspace is None:
        workspace = allocate_workspace(shapes, ws[0].dtype, dev, fp8=fp8_steps > 0,
                                       momentum_host=momentum_host)
    _check_workspace(workspace, dev)
    a, b, c = (float(v) for v in coeffs)
    p = StepParams(float(lr), float(beta), 1 if nesterov else 0,
                   NsParams(int(steps), a, b, c, float(eps), int(cu_budget), int(fp8_steps)),
                   1 if momentum_host else 0)
    fn, scale = lib.muon_step_batched, ()
    if grad_scale is not None:
        fn, scale = lib.muon_step_batched_scaled, (_scale_pointer(grad_scale, dev),)
    with torch.cuda.device(dev):
        st = fn(len(ws), _i64_array([s[0] for s in shapes]), _i64_array([s[1] for s in shapes]),
                _ptr_array([w.data_ptr() for w in ws]), _ptr_array([g.data_ptr() for g in gs]),
                _ptr_array([m.data_ptr() for m in ms]), code, ctypes.byref(p), *scale,
                ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                ctypes.c_void_p(_stream_handle(dev)))
    _check(st, fn.__name__)


def _scale_pointer(t, dev):
    import torch

    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != torch.float32 or \
            t.numel() != 1:
        raise ValueError("the factor must be a float32 tensor of one element on the device of the "
                         "other tensors")
    return t.data_ptr()


def adamw_workspace_bytes(numels: Sequence[int]) -> int:
    lib = load_library()
    numels = list(numels)
    n = lib.muon_adamw_workspace_bytes(len(numels), _i64_array(numels) if numels else None)
    if n == SIZE_MAX:
        raise MuonError(MUON_ERR_INVALID_ARG, "muon_adamw_workspace_bytes", last_error_detail())
    return n


def adamw_batched(params: Sequence, grads: Sequence, exp_avgs: Sequence, exp_avg_sqs: Sequence,
                  lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                  weight_decay: float = 1e-2, step: int = 1, workspace=None,
                  grad_scale=None) -> None:
    """One AdamW step over a ragged batch of tensors, in place on params and the moments.

    grad_scale: a one-element float32 tensor on the parameters' device (the clip
    factor of grad_norm_batched); every gradient is multiplied by it in fp32 as
    it is read.

    params/grads: bf16 or fp32 (one dtype for all), contiguous; exp_avgs and
    exp_avg_sqs: fp32, same shapes.  `step` is the number of the step being
    taken (1 for the first).  Runs on the current HIP stream.
    """
    import torch

    lib = load_library()
    ps, gs, ms, vs = list(params), list(grads), list(exp_avgs), list(exp_avg_sqs)
    if not ps:
        return
    if not (len(ps) == len(gs) == len(ms) == len(vs)):
        raise ValueError("params, grads and moments must have one tensor each per entry")
    dev = ps[0].device
    if dev.type != "cuda":
        raise ValueError(f"params must live on a HIP device, got {dev}")
    lists = _lists()
    ptrs = {}
    for name, group, want in (("p", ps, ps[0].dtype), ("m", ms, torch.float32),
                              ("v", vs, torch.float32), ("g", gs, ps[0].dtype)):
        index, flags, _, numels, where, _, _ = lists.scan(group, name != "g")
        if index != dev.index or group[0].dtype != want or flags & _FLAT != _FLAT:
            raise ValueError("tensors must be contiguous on one device; p and g share a "
                             "dtype, the moments are float32")
        ptrs[name] = where
    if not all(lists.same_shapes(ps, group) for group in (gs, ms, vs)):
        raise ValueError("p, g, m and v of one entry must have the same shape")
    code = _dtype_code(ps[0].dtype)
    if workspace is None:
        workspace = _byte_workspace(_adamw_table_bytes(len(ps)), dev)
    _check_workspace(workspace, dev)
    b1, b2 = (float(b) for b in betas)
    prm = AdamWParams(float(lr), b1, b2, float(eps), float(weight_decay), int(step))
    fn, scale = lib.muon_adamw_batched, ()
    if grad_scale is not None:
        fn, scale = lib.muon_adamw_batched_scaled, (_scale_pointer(grad_scale, dev),)
    _call(fn, dev, workspace, len(ps), numels, ptrs["p"], ptrs["g"], ptrs["m"], ptrs["v"],
          code, ctypes.byref(prm), *scale)


_FLAT = 7  # of the lists' flags: one device, contiguous, one dtype
_SAME_DEVICE, _CONTIGUOUS, _SAME_DTYPE, _MATRICES = 1, 2, 4, 8


@functools.lru_cache(maxsize=None)
def _adamw_table_bytes(batch: int) -> int:
    # the workspace is the descriptor table, whatever the sizes
    return adamw_workspace_bytes([0] * batch)


def _call(fn, dev, workspace, *args) -> None:
    """Runs an entry point whose last arguments are the workspace, its size and
    the stream, on `dev` and its current stream."""
    import torch

    args += (workspace.data_ptr(), workspace.numel(), _stream_handle(dev))
    if torch.cuda.current_device() == dev.index:
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != MUON_OK:
        _check(st, fn.__name__)


# ---------------------------------------------------------------------------
# Gradient norm and clip
# ---------------------------------------------------------------------------

_NORM_KINDS = {2: 0, math.inf: 1}  # MUON_NORM_L2, MUON_NORM_MAX


def _byte_workspace(nbytes: int, dev):
    import torch

    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if ws.data_ptr() % 256 == 0:  # as torch's allocator gives it
        return ws
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes]


def _workspace(given, nbytes, dev):
    import torch

    if given is None:
        return _byte_workspace(nbytes, dev)
    if given.device != dev or given.dtype != torch.uint8 or not given.is_contiguous():
        raise ValueError("workspace: a contiguous uint8 tensor on the device of the other tensors")
    return given


def _flat_tensors(ts, name, written):
    """(device, dtype codes, element counts, pointers) of contiguous bf16 / fp32
    tensors, the last three as the bytes of C arrays.  The lists that a call writes
    are asked for before those it only reads."""
    import torch

    index, flags, codes, numels, ptrs, _, _ = _lists().scan(ts, written)
    dev = ts[0].device
    if index < 0:
        raise ValueError(f"{name}: tensors must live on a HIP device, got {dev}")
    if flags & (_SAME_DEVICE | _CONTIGUOUS) != _SAME_DEVICE | _CONTIGUOUS:
        raise ValueError(f"{name}: tensors must be contiguous on one device")
    if b"\xff\xff\xff\xff" in codes:
        bad = next(t.dtype for t in ts if t.dtype not in (torch.bfloat16, torch.float32))
        raise TypeError(f"{name}: unsupported dtype {bad}: use torch.bfloat16 or torch.float32")
    return dev, codes, numels, ptrs


def grad_workspace_bytes(numels: Sequence[int]) -> int:
    """Device workspace bytes of a gradient norm, scale or clip call."""
    numels = list(numels)
    n = load_library().muon_grad_workspace_bytes(len(numels), _i64_array(numels))
    if n == SIZE_MAX:
        raise MuonError(MUON_ERR_INVALID_ARG, "muon_grad_workspace_bytes", last_error_detail())
    return int(n)


@functools.lru_cache(maxsize=None)
def _grad_table_bytes(batch: int) -> int:
    # the workspace depends on the number of tensors only
    return grad_workspace_bytes([0] * batch)


def _norm_params(max_norm, norm_type, eps) -> GradNormParams:
    kind = _NORM_KINDS.get(norm_type)
    if kind is None:
        raise ValueError(f"norm_type {norm_type!r}: use 2 or math.inf")
    return GradNormParams(kind, 0 if max_norm is None else 1,
                          0.0 if max_norm is None else float(max_norm), float(eps))


def _norm_room(workspace, result, batch, dev):
    """(workspace, result) of a norm: those given, or new ones."""
    import torch

    nbytes = _grad_table_bytes(batch)
    if workspace is None and result is None:
        workspace, result = _lists().room_norm(nbytes, dev.index)
        if workspace.data_ptr() % 256 == 0:  # as torch's allocator gives it
            return workspace, result
        workspace = None
    if result is None:
        result = torch.empty(2, dtype=torch.float32, device=dev)
    elif result.device != dev or result.dtype != torch.float32 or tuple(result.shape) != (2,) or \
            not result.is_contiguous():
        raise ValueError("result: a contiguous float32 tensor of 2 elements on the gradients' device")
    return _workspace(workspace, nbytes, dev), result


def grad_norm_batched(grads: Sequence, max_norm: Optional[float] = None, norm_type: float = 2.0,
                      eps: float = 1e-6, result=None, workspace=None):
    """Global norm over a ragged batch of gradients, and the clip factor.

    Returns a float32 tensor of 2 on the gradients' device (`result`, if given):
    the norm (norm_type 2, or math.inf: the largest magnitude), and the factor
    min(1, max_norm / (norm + eps)), 1 without max_norm.  grads: contiguous
    bf16 and fp32 tensors, mixed as they come, on one device.  Runs on the
    current HIP stream; nothing waits for the GPU.
    """
    grads = list(grads)
    if not grads:
        raise ValueError("grads: at least one tensor (its device holds the result)")
    p = _norm_params(max_norm, norm_type, eps)
    dev, codes, numels, ptrs = _flat_tensors(grads, "grads", False)
    workspace, result = _norm_room(workspace, result, len(grads), dev)
    _call(load_library().muon_grad_norm_batched, dev, workspace, len(grads), numels,
          ptrs, codes, ctypes.byref(p), result.data_ptr())
    return result


def _grads_and_outputs(grads, out):
    """(device, dtype codes, element counts, pointers) of the gradients, then the
    outputs, their dtype codes and pointers."""
    if out is None:
        dev, codes, numels, ptrs = _flat_tensors(grads, "grads", True)
        return dev, codes, numels, ptrs, grads, codes, ptrs
    out = list(out)
    if len(out) != len(grads):
        raise ValueError("out must have one tensor per gradient")
    odev, ocodes, onumels, optrs = _flat_tensors(out, "out", True)
    dev, codes, numels, ptrs = _flat_tensors(grads, "grads", False)
    if odev != dev:
        raise ValueError("out must live on the gradients' device")
    if onumels != numels:
        raise ValueError("out must have the gradients' sizes")
    return dev, codes, numels, ptrs, out, ocodes, optrs


def grad_scale_batched(grads: Sequence, scale, out: Optional[Sequence] = None,
                       workspace=None) -> List:
    """out[i] = scale * grads[i]; scale: a one-element float32 tensor on their
    device.  In place without `out`; out[i] may have the other dtype.  Returns
    the outputs."""
    grads = list(grads)
    if not grads:
        return []
    dev, codes, numels, ptrs, out, ocodes, optrs = _grads_and_outputs(grads, out)
    factor = _scale_pointer(scale, dev)
    workspace = _workspace(workspace, _grad_table_bytes(len(grads)), dev)
    _call(load_library().muon_grad_scale_batched, dev, workspace, len(grads), numels,
          ptrs, codes, optrs, ocodes, factor)
    return out


def grad_clip_batched(grads: Sequence, max_norm: float, norm_type: float = 2.0, eps: float = 1e-6,
                      out: Optional[Sequence] = None, result=None, workspace=None):
    """Clips a ragged batch of gradients by their global norm: in place, or into
    `out` (whose tensors may have the other dtype: fp32 sums into bf16
    gradients).  Returns the float32 tensor (norm, factor) of grad_norm_batched.
    Nothing waits for the GPU."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads: at least one tensor (its device holds the result)")
    if max_norm is None:
        raise ValueError("max_norm is needed")
    p = _norm_params(max_norm, norm_type, eps)
    dev, codes, numels, ptrs, _, ocodes, optrs = _grads_and_outputs(grads, out)
    workspace, result = _norm_room(workspace, result, len(grads), dev)
    _call(load_library().muon_grad_clip_batched, dev, workspace, len(grads), numels,
          ptrs, codes, optrs, ocodes, ctypes.byref(p),
          result.data_ptr())
    return result


# ---------------------------------------------------------------------------
# Block-scaled e4m3 operands and their product
# ---------------------------------------------------------------------------

F8_BLOCK = 128
F8_MAX_DIM = 1 << 20


class F8Operand(NamedTuple):
    """An operand of f8_matmul_batched: R rows, contracted over Kp columns (a
    multiple of F8_BLOCK).  q: float8_e4m3fn, R x Kp; scales: uint8,
    Kp/128 x Rp (Rp: R up to a multiple of 16), byte [kb][r] = e + 127 for the
    power of two 2^e of columns 128 kb .. 128 kb + 127 of row r.  Columns and
    scale entries past the matrix are zero."""

    q: object
    scales: object


def f8_empty(rows: int, cols: int, device) -> F8Operand:
    """Room for the operand of a rows x cols matrix (contracted over cols)."""
    import torch

    kp, rp = -(-cols // F8_BLOCK) * F8_BLOCK, -(-rows // 16) * 16
    return F8Operand(torch.empty((rows, kp), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
                     torch.empty((kp // F8_BLOCK, rp), dtype=torch.uint8, device=device))


def _f8_pointers(ops, name, dev, written=False):
    """(rows, padded contracted sides, value pointers, scale pointers) of operands,
    as the bytes of C arrays."""
    index, bad, kind, rows, kps, qs, ss = _lists().scan_f8(ops, F8_BLOCK, written)
    if bad >= 0 and kind == 1:
        raise TypeError(f"{name}: an operand is a float8_e4m3fn tensor and a uint8 tensor")
    if index != dev.index or (bad >= 0 and kind == 2):
        raise ValueError(f"{name}: operands must be contiguous 2-D tensors on one HIP device")
    if bad >= 0:
        q, s = ops[bad]
        raise ValueError(f"{name}: operand {bad} has values {tuple(q.shape)} and scales "
                         f"{tuple(s.shape)}: want (R, Kp) with Kp a multiple of {F8_BLOCK}, and "
                         "(Kp / 128, R up to a multiple of 16)")
    return rows, kps, qs, ss


def _i64_bytes(vals) -> bytes:
    return array("q", vals).tobytes()


def f8_workspace_bytes(batch: int) -> int:
    """Device workspace bytes of an f8_quantize_batched or f8_matmul_batched call."""
    n = load_library().muon_f8_workspace_bytes(int(batch))
    if n == SIZE_MAX:
        raise MuonError(MUON_ERR_INVALID_ARG, "muon_f8_workspace_bytes", last_error_detail())
    return int(n)


def f8_quantize_batched(xs: Sequence, block_rows: int = 1, normal: bool = True,
                        transpose: bool = False, out: Optional[Sequence] = None,
                        out_t: Optional[Sequence] = None, workspace=None):
    """Block-scaled e4m3 operands of a ragged batch of matrices.

    xs: contiguous 2-D bf16 or fp32 tensors (one dtype).  normal: the operands
    of the matrices (contracted over their columns); transpose: those of their
    transposes (contracted over their rows); both come from one read.
    block_rows: 1 for a scale per 1 x 128 block along the contracted side
    (activations, gradients), 128 for one per 128 x 128 block (weights).
    Returns the operands, the transposes' operands, or a pair of both lists, in
    `out` and `out_t` where given; new ones of one list share an allocation, which
    lives as long as any of them (torch.save of one writes all: save a clone).
    """
    xs = list(xs)
    if not normal and not transpose:
        raise ValueError("one of normal and transpose must be set")
    if (out is not None and not normal) or (out_t is not None and not transpose):
        raise ValueError("out goes with normal, out_t with transpose")
    if not xs:
        return ([], []) if normal and transpose else []

    def written(given, name):
        if given is None:
            return None
        ops = list(given)
        if len(ops) != len(xs):
            raise ValueError(f"{name} must have one operand per matrix")
        return ops, *_f8_pointers(ops, name, xs[0].device, True)

    out, out_t = written(out, "out"), written(out_t, "out_t")  # before what is read
    dev, rows, cols, ptrs = _matrices(xs, "xs")
    code = _dtype_code(xs[0].dtype)

    def side(wanted, given, name, r, k):
        if not wanted:
            return None, None, None
        if given is None:
            ops = _lists().room_f8(r, k, F8_BLOCK, dev.index, F8Operand)
            return ops, *_f8_pointers(ops, name, dev)[2:]
        ops, got_r, got_k, q, s = given
        if got_r != r or got_k != _i64_bytes(-(-x // F8_BLOCK) * F8_BLOCK for x in array("q", k)):
            raise ValueError(f"{name}: an operand's values must be (rows, contracted side up to a "
                             f"multiple of {F8_BLOCK})")
        return ops, q, s

    ops, q, s = side(normal, out, "out", rows, cols)
    ops_t, qt, st_ = side(transpose, out_t, "out_t", cols, rows)
    workspace = _workspace(workspace, f8_workspace_bytes(len(xs)), dev)
    _call(load_library().muon_f8_quantize_batched, dev, workspace, len(xs), rows, cols, ptrs, code,
          int(block_rows), q, s, qt, st_)
    return (ops, ops_t) if normal and transpose else ops if normal else ops_t


def f8_matmul_batched(a: Sequence, b: Sequence, out: Optional[Sequence] = None, out_dtype=None,
                      accumulate: bool = False, workspace=None) -> List:
    """out[i] = A_i B_i^T over block-scaled e4m3 operands, ragged over the batch.

    a, b: sequences of F8Operand (or (values, scales) pairs) with equal
    contracted sides.  out: contiguous bf16 or fp32 tensors of (A's rows, B's
    rows); without it new ones of out_dtype (bfloat16), which share an allocation
    as those of f8_quantize_batched do.
    accumulate: the products are added to `out`.  Sums are fp32, rounded once;
    for bfloat16 outputs 8 consecutive products at a time first lose what is
    below 2^-13 of the largest of them.  For float32 outputs operand values of
    2^128 and more are infinite.  For Y = X W^T: dX = dY W takes the operands of
    dY and W^T, and dW = dY^T X those of dY^T and X^T (f8_quantize_batched's
    transpose).  Returns the outputs.
    """
    import torch

    a, b = list(a), list(b)
    if len(a) != len(b):
        raise ValueError("a and b must have the same length")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if not a:
        return [] if out is None else list(out)
    dev = a[0][0].device
    if dev.type != "cuda":
        raise ValueError(f"a: operands must live on a HIP device, got {dev}")
    if out is not None:
        out = list(out)
        if len(out) != len(a):
            raise ValueError("out must have one tensor per product")
        if out_dtype is not None and any(o.dtype != out_dtype for o in out):
            raise ValueError("out has another dtype than out_dtype")
        odev, rows, cols, ptrs = _matrices(out, "out", True)  # before what is read
        if odev != dev:
            raise ValueError("out must live on the operands' device")
    m, ka, aq, asc = _f8_pointers(a, "a", dev)
    n, kb, bq, bsc = _f8_pointers(b, "b", dev)
    if ka != kb:
        i, x, y = next((i, x, y) for i, (x, y) in enumerate(zip(array("q", ka), array("q", kb)))
                       if x != y)
        raise ValueError(f"product {i}: contracted sides {x} and {y} differ")
    if out is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        out = _lists().room(m, n, _dtype_code(dt), dev.index)
        _, rows, cols, ptrs = _matrices(out, "out")
    if rows != m or cols != n:
        raise ValueError("out must have the shape (rows of a, rows of b)")
    code = _dtype_code(out[0].dtype)
    workspace = _workspace(workspace, f8_workspace_bytes(len(a)), dev)
    _call(load_library().muon_f8_matmul_batched, dev, workspace, len(a), m, n, ka, aq, asc, bq, bsc,
          ptrs, code, 1 if accumulate else 0)
    return out


def _matrices(ts, name, written=False):
    """(device, rows, columns, pointers) of contiguous 2-D tensors of one dtype, the
    last three as the bytes of C arrays."""
    index, flags, _, _, ptrs, rows, cols = _lists().scan(ts, written)
    if index < 0 or flags & (_FLAT | _MATRICES) != _FLAT | _MATRICES:
        _check_tensors(ts, name)  # says what is wrong
    return ts[0].device, rows, cols, ptrs


def hbm_stream(ins: Sequence, outs: Sequence, nontemporal: bool = False) -> None:
    """Plain HBM stream (measurement aid): outs[k] <- ins[k % len(ins)] (two inputs
    into one output: their bitwise XOR), on the current stream.  1 or 2 inputs
    and outputs, uint8 device tensors of one size, a multiple of 16384 bytes."""
    import torch

    ins, outs = list(ins), list(outs)
    n = ins[0].numel() * ins[0].element_size()
    for t in ins + outs:
        if t.device.type != "cuda" or not t.is_contiguous() or t.numel() * t.element_size() != n:
            raise ValueError("hbm_stream: contiguous device tensors of one size")
    dev = ins[0].device
    with torch.cuda.device(dev):
        st = load_library().muon_hbm_stream(len(ins), _ptr_array([t.data_ptr() for t in ins]),
                                            len(outs), _ptr_array([t.data_ptr() for t in outs]),
                                            n, 1 if nontemporal else 0,
                                            ctypes.c_void_p(_stream_handle(dev)))
    _check(st, "muon_hbm_stream")


def timing_enable(on: bool = True) -> None:
    """Record HIP events around every kernel launch (process-wide) while on."""
    _check(load_library().muon_timing_enable(1 if on else 0), "muon_timing_enable")


def timing_reset() -> None:
    _check(load_library().muon_timing_reset(), "muon_timing_reset")


def timing_read() -> dict:
    """{kernel name: (total milliseconds, launches)} since the last reset."""
    lib = load_library()
    out = {}
    for k, name in enumerate(KERNELS):
        ms, n = ctypes.c_double(), ctypes.c_int64()
        _check(lib.muon_timing_read(k, ctypes.byref(ms), ctypes.byref(n)), "muon_timing_read")
        out[name] = (ms.value, n.value)
    return out
