"""AdaComp for AMD Instinct MI355X: Python binding of ``libadacomp.so``.

A thin layer over the C ABI declared in ``include/adacomp.h`` (ctypes; for the
training-step operators the extension module ``_binding.so``): it marshals
torch tensors (device memory) and the current HIP stream into plain pointers
and sizes.  Every step of compression and decoding runs in the HIP
kernels of the library; nothing here computes.  If the library is not built,
every call raises ``HipLibraryMissing``; there is no fallback.

Method: "AdaComp (Adaptive Residual Gradient Compression)", AIMech curated
page, definition paragraph and Mechanism claim on local-bin soft threshold
and mean-g_max quantization (Algorithm 2).
"""
from __future__ import annotations

import ctypes
import pathlib
from typing import Iterable, List, Optional, Sequence

_HERE = pathlib.Path(__file__).resolve().parent
LIB_PATH = _HERE / "libadacomp.so"

OK = 0
NUM_STAGES = 11
STAGES = ("tile_pass", "chunk_scan", "finalize", "encode",
          "decode_count", "decode_base", "decode_apply", "compress_call", "decode_call",
          "decode_sgd_call", "decode_adam_call")
MAX_MESSAGES = 256
MAX_BIN_LEN = 32768
SEG_LS = 1   # segment flag: hard local selection (see include/adacomp.h)
PLAN_SEPARATE_FINISH = 1   # plan flag: finish with three kernels whatever the table
PLAN_SINGLE_LAUNCH = 2     # plan flag: a small table in one launch (slower; for comparison)
PLAN_DECODE_RECORDS = 4    # plan flag: plain sums always take the entry-record decode
SMALL_TABLE_MAX_SPAN = 1 << 21     # tables up to this span and this many segments
SMALL_TABLE_MAX_SEGMENTS = 256     # finish in one launch after the tile pass
NOALLOC_SCRATCH_BYTES = 128 << 20  # largest compress workspace compress_noalloc takes
CHUNK_FINISH_MAX_TILES = 1 << 20   # larger tables of <= 256 segments and this many tiles: two


class HipLibraryMissing(RuntimeError):
    pass


class AdaCompError(RuntimeError):
    def __init__(self, where: str, status: int):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} ({status})")


class _Segment(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_uint64), ("numel", ctypes.c_uint64),
                ("bin_len", ctypes.c_uint32), ("flags", ctypes.c_uint32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("nseg", ctypes.c_uint32), ("plan_hash", ctypes.c_uint32),
                ("total_numel", ctypes.c_uint64), ("span", ctypes.c_uint64),
                ("total_bins", ctypes.c_uint64), ("ntiles", ctypes.c_uint64),
                ("header_bytes", ctypes.c_uint64), ("message_capacity", ctypes.c_uint64),
                ("compress_workspace_bytes", ctypes.c_uint64),
                ("decode_workspace_bytes_per_message", ctypes.c_uint64),
                ("decode_workspace_bytes_fixed", ctypes.c_uint64),
                ("compress_launches", ctypes.c_uint64)]

    def as_dict(self):
        return {name: int(getattr(self, name)) for name, _ in self._fields_}

    def decode_workspace_bytes(self, K: int) -> int:
        return int(self.decode_workspace_bytes_fixed) + K * int(self.decode_workspace_bytes_per_message)


class Sgd(ctypes.Structure):
    """One step of SGD with momentum: g = scale*sum (+ weight_decay*w),
    m = momentum*m + g, w = w - lr*m."""
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_float)]


class Adam(ctypes.Structure):
    """One Adam step (bias-corrected moments); see include/adacomp.h."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale", ctypes.c_float), ("step", ctypes.c_uint32)]


class _Tensor(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_uint64), ("numel", ctypes.c_uint64),
                ("weight_decay", ctypes.c_float), ("lr_scale", ctypes.c_float)]


class OptimizerInfo(ctypes.Structure):
    _fields_ = [("ntensors", ctypes.c_uint64), ("total_numel", ctypes.c_uint64),
                ("span", ctypes.c_uint64), ("nblocks", ctypes.c_uint64),
                ("norm_workspace_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


class AdamW(ctypes.Structure):
    """One AdamW step; see include/adacomp.h."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("step", ctypes.c_uint32)]


class _ScanShape(ctypes.Structure):
    _fields_ = [("length", ctypes.c_uint64), ("batch", ctypes.c_uint32), ("channels", ctypes.c_uint32),
                ("type", ctypes.c_int), ("sigmoid", ctypes.c_int)]


class _View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_uint64),
                ("time_stride", ctypes.c_uint64)]


# Every exported symbol, with its C signature (argtypes, restype).
_P = ctypes.c_void_p
_U32, _U64, _INT, _FLT = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int, ctypes.c_float
_SHAPE, _VIEW = ctypes.POINTER(_ScanShape), ctypes.POINTER(_View)
SIGNATURES = {
    "adacomp_plan_query": ([ctypes.POINTER(_Segment), _U32, ctypes.POINTER(PlanInfo)], _INT),
    "adacomp_plan_create": ([ctypes.POINTER(_Segment), _U32, ctypes.POINTER(_P)], _INT),
    "adacomp_plan_create_ex": ([ctypes.POINTER(_Segment), _U32, _U32, ctypes.POINTER(_P)], _INT),
    "adacomp_plan_destroy": ([_P], _INT),
    "adacomp_plan_get_info": ([_P, ctypes.POINTER(PlanInfo)], _INT),
    "adacomp_compress": ([_P, _P, _P, _U64, _P, _U64, _P, _U64, _P, _P], _INT),
    "adacomp_compress_noalloc": ([_P, _P, _P, _U64, _P, _U64, _P, _P], _INT),
    "adacomp_decode_accumulate": ([_P, ctypes.POINTER(_P), _U32, _P, _U64, _INT, _P, _U64, _P], _INT),
    "adacomp_compress_timed": ([_P, _P, _P, _U64, _P, _U64, _P, _U64, _P, _P, _P], _INT),
    "adacomp_decode_accumulate_timed": ([_P, ctypes.POINTER(_P), _U32, _P, _U64, _INT, _P, _U64,
                                         _P, _P], _INT),
    "adacomp_decode_sgd": ([_P, ctypes.POINTER(_P), _U32, _P, _P, _U64, ctypes.POINTER(Sgd), _P, _U64,
                            _P], _INT),
    "adacomp_decode_sgd_timed": ([_P, ctypes.POINTER(_P), _U32, _P, _P, _U64, ctypes.POINTER(Sgd), _P,
                                  _U64, _P, _P], _INT),
    "adacomp_decode_sgd_workspace_bytes": ([_P, _U32, ctypes.POINTER(_U64)], _INT),
    "adacomp_decode_adam": ([_P, ctypes.POINTER(_P), _U32, _P, _P, _P, _U64, ctypes.POINTER(Adam), _P,
                             _U64, _P], _INT),
    "adacomp_decode_adam_timed": ([_P, ctypes.POINTER(_P), _U32, _P, _P, _P, _U64, ctypes.POINTER(Adam),
                                   _P, _U64, _P, _P], _INT),
    "adacomp_timer_create": ([ctypes.POINTER(_P)], _INT),
    "adacomp_timer_destroy": ([_P], _INT),
    "adacomp_timer_read": ([_P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_U64), _U32], _INT),
    "adacomp_timer_reset": ([_P], _INT),
    "adacomp_optimizer_query": ([ctypes.POINTER(_Tensor), _U32, ctypes.POINTER(OptimizerInfo)], _INT),
    "adacomp_optimizer_create": ([ctypes.POINTER(_Tensor), _U32, ctypes.POINTER(_P)], _INT),
    "adacomp_optimizer_destroy": ([_P], _INT),
    "adacomp_optimizer_get_info": ([_P, ctypes.POINTER(OptimizerInfo)], _INT),
    "adacomp_grad_norm": ([_P, _P, _INT, _U64, _FLT, _FLT, _P, _P, _U64, _P], _INT),
    "adacomp_adamw_step": ([_P, _P, _P, _INT, _P, _P, _P, _U64, ctypes.POINTER(AdamW), _P, _P], _INT),
    "adacomp_adamw_packed_step": ([_P, _P, _P, _INT, _P, _P, _P, _P, _U64, ctypes.POINTER(AdamW), _U32,
                                   _P, _P], _INT),
    "adacomp_layer_norm": ([_P, _U64, _P, _P, _P, _U64, _P, _P, _U64, _U32, _INT, _FLT, _P], _INT),
    "adacomp_layer_norm_backward": ([_P, _U64, _P, _U64, _P, _P, _P, _P, _U64, _P, _P, _U64, _U32, _INT,
                                     _P, _U64, _P], _INT),
    "adacomp_layer_norm_workspace_bytes": ([_U64, _U32, ctypes.POINTER(_U64)], _INT),
    "adacomp_gated_scan": ([_SHAPE, _VIEW, _VIEW, _VIEW, _P, _P, _P, _P, _U64, _P], _INT),
    "adacomp_gated_scan_backward": ([_SHAPE, _VIEW, _VIEW, _VIEW, _VIEW, _VIEW, _VIEW, _P, _P, _P, _P, _P,
                                     _U64, _P], _INT),
    "adacomp_gated_scan_workspace_bytes": ([_SHAPE, ctypes.POINTER(_U64)], _INT),
    "adacomp_status_str": ([_INT], ctypes.c_char_p),
}

_lib = None


def lib():
    """The loaded HIP library; raises HipLibraryMissing if it is not built."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise HipLibraryMissing(
                f"{LIB_PATH} is not built; build it with __graft_entry__.build() "
                "(hipcc --offload-arch=gfx950)")
        h = ctypes.CDLL(str(LIB_PATH))
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = res
        _lib = h
    return _lib


def status_str(status: int) -> str:
    try:
        return lib().adacomp_status_str(int(status)).decode()
    except HipLibraryMissing:
        return "unknown"


def _check(where: str, st: int) -> None:
    if st != OK:
        raise AdaCompError(where, st)


def _segments(segments: Iterable[Sequence[int]]):
    segs = list(segments)
    arr = (_Segment * max(1, len(segs)))()
    for i, s in enumerate(segs):
        arr[i] = _Segment(int(s[0]), int(s[1]), int(s[2]), int(s[3]) if len(s) > 3 else 0)
    return arr, len(segs)


def plan_query(segments) -> PlanInfo:
    """Host-only: validate a segment table and return the sizes of its plan."""
    arr, n = _segments(segments)
    info = PlanInfo()
    _check("adacomp_plan_query", lib().adacomp_plan_query(arr, n, ctypes.byref(info)))
    return info


def _stream_handle(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    import torch
    try:   # the handle alone, without the Stream object around it (2.7 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _f32_ptr(t, name: str) -> int:
    import torch
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    return t.data_ptr()


def _u8_ptr(t, name: str) -> int:
    import torch
    if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous uint8 CUDA tensor")
    return t.data_ptr()


class Timer:
    """Per-kernel-stage device time recorded with HIP events on the stream."""

    def __init__(self):
        h = _P()
        _check("adacomp_timer_create", lib().adacomp_timer_create(ctypes.byref(h)))
        self.handle = h

    def read(self):
        ms = (ctypes.c_double * NUM_STAGES)()
        n = (_U64 * NUM_STAGES)()
        _check("adacomp_timer_read", lib().adacomp_timer_read(self.handle, ms, n, NUM_STAGES))
        return {STAGES[i]: (float(ms[i]), int(n[i])) for i in range(NUM_STAGES)}

    def reset(self):
        _check("adacomp_timer_reset", lib().adacomp_timer_reset(self.handle))

    def close(self):
        if self.handle:
            lib().adacomp_timer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Plan:
    """A segment table made into device tile tables on the current device.

    ``segments``: (offset, numel, bin_len) or (offset, numel, bin_len, flags)
    per layer, offsets in elements of the flat float32 buffers (multiples of
    4); flags 0 (AdaComp) or SEG_LS.  ``plan_flags``: 0, PLAN_SEPARATE_FINISH
    or PLAN_SINGLE_LAUNCH (``info.compress_launches`` says how many launches
    a compress call makes)."""

    def __init__(self, segments, plan_flags: int = 0):
        self.segments = [tuple(int(x) for x in s) for s in segments]
        arr, n = _segments(self.segments)
        h = _P()
        _check("adacomp_plan_create_ex",
               lib().adacomp_plan_create_ex(arr, n, int(plan_flags), ctypes.byref(h)))
        self.handle = h
        info = PlanInfo()
        _check("adacomp_plan_get_info", lib().adacomp_plan_get_info(h, ctypes.byref(info)))
        self.info = info

    def close(self):
        if getattr(self, "handle", None):
            lib().adacomp_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # Buffer helpers (torch allocations are 256-byte aligned).
    def message_buffer(self, device="cuda"):
        import torch
        return torch.empty(int(self.info.message_capacity), dtype=torch.uint8, device=device)

    def compress_workspace(self, device="cuda"):
        import torch
        return torch.empty(int(self.info.compress_workspace_bytes), dtype=torch.uint8, device=device)

    def decode_workspace(self, K: int, device="cuda"):
        import torch
        return torch.empty(self.info.decode_workspace_bytes(K), dtype=torch.uint8, device=device)

    def decode_sgd_workspace_bytes(self, K: int) -> int:
        n = _U64(0)
        _check("adacomp_decode_sgd_workspace_bytes",
               lib().adacomp_decode_sgd_workspace_bytes(self.handle, int(K), ctypes.byref(n)))
        return int(n.value)

    def decode_sgd_workspace(self, K: int, device="cuda"):
        import torch
        return torch.empty(self.decode_sgd_workspace_bytes(K), dtype=torch.uint8, device=device)


def compress(plan: Plan, residue, dW, msg, ws, bin_max_out=None, stream=None,
             timer: Optional[Timer] = None) -> None:
    """One AdaComp step: residue updated in place, message written to msg."""
    bm = _f32_ptr(bin_max_out, "bin_max_out") if bin_max_out is not None else None
    if bin_max_out is not None and bin_max_out.numel() < plan.info.total_bins:
        raise ValueError("bin_max_out shorter than the plan's total_bins")
    n = min(residue.numel(), dW.numel())
    st = lib().adacomp_compress_timed(
        plan.handle, _f32_ptr(residue, "residue"), _f32_ptr(dW, "dW"), n,
        _u8_ptr(msg, "msg"), msg.numel(), _u8_ptr(ws, "ws"), ws.numel(), bm,
        _stream_handle(stream), timer.handle if timer is not None else None)
    _check("adacomp_compress", st)


def compress_noalloc(plan: Plan, residue, dW, msg, bin_max_out=None, stream=None) -> None:
    """One AdaComp step as compress(), its workspace the library's own
    per-GPU scratch: the call allocates no device memory.  Calls that may
    overlap on one GPU race on that scratch."""
    bm = _f32_ptr(bin_max_out, "bin_max_out") if bin_max_out is not None else None
    if bin_max_out is not None and bin_max_out.numel() < plan.info.total_bins:
        raise ValueError("bin_max_out shorter than the plan's total_bins")
    n = min(residue.numel(), dW.numel())
    st = lib().adacomp_compress_noalloc(
        plan.handle, _f32_ptr(residue, "residue"), _f32_ptr(dW, "dW"), n,
        _u8_ptr(msg, "msg"), msg.numel(), bm, _stream_handle(stream))
    _check("adacomp_compress_noalloc", st)


def decode_accumulate(plan: Plan, msgs: List, out, accumulate: bool, ws, stream=None,
                      timer: Optional[Timer] = None) -> None:
    """Sum the messages (in list order) into out."""
    ptrs = (_P * max(1, len(msgs)))(*[_u8_ptr(m, "msgs[k]") for m in msgs])
    st = lib().adacomp_decode_accumulate_timed(
        plan.handle, ptrs, len(msgs), _f32_ptr(out, "out"), out.numel(),
        1 if accumulate else 0, _u8_ptr(ws, "ws"), ws.numel(), _stream_handle(stream),
        timer.handle if timer is not None else None)
    _check("adacomp_decode_accumulate", st)


def decode_sgd(plan: Plan, msgs: List, weights, momentum, lr: float, momentum_coef: float,
               ws, weight_decay: float = 0.0, scale: float = 1.0, stream=None,
               timer: Optional[Timer] = None) -> None:
    """Sum the messages (in list order) and take one SGD-with-momentum step on
    weights and momentum (in place), without writing the sum."""
    ptrs = (_P * max(1, len(msgs)))(*[_u8_ptr(m, "msgs[k]") for m in msgs])
    n = min(weights.numel(), momentum.numel())
    p = Sgd(lr, momentum_coef, weight_decay, scale)
    st = lib().adacomp_decode_sgd_timed(
        plan.handle, ptrs, len(msgs), _f32_ptr(weights, "weights"), _f32_ptr(momentum, "momentum"),
        n, ctypes.byref(p), _u8_ptr(ws, "ws"), ws.numel(), _stream_handle(stream),
        timer.handle if timer is not None else None)
    _check("adacomp_decode_sgd", st)


def decode_adam(plan: Plan, msgs: List, weights, m, v, lr: float, beta1: float, beta2: float,
                eps: float, step: int, ws, weight_decay: float = 0.0, scale: float = 1.0,
                stream=None, timer: Optional[Timer] = None) -> None:
    """Sum the messages (in list order) and take Adam step number ``step``
    (>= 1) on weights, m and v (in place), without writing the sum.  ws as
    for decode_sgd (Plan.decode_sgd_workspace)."""
    ptrs = (_P * max(1, len(msgs)))(*[_u8_ptr(x, "msgs[k]") for x in msgs])
    n = min(weights.numel(), m.numel(), v.numel())
    p = Adam(lr, beta1, beta2, eps, weight_decay, scale, int(step))
    st = lib().adacomp_decode_adam_timed(
        plan.handle, ptrs, len(msgs), _f32_ptr(weights, "weights"), _f32_ptr(m, "m"),
        _f32_ptr(v, "v"), n, ctypes.byref(p), _u8_ptr(ws, "ws"), ws.numel(),
        _stream_handle(stream), timer.handle if timer is not None else None)
    _check("adacomp_decode_adam", st)


def message_header(plan: Plan, msg):
    """Copy a message's header and directory to the host (synchronizes):
    (total_bytes, total_survivors, [(s, nsurv, entries_offset)] per segment)."""
    from .stats import read_header
    raw = bytes(msg[: int(plan.info.header_bytes)].cpu().numpy().tobytes())
    return read_header(raw, int(plan.info.nseg))


# --------------------------------------------------------------------------
# Operators of the training step around the compressor (include/adacomp.h).
# --------------------------------------------------------------------------

MOMENT_BLOCK = 32        # elements of one tensor that share the scales of their 8-bit moments
NORM_MAX_COLS = 65536    # longest row of layer_norm


_ops = None


def _operators():
    """The operators' native entry points (csrc/binding.cpp), which check the tensors and make the calls;
    raises HipLibraryMissing if they are not built."""
    global _ops
    if _ops is None:
        lib()
        import torch  # noqa: F401  the module is linked against torch's libraries
        try:
            from . import _binding
        except ImportError as e:
            raise HipLibraryMissing(f"the operators' entry points are not built ({e}); build them with "
                                    "__graft_entry__.build()") from e
        _ops = _binding
    return _ops


def _grad(grad):
    """(type code, address) of a gradient."""
    return _operators().gradient(grad)


class Optimizer:
    """A table of tensors made into the work tiles of the optimizer kernels on
    the current device.

    ``tensors``: (offset, numel, weight_decay, lr_scale) per tensor, offsets in
    elements of the flat buffers (multiples of 4)."""

    def __init__(self, tensors):
        self.tensors = [(int(o), int(n), float(d), float(r)) for o, n, d, r in tensors]
        arr, n = _tensors(self.tensors)
        h = _P()
        _check("adacomp_optimizer_create", lib().adacomp_optimizer_create(arr, n, ctypes.byref(h)))
        self.handle = h
        info = OptimizerInfo()
        _check("adacomp_optimizer_get_info", lib().adacomp_optimizer_get_info(h, ctypes.byref(info)))
        self.info = info
        self.span, self.nblocks, self.address = int(info.span), int(info.nblocks), h.value

    def close(self):
        if getattr(self, "handle", None):
            lib().adacomp_optimizer_destroy(self.handle)
            self.handle, self.address = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def norm_workspace(self, device="cuda"):
        import torch
        return torch.empty(int(self.info.norm_workspace_bytes), dtype=torch.uint8, device=device)

    def moment_scales(self, device="cuda"):
        """The scale bytes of 8-bit moments before the first step."""
        import torch
        return torch.zeros(2 * int(self.info.nblocks), dtype=torch.uint8, device=device)


def _tensors(tensors):
    arr = (_Tensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        arr[i] = _Tensor(int(t[0]), int(t[1]), float(t[2]), float(t[3]))
    return arr, len(tensors)


def optimizer_query(tensors) -> OptimizerInfo:
    """Host-only: validate a table of tensors and return the sizes its optimizer would have."""
    arr, n = _tensors(list(tensors))
    info = OptimizerInfo()
    _check("adacomp_optimizer_query", lib().adacomp_optimizer_query(arr, n, ctypes.byref(info)))
    return info


def grad_norm(opt: Optimizer, grad, clip, ws, max_norm: float, scale: float = 1.0, stream=None) -> None:
    """clip[0] = norm of scale * grad over the table's tensors, clip[1] = the factor that brings it
    down to max_norm."""
    st = _operators().grad_norm(opt.address, grad, clip, ws, max_norm, scale, stream)
    if st:
        raise AdaCompError("adacomp_grad_norm", st)


def adamw(opt: Optimizer, weights, grad, m, v, lr: float, beta1: float = 0.9, beta2: float = 0.999,
          eps: float = 1e-8, step: int = 1, scale: float = 1.0, clip=None, weights_bf16=None,
          stream=None) -> None:
    """AdamW step number ``step`` (>= 1) on weights, m and v (float32, in place) with the gradient
    scale * clip[1] * grad; weights_bf16 receives the new weights rounded."""
    st = _operators().adamw(opt.address, opt.span, opt.nblocks, weights, grad, m, v, None, lr, beta1, beta2, eps, step,
                            scale, 0, clip, weights_bf16, stream)
    if st:
        raise AdaCompError("adacomp_adamw_step", st)


def adamw_packed(opt: Optimizer, weights, grad, m, v, scales, lr: float, beta1: float = 0.9,
                 beta2: float = 0.999, eps: float = 1e-8, step: int = 1, scale: float = 1.0, seed: int = 0,
                 clip=None, weights_bf16=None, stream=None) -> None:
    """As adamw with moments in 8 bits: m and v e4m3 codes (float8_e4m3fn or uint8), scales as
    Optimizer.moment_scales gives them, updated in place; ``seed`` chooses the rounding's random bits."""
    if scales is None:
        raise TypeError("scales must be a tensor")
    st = _operators().adamw(opt.address, opt.span, opt.nblocks, weights, grad, m, v, scales, lr, beta1, beta2, eps, step,
                            scale, int(seed) & 0xFFFFFFFF, clip, weights_bf16, stream)
    if st:
        raise AdaCompError("adacomp_adamw_packed_step", st)


def layer_norm(x, weight, bias, out, mean=None, rstd=None, eps: float = 1e-5, stream=None) -> None:
    """Layer norm of x over its last axis into out; weight and bias float32 or None; mean and rstd
    (float32, one a row) are what layer_norm_backward needs."""
    st = _operators().layer_norm(x, weight, bias, out, mean, rstd, eps, stream)
    if st:
        raise AdaCompError("adacomp_layer_norm", st)


def layer_norm_workspace(rows: int, cols: int, device="cuda"):
    import torch
    n = _U64(0)
    _check("adacomp_layer_norm_workspace_bytes",
           lib().adacomp_layer_norm_workspace_bytes(int(rows), int(cols), ctypes.byref(n)))
    return torch.empty(int(n.value), dtype=torch.uint8, device=device)


def layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, ws=None,
                        stream=None) -> None:
    """Gradients of layer_norm: dx, and dweight and dbias (float32, both or neither)."""
    st = _operators().layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, ws, stream)
    if st:
        raise AdaCompError("adacomp_layer_norm_backward", st)


def gated_scan_workspace(batch: int, length: int, channels: int, device="cuda"):
    """Workspace of gated_scan and gated_scan_backward for one shape."""
    import torch
    n = _U64(0)
    shape = _ScanShape(int(length), int(batch), int(channels), 0, 0)
    _check("adacomp_gated_scan_workspace_bytes",
           lib().adacomp_gated_scan_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)))
    return torch.empty(int(n.value), dtype=torch.uint8, device=device)


def gated_scan(gate, x, h, h0=None, h_last=None, lengths=None, sigmoid: bool = True, ws=None,
               stream=None) -> None:
    """h_t = a_t h_(t-1) + k_t x_t along axis 1 of [batch, length, channels] tensors, with
    (a, k) = (sigmoid(gate), sigmoid(-gate)) or (gate, 1); h0 and h_last float32 [batch, channels]."""
    st = _operators().gated_scan(gate, x, h, h0, h_last, lengths, sigmoid, ws, stream)
    if st:
        raise AdaCompError("adacomp_gated_scan", st)


def gated_scan_backward(gate, x, h, dh, dgate, dx, h0=None, dh_last=None, dh0=None, lengths=None,
                        sigmoid: bool = True, ws=None, stream=None) -> None:
    """Gradients of gated_scan from the states h it wrote (x is not needed, and may be None, without
    the sigmoid)."""
    st = _operators().gated_scan_backward(gate, x, h, dh, dgate, dx, h0, dh_last, dh0, lengths, sigmoid, ws, stream)
    if st:
        raise AdaCompError("adacomp_gated_scan_backward", st)