"""Thin Python binding of the C ABI in include/qgemv.h.

Argument marshalling only: tensors are passed to the library as raw device
pointers with the current HIP stream, every step of the computation runs in
the library's kernels.  PyTorch supplies device memory and streams; output
tensors the caller does not provide are allocated here with torch.

The binding refuses to run without the compiled library: there is no
fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

from .build import LIB_PATH

FMT_Q4_ASYM_G64 = 1
FMT_Q8_SYM_G32 = 2
FMT_MXFP4_G32 = 3
FMT_Q8_ROW = 4


def affine_format(bits: int, group: int, bf16_scales: bool = False) -> int:
    """QG_FMT_AFFINE(bits, group, bf16_scales) of qgemv.h."""
    gc = {32: 0, 64: 1, 128: 2}.get(group, 3)
    return 0x100 | ((bits & 0xF) << 4) | (gc << 2) | (1 if bf16_scales else 0)

OUT_BF16 = 0
OUT_F32 = 1
OUT_I32_GROUPS = 2

KV_INT8 = 0
KV_E4M3 = 1

KERNEL_AUTO = 0
KERNEL_VALU = 1
KERNEL_MFMA = 2

QG_OK = 0
QG_EINVAL = -1
QG_ESHAPE = -2
QG_EALIGN = -3
QG_ESIZE = -4
QG_EUNSUPPORTED = -5
QG_EHIP = -6
QG_EINTERNAL = -7

# every function include/qgemv.h declares
EXPORTS = (
    "qg_status_string",
    "qg_version",
    "qgemv_pack",
    "qgemv_run",
    "qgemm_skinny_run",
    "hadamard32_quant_run",
    "qg_moe_workspace_bytes",
    "moe_expert_gemv_run",
    "moe_expert_gemv_run_noalloc",
    "qg_moe_skinny_workspace_bytes",
    "moe_expert_skinny_run",
    "qg_batch_worklist_bytes",
    "qg_batch_plan_build",
    "qg_batch_run",
    "qg_plain_read",
    "rmsnorm_quant_run",
    "kv_tables_run",
    "kv_append_run",
    "qg_kv_attention_workspace_bytes",
    "kv_attention_run",
)


class GemvDesc(C.Structure):
    """struct qg_gemv_desc"""
    _fields_ = [("packed", C.c_void_p), ("packed_bytes", C.c_size_t), ("N", C.c_int64),
                ("K", C.c_int64), ("x", C.c_void_p), ("y", C.c_void_p)]


class BatchPlan(C.Structure):
    """struct qg_batch_plan"""
    _fields_ = [("fmt", C.c_int32), ("M", C.c_int32), ("count", C.c_int32),
                ("out_dtype", C.c_int32), ("grid", C.c_int32), ("kmax", C.c_int32),
                ("kernel", C.c_int32), ("reserved1", C.c_int32), ("worklist", C.c_void_p),
                ("worklist_bytes", C.c_size_t)]


class CacheDesc(C.Structure):
    """struct qg_kv_cache"""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scales", C.c_void_p),
                ("v_scales", C.c_void_p), ("pages", C.c_int64), ("page", C.c_int32),
                ("Hkv", C.c_int32), ("D", C.c_int32), ("fmt", C.c_int32)]


_lock = threading.Lock()
_lib = None


class QGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


def raw():
    """The loaded library with argument types set (loads on first use)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    "libqgemv.so is not built (%s); run __graft_entry__.build() or "
                    "python -m quantized_weight_decode_dequant_amd.build" % LIB_PATH)
            lib = C.CDLL(LIB_PATH)
            i64, p, i, sz = C.c_int64, C.c_void_p, C.c_int, C.c_size_t
            lib.qg_status_string.argtypes = [i]
            lib.qg_status_string.restype = C.c_char_p
            lib.qg_version.argtypes = []
            lib.qg_version.restype = i
            lib.qgemv_pack.argtypes = [i, i64, i64, p, p, p, p, C.POINTER(sz), p]
            lib.qgemv_pack.restype = i
            lib.qgemv_run.argtypes = [i, p, sz, i64, i64, p, p, i, p]
            lib.qgemv_run.restype = i
            lib.qgemm_skinny_run.argtypes = [i, p, sz, i64, i64, i64, p, p, p, i, p]
            lib.qgemm_skinny_run.restype = i
            lib.hadamard32_quant_run.argtypes = [p, p, i64, i64, p, p, p]
            lib.hadamard32_quant_run.restype = i
            lib.qg_moe_workspace_bytes.argtypes = [i64, i64, i64]
            lib.qg_moe_workspace_bytes.restype = sz
            lib.moe_expert_gemv_run.argtypes = [p, p, p, sz, sz, sz, i64, i64, i64, p, i, p, p,
                                                p, sz, p, i, p]
            lib.moe_expert_gemv_run.restype = i
            lib.moe_expert_gemv_run_noalloc.argtypes = [p, p, p, sz, sz, sz, i64, i64, i64, p, i,
                                                        p, p, p, p, i, p]
            lib.moe_expert_gemv_run_noalloc.restype = i
            lib.qg_moe_skinny_workspace_bytes.argtypes = [i64, i64, i64, i64]
            lib.qg_moe_skinny_workspace_bytes.restype = sz
            lib.moe_expert_skinny_run.argtypes = [p, p, p, sz, sz, sz, i64, i64, i64, i64, p, i,
                                                  p, p, p, sz, p, i, p]
            lib.moe_expert_skinny_run.restype = i
            lib.qg_batch_worklist_bytes.argtypes = [C.c_int32]
            lib.qg_batch_worklist_bytes.restype = sz
            lib.qg_batch_plan_build.argtypes = [i, i64, C.c_int32, C.POINTER(GemvDesc), i, i, p, sz,
                                                C.POINTER(BatchPlan), p]
            lib.qg_batch_plan_build.restype = i
            lib.qg_batch_run.argtypes = [C.POINTER(BatchPlan), p]
            lib.qg_batch_run.restype = i
            lib.qg_plain_read.argtypes = [p, sz, p, i, p]
            lib.qg_plain_read.restype = i
            lib.rmsnorm_quant_run.argtypes = [p, i, p, p, i, p, C.c_float, p, i64, i64, p, p, p, p]
            lib.rmsnorm_quant_run.restype = i
            lib.kv_tables_run.argtypes = [i64, i64, i64, i64, i64, p, p, p, p, p, p, p, p, p, p, p]
            lib.kv_tables_run.restype = i
            lib.kv_append_run.argtypes = [p, i64, p, i64, p, i64, p, p]
            lib.kv_append_run.restype = i
            lib.qg_kv_attention_workspace_bytes.argtypes = [i64] * 9
            lib.qg_kv_attention_workspace_bytes.restype = sz
            lib.kv_attention_run.argtypes = [p, i64, i64, i64, p, i64, p, p, p, i64, p, i64,
                                             C.c_float, i64, i64, p, sz, p, i64, i, p]
            lib.kv_attention_run.restype = i
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return raw().qg_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != QG_OK:
        raise QGError(status, where)


# ------------------------------------------------------------------ torch glue
def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return C.c_void_p(stream)
    return C.c_void_p(stream.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


def _out_torch_dtype(out_dtype):
    torch = _torch()
    return {OUT_BF16: torch.bfloat16, OUT_F32: torch.float32, OUT_I32_GROUPS: torch.int32}[out_dtype]


# ------------------------------------------------------------------ API
def packed_bytes(fmt: int, rows: int, K: int) -> int:
    n = C.c_size_t(0)
    _check(raw().qgemv_pack(fmt, rows, K, None, None, None, None, C.byref(n), None), "qgemv_pack")
    return n.value


def qgemv_pack(fmt: int, rows: int, K: int, codes, scales, biases=None, out=None, stream=None):
    """Pack canonical device tensors; returns the packed uint8 device tensor."""
    torch = _torch()
    nbytes = packed_bytes(fmt, rows, K)
    if out is None:
        out = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=codes.device)
    cap = C.c_size_t(out.numel() * out.element_size())
    _check(raw().qgemv_pack(fmt, rows, K, _ptr(codes), _ptr(scales), _ptr(biases), _ptr(out),
                            C.byref(cap), _stream(stream)), "qgemv_pack")
    return out[:nbytes] if out.numel() != nbytes else out


def qgemv_run(fmt: int, packed, N: int, K: int, x, y=None, out_dtype: int = OUT_BF16,
              stream=None):
    torch = _torch()
    if y is None:
        y = torch.empty(N, dtype=_out_torch_dtype(out_dtype), device=x.device)
    _check(raw().qgemv_run(fmt, _ptr(packed), packed.numel(), N, K, _ptr(x), _ptr(y), out_dtype,
                           _stream(stream)), "qgemv_run")
    return y


def qgemm_skinny_run(fmt: int, packed, M: int, N: int, K: int, X, x_scales=None, Y=None,
                     out_dtype: int = OUT_BF16, stream=None):
    torch = _torch()
    if Y is None:
        shape = (M, N, K // 32) if out_dtype == OUT_I32_GROUPS else (M, N)
        Y = torch.empty(shape, dtype=_out_torch_dtype(out_dtype), device=X.device)
    _check(raw().qgemm_skinny_run(fmt, _ptr(packed), packed.numel(), M, N, K, _ptr(X),
                                  _ptr(x_scales), _ptr(Y), out_dtype, _stream(stream)),
           "qgemm_skinny_run")
    return Y


def hadamard32_quant_run(X, signs, M: int, K: int, Xq=None, x_scales=None, stream=None):
    torch = _torch()
    if Xq is None:
        Xq = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if x_scales is None:
        x_scales = torch.empty(M, dtype=torch.float32, device=X.device)
    _check(raw().hadamard32_quant_run(_ptr(X), _ptr(signs), M, K, _ptr(Xq), _ptr(x_scales),
                                      _stream(stream)), "hadamard32_quant_run")
    return Xq, x_scales


def moe_workspace_bytes(top_k: int, H: int, F: int) -> int:
    return raw().qg_moe_workspace_bytes(top_k, H, F)


def moe_expert_gemv_run(packed_gate, packed_up, packed_down, E: int, H: int, F: int, x,
                        expert_ids, expert_w, workspace=None, y=None, out_dtype: int = OUT_BF16,
                        stream=None):
    torch = _torch()
    top_k = int(expert_ids.numel())
    if workspace is None:
        workspace = torch.empty(moe_workspace_bytes(top_k, H, F), dtype=torch.uint8,
                                device=x.device)
    if y is None:
        y = torch.empty(H, dtype=_out_torch_dtype(out_dtype), device=x.device)
    _check(raw().moe_expert_gemv_run(_ptr(packed_gate), _ptr(packed_up), _ptr(packed_down),
                                     packed_gate.numel(), packed_up.numel(), packed_down.numel(),
                                     E, H, F, _ptr(x), top_k, _ptr(expert_ids), _ptr(expert_w),
                                     _ptr(workspace), workspace.numel(), _ptr(y), out_dtype,
                                     _stream(stream)), "moe_expert_gemv_run")
    return y


# the largest workspace moe_expert_gemv_run_noalloc serves (QG_MOE_NOALLOC_SCRATCH_BYTES)
MOE_NOALLOC_SCRATCH_BYTES = 2 << 20


def moe_expert_gemv_run_noalloc(packed_gate, packed_up, packed_down, E: int, H: int, F: int, x,
                                expert_ids, expert_w, status=None, y=None,
                                out_dtype: int = OUT_BF16, stream=None):
    """moe_expert_gemv_run on the library's own device array instead of a
    workspace; status: optional int32 device tensor [1] receiving the
    invalid-id flag."""
    torch = _torch()
    top_k = int(expert_ids.numel())
    if y is None:
        y = torch.empty(H, dtype=_out_torch_dtype(out_dtype), device=x.device)
    _check(raw().moe_expert_gemv_run_noalloc(
        _ptr(packed_gate), _ptr(packed_up), _ptr(packed_down), packed_gate.numel(),
        packed_up.numel(), packed_down.numel(), E, H, F, _ptr(x), top_k, _ptr(expert_ids),
        _ptr(expert_w), _ptr(status), _ptr(y), out_dtype, _stream(stream)),
        "moe_expert_gemv_run_noalloc")
    return y


def moe_skinny_workspace_bytes(T: int, top_k: int, H: int, F: int) -> int:
    return raw().qg_moe_skinny_workspace_bytes(T, top_k, H, F)


def moe_expert_skinny_run(packed_gate, packed_up, packed_down, E: int, H: int, F: int, X,
                          expert_ids, expert_w, workspace=None, Y=None,
                          out_dtype: int = OUT_BF16, stream=None):
    """X [T, H] bf16; expert_ids int32 / expert_w fp32 [T, top_k]; Y [T, H]."""
    torch = _torch()
    T = int(X.shape[0])
    top_k = int(expert_ids.shape[1]) if expert_ids.dim() == 2 else 0
    if tuple(expert_ids.shape) != (T, top_k) or tuple(expert_w.shape) != (T, top_k):
        raise ValueError("expert_ids and expert_w must be [T, top_k]")
    if workspace is None:
        workspace = torch.empty(moe_skinny_workspace_bytes(T, top_k, H, F), dtype=torch.uint8,
                                device=X.device)
    if Y is None:
        Y = torch.empty(T, H, dtype=_out_torch_dtype(out_dtype), device=X.device)
    _check(raw().moe_expert_skinny_run(_ptr(packed_gate), _ptr(packed_up), _ptr(packed_down),
                                       packed_gate.numel(), packed_up.numel(),
                                       packed_down.numel(), E, H, F, T, _ptr(X), top_k,
                                       _ptr(expert_ids), _ptr(expert_w), _ptr(workspace),
                                       workspace.numel(), _ptr(Y), out_dtype, _stream(stream)),
           "moe_expert_skinny_run")
    return Y


# ------------------------------------------------------------------ grouped launches
class Plan:
    """A built qg_batch_plan plus the device work list and the tensors its
    descriptors point at (kept alive as long as the plan)."""

    def __init__(self, plan, worklist, keep):
        self.plan = plan
        self.worklist = worklist
        self._keep = keep

    @property
    def grid(self) -> int:
        return self.plan.grid


def qg_batch_worklist_bytes(count: int) -> int:
    return raw().qg_batch_worklist_bytes(count)


def qg_batch_plan_build(fmt: int, M: int, entries, out_dtype: int = OUT_BF16, worklist=None,
                        stream=None, kernel: int = KERNEL_AUTO) -> Plan:
    """entries: sequence of (packed, N, K, x, y) with device tensors; x is bf16
    [M, K] ([K] for M = 1), y is [M, N] of the output type.  kernel: one of
    KERNEL_AUTO, KERNEL_VALU, KERNEL_MFMA."""
    torch = _torch()
    entries = list(entries)
    descs = (GemvDesc * len(entries))()
    keep = []
    for d, (packed, N, K, x, y) in zip(descs, entries):
        d.packed = _ptr(packed)
        d.packed_bytes = packed.numel()
        d.N, d.K = N, K
        d.x = _ptr(x)
        d.y = _ptr(y)
        keep.extend((packed, x, y))
    nbytes = qg_batch_worklist_bytes(len(entries))
    if worklist is None:
        dev = entries[0][0].device if entries else None
        worklist = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    plan = BatchPlan()
    _check(raw().qg_batch_plan_build(fmt, M, len(entries), descs, out_dtype, kernel, _ptr(worklist),
                                     worklist.numel(), C.byref(plan), _stream(stream)),
           "qg_batch_plan_build")
    return Plan(plan, worklist, keep)


def qg_plain_read(buf, sink, grid: int, stream=None):
    """Read the whole device tensor `buf` once (plain streaming loads); the
    XOR of each workgroup's words lands in sink[j] (int32 device tensor of at
    least `grid` elements)."""
    nbytes = buf.numel() * buf.element_size()
    if sink.numel() < grid:
        raise ValueError("sink holds %d words, grid is %d" % (sink.numel(), grid))
    _check(raw().qg_plain_read(_ptr(buf), nbytes, _ptr(sink), grid, _stream(stream)),
           "qg_plain_read")


def qg_batch_run(plan: Plan, stream=None):
    _check(raw().qg_batch_run(C.byref(plan.plan), _stream(stream)), "qg_batch_run")


# ------------------------------------------------------------------ norm, cache and attention
# These calls are short on the GPU (a few microseconds), so their checks are
# kept to a few attribute reads a tensor.
def _device(t):
    """The index of the device a tensor lies on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("expected a device tensor")
    return dev


def _arg(t, dtype, shape, dev, name):
    """The address of a contiguous tensor of this type and shape on `dev`
    (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s (got %s %s)"
                         % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be a device tensor on device %d (got %s)" % (name, dev, t.device))
    return t.data_ptr()


def _rows(t, H, D, dtype, dev, name):
    """Address and row stride of a [M, H, D] tensor whose rows are dense."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or shape[1] != H or shape[2] != D:
        raise ValueError("%s must be a %s tensor [M, %d, %d] (got %s %s)"
                         % (name, dtype, H, D, t.dtype, tuple(shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be a device tensor on device %d (got %s)" % (name, dev, t.device))
    row, head, dim = t.stride()
    if dim != 1 or (H > 1 and head != D):
        raise ValueError("%s: the heads and dimensions of a token must be dense" % name)
    return t.data_ptr(), (row if shape[0] > 1 else H * D)


def _call(dev, stream, where, fn, *args):
    """fn(*args, stream) with `dev` current; stream: as given, or dev's current one."""
    torch = _torch()
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _call(dev, stream, where, fn, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    status = fn(*args, stream)
    if status != QG_OK:
        raise QGError(status, where)


def _empty(shape, dtype, device, stream):
    """torch.empty for a call on `stream`: from that stream's memory, which
    work on no other stream may still be using."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _float_type(t, name):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return OUT_BF16
    if t.dtype is torch.float32:
        return OUT_F32
    raise ValueError("%s must be bfloat16 or float32 (got %s)" % (name, t.dtype))


def rmsnorm_quant_run(x, weight, eps: float, residual=None, residual_out=None, signs=None, y=None,
                      Xq=None, x_scales=None, stream=None):
    """Root-mean-square norm of x + residual; x [M, K] bf16 or fp32.  Outputs
    are written where a tensor is given: residual_out (may be residual), y
    (bf16 [M, K]), Xq and x_scales (int8 [M, K], fp32 [M]; one without the
    other is allocated); with none of them given, Xq and x_scales are.
    signs: rotate before quantizing.  Returns (residual_out, y, Xq, x_scales)."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    xt = _float_type(x, "x")
    if Xq is not None or x_scales is not None or y is None:
        if Xq is None:
            Xq = _empty((M, K), torch.int8, x.device, stream)
        if x_scales is None:
            x_scales = _empty(M, torch.float32, x.device, stream)
    if M == 0:
        return residual_out, y, Xq, x_scales
    dev, mk, i8 = _device(x), (M, K), torch.int8
    rt, rdt = (xt, x.dtype) if residual is None else (_float_type(residual, "residual"), residual.dtype)
    _call(dev, stream, "rmsnorm_quant_run", raw().rmsnorm_quant_run,
          _arg(x, x.dtype, mk, dev, "x"), xt, _arg(residual, rdt, mk, dev, "residual"),
          _arg(residual_out, rdt, mk, dev, "residual_out"), rt,
          _arg(weight, torch.bfloat16, (K,), dev, "weight"), eps, _arg(signs, i8, (K,), dev, "signs"),
          M, K, _arg(y, torch.bfloat16, mk, dev, "y"), _arg(Xq, i8, mk, dev, "Xq"),
          _arg(x_scales, torch.float32, (M,), dev, "x_scales"))
    return residual_out, y, Xq, x_scales


class KVCache:
    """One layer's paged cache: k and v [pages, Hkv, page, D] of torch.int8 or
    torch.float8_e4m3fn, k_scales and v_scales fp32 [pages, Hkv].  The bytes
    of a [page, D] block are in the order include/qgemv.h states."""

    def __init__(self, k, v, k_scales, v_scales):
        torch = _torch()
        if k.dim() != 4:
            raise ValueError("k must be [pages, Hkv, page, D]")
        pages, Hkv, page, D = k.shape
        fmt = {torch.int8: KV_INT8, torch.float8_e4m3fn: KV_E4M3}.get(k.dtype)
        if fmt is None:
            raise ValueError("codes must be int8 or float8_e4m3fn (got %s)" % k.dtype)
        dev, sc = _device(k), (pages, Hkv)
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.pages, self.page, self.Hkv, self.D, self.fmt, self.device = pages, page, Hkv, D, fmt, dev
        self.desc = CacheDesc(_arg(k, k.dtype, k.shape, dev, "k"), _arg(v, k.dtype, k.shape, dev, "v"),
                              _arg(k_scales, torch.float32, sc, dev, "k_scales"),
                              _arg(v_scales, torch.float32, sc, dev, "v_scales"), pages, page, Hkv, D, fmt)
        self._ref = C.addressof(self.desc)

    @classmethod
    def empty(cls, pages: int, page: int, Hkv: int, D: int, fmt: int = KV_INT8, device="cuda"):
        """A cache of unwritten pages."""
        torch = _torch()
        if fmt not in (KV_INT8, KV_E4M3):
            raise ValueError("unknown cache format %r" % (fmt,))
        dt = torch.int8 if fmt == KV_INT8 else torch.float8_e4m3fn
        codes = [torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device=device).view(dt)
                 for _ in range(2)]
        scales = [torch.zeros((pages, Hkv), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)


def kv_tables_run(page: int, lens, add, table, free_pages, free_count, max_tokens: int, keep=None,
                  q_start=None, slots=None, positions=None, status=None, stream=None):
    """One step of block tables, lengths and the free list (all updated in
    place); int32 tensors: lens, add, keep [R], table [R, max_blocks],
    free_pages [pages], free_count [1].  Returns (q_start [R + 1], slots
    [max_tokens], positions [max_tokens], status [1]); one that was given comes
    back as it is, and what it holds behind these sizes is left alone (not
    cut off: two views cost a tenth of a step of the tables)."""
    torch = _torch()
    i32 = torch.int32
    if lens.dim() != 1 or table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("lens, table and free_pages must be [R], [R, max_blocks] and [pages]")
    R, pages, nb = lens.shape[0], free_pages.shape[0], table.shape[1]

    def out(t, n, name):
        if t is None:
            return _empty(n, i32, lens.device, stream)
        if t.dim() != 1 or t.shape[0] < n:
            raise ValueError("%s must hold at least %d values" % (name, n))
        return t

    q_start, status = out(q_start, R + 1, "q_start"), out(status, 1, "status")
    slots, positions = out(slots, max_tokens, "slots"), out(positions, max_tokens, "positions")
    dev, r = _device(lens), (R,)
    _call(dev, stream, "kv_tables_run", raw().kv_tables_run, R, page, pages, nb, max_tokens,
          _arg(lens, i32, r, dev, "lens"), _arg(keep, i32, r, dev, "keep"), _arg(add, i32, r, dev, "add"),
          _arg(table, i32, (R, nb), dev, "table"), _arg(free_pages, i32, (pages,), dev, "free_pages"),
          _arg(free_count, i32, (1,), dev, "free_count"), _arg(q_start, i32, q_start.shape, dev, "q_start"),
          _arg(slots, i32, slots.shape, dev, "slots"), _arg(positions, i32, positions.shape, dev, "positions"),
          _arg(status, i32, status.shape, dev, "status"))
    return q_start, slots, positions, status


def kv_append_run(cache: KVCache, K, V, slots, stream=None):
    """Write K and V (bf16 [M, Hkv, D], rows at any multiple of 8 elements)
    into the cache's slots (int32 [M])."""
    torch = _torch()
    M = K.shape[0]
    if V.shape[0] != M:
        raise ValueError("K and V have %d and %d tokens" % (M, V.shape[0]))
    if M == 0:
        return
    dev, H, D, bf16 = cache.device, cache.Hkv, cache.D, torch.bfloat16
    kp, ks = _rows(K, H, D, bf16, dev, "K")
    vp, vs = _rows(V, H, D, bf16, dev, "V")
    _call(dev, stream, "kv_append_run", raw().kv_append_run, cache._ref, M, kp, ks, vp, vs,
          _arg(slots, torch.int32, (M,), dev, "slots"))


def kv_attention_workspace_bytes(R: int, M: int, Hq: int, Hkv: int, D: int, page: int, max_q: int,
                                 max_len: int, window: int = 0) -> int:
    return raw().qg_kv_attention_workspace_bytes(R, M, Hq, Hkv, D, page, max_q, max_len, window)


def kv_attention_run(cache: KVCache, q, q_start, lens, table, max_q: int, max_len=None,
                     tree_mask=None, window: int = 0, scale=None, workspace=None, out=None,
                     out_dtype: int = OUT_BF16, stream=None):
    """Attention of the new tokens q (bf16 [M, Hq, D]) over the cache; q_start
    int32 [R + 1], lens int32 [R] (new tokens included), table int32 [R,
    max_blocks]; max_q: the most new tokens a request has; max_len: the
    longest request (the table's width by default); tree_mask int32 [M].
    scale: 1 / sqrt(D) by default.  Returns out [M, Hq, D]."""
    torch = _torch()
    i32 = torch.int32
    if q.dim() != 3 or table.dim() != 2:
        raise ValueError("q must be [M, Hq, D] and table [R, max_blocks]")
    M, Hq, D = q.shape
    R, nb = table.shape
    if max_len is None:
        max_len = nb * cache.page
    if out is None:
        out = _empty((M, Hq, D), _out_torch_dtype(out_dtype), q.device, stream)
    else:
        out_dtype = _float_type(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if M == 0 or R == 0:
        return out
    dev, D = cache.device, cache.D
    qp, qs = _rows(q, Hq, D, torch.bfloat16, dev, "q")
    op, os_ = _rows(out, Hq, D, out.dtype, dev, "out")
    lib = raw()
    if workspace is None:
        nbytes = lib.qg_kv_attention_workspace_bytes(R, M, Hq, cache.Hkv, D, cache.page, max_q, max_len, window)
        workspace = _empty(nbytes, torch.uint8, q.device, stream) if nbytes else None
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _call(dev, stream, "kv_attention_run", lib.kv_attention_run, cache._ref, R, M, Hq, qp, qs,
          _arg(q_start, i32, (R + 1,), dev, "q_start"), _arg(lens, i32, (R,), dev, "lens"),
          _arg(table, i32, (R, nb), dev, "table"), nb, _arg(tree_mask, i32, (M,), dev, "tree_mask"), window,
          scale if scale is not None else D ** -0.5, max_q, max_len,
          _arg(workspace, workspace.dtype, workspace.shape, dev, "workspace") if nbytes else None, nbytes,
          op, os_, out_dtype)
    return out
