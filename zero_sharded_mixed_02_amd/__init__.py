"""Python binding of libzero.so: one data-parallel rank's share of a ZeRO
mixed-precision training step on an MI355X (gfx950).

Thin ctypes marshalling over the C ABI in ``include/zero.h``: every function
here has the C entry point's name and arguments, converts tensors to device
addresses and streams to ``hipStream_t`` handles, and raises ``ZeroError`` on a
non-OK status.  All computation happens in the HIP kernels of libzero.so; if
the library has not been built, loading fails loudly (there is no fallback).

Tensors may be passed as ``torch.Tensor`` or as plain integer device
addresses.  A tensor is checked against the plan before the C call -- a
contiguous GPU tensor of the right element size holding at least the elements
the plan needs (exactly tensor t's size for flatten inputs) -- and pointer
lists must have one entry per rank or tensor; a failed check raises
``ValueError`` and nothing is launched.  A plain integer address is passed
through unchecked: the caller vouches for it.  ``stream=None`` means torch's
current stream on the current device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libzero.so")

ZERO_F32, ZERO_F16, ZERO_BF16 = 0, 1, 2
ZERO_I32, ZERO_I64 = 0, 1
ZERO_OK, ZERO_EINVAL, ZERO_EUNSUPPORTED, ZERO_ENOMEM, ZERO_EHIP = 0, -1, -2, -3, -4
ZERO_MAX_RANKS = 128

STATUS_NAMES = {0: "ZERO_OK", -1: "ZERO_EINVAL", -2: "ZERO_EUNSUPPORTED", -3: "ZERO_ENOMEM",
                -4: "ZERO_EHIP"}

# Names of every entry point include/zero.h declares.
ENTRY_POINTS = ("zero_version", "zero_last_error", "zero_plan", "zero_plan_destroy",
                "zero_plan_info", "zero_plan_bucket", "zero_plan_tensor", "zero_flatten_workspace_bytes",
                "zero_flatten", "zero_shard_reduce", "zero_adam_step", "zero_gather_pack", "zero_reshard",
                "zero_set_write_window", "zero_set_stream_write_window", "zero_set_warm_read",
                "zero_embed", "zero_token_order_workspace_bytes", "zero_token_order",
                "zero_embed_grad_workspace_bytes", "zero_embed_grad", "zero_dropout",
                "zero_token_logp_workspace_bytes", "zero_token_logp", "zero_preference_loss",
                "zero_token_logp_grad")


class ZeroError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class _AdamHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("grad_scale", ctypes.c_double)]


class _GradSrc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n", ctypes.c_int32),
                ("ptrs", ctypes.POINTER(ctypes.c_void_p)), ("is_full", ctypes.POINTER(ctypes.c_uint8))]


class _Drop(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("site", ctypes.c_uint64),
                ("step", ctypes.c_uint64), ("step_dev", ctypes.c_void_p), ("first", ctypes.c_int64)]


_lib = None


def _share_torch_hip_runtime():
    """PyTorch brings its own copy of the HIP runtime (same soname as
    /opt/rocm's).  Device memory and streams come from torch, so libzero.so
    must bind to that same runtime: loading torch first makes the dynamic
    loader resolve libzero's libamdhip64.so.7 to torch's already-loaded copy
    instead of opening a second runtime in the process."""
    try:
        import torch  # noqa: F401
    except ImportError:
        pass


def load():
    """Load libzero.so.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libzero.so not built at {LIB_PATH}; run __graft_entry__.build()")
    _share_torch_hip_runtime()
    L = ctypes.CDLL(LIB_PATH)
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    p_i64, p_i32 = ctypes.POINTER(i64), ctypes.POINTER(i32)
    L.zero_version.restype = i32
    L.zero_version.argtypes = []
    L.zero_last_error.restype = ctypes.c_char_p
    L.zero_last_error.argtypes = []
    L.zero_plan.restype = i32
    L.zero_plan.argtypes = [i64, i32, p_i64, i32, i64, i32, ctypes.POINTER(vp)]
    L.zero_plan_destroy.restype = None
    L.zero_plan_destroy.argtypes = [vp]
    L.zero_plan_info.restype = i32
    L.zero_plan_info.argtypes = [vp, p_i64, p_i64, p_i32, p_i32]
    L.zero_plan_bucket.restype = i32
    L.zero_plan_bucket.argtypes = [vp, i32, p_i64, p_i64, p_i64, p_i64, p_i64]
    L.zero_plan_tensor.restype = i32
    L.zero_plan_tensor.argtypes = [vp, i32, p_i32, p_i64]
    L.zero_flatten_workspace_bytes.restype = ctypes.c_size_t
    L.zero_flatten_workspace_bytes.argtypes = [vp]
    L.zero_flatten.restype = i32
    L.zero_flatten.argtypes = [vp, ctypes.POINTER(vp), i32, vp, vp, ctypes.c_size_t, vp]
    L.zero_shard_reduce.restype = i32
    L.zero_shard_reduce.argtypes = [vp, i32, ctypes.POINTER(_GradSrc), ctypes.c_double, vp, vp]
    L.zero_adam_step.restype = i32
    L.zero_adam_step.argtypes = [vp, i32, ctypes.POINTER(_AdamHyper), i64, ctypes.POINTER(_GradSrc),
                                 vp, vp, vp, vp, vp, i32, i32, vp]
    L.zero_gather_pack.restype = i32
    L.zero_gather_pack.argtypes = [vp, ctypes.POINTER(vp), i32, vp, vp]
    L.zero_reshard.restype = i32
    L.zero_reshard.argtypes = [vp, vp, i32, ctypes.POINTER(vp), i32, vp, vp]
    L.zero_set_write_window.restype = i32
    L.zero_set_write_window.argtypes = [i64, i64]
    L.zero_set_stream_write_window.restype = i32
    L.zero_set_stream_write_window.argtypes = [vp, i64, i64]
    L.zero_set_warm_read.restype = i32
    L.zero_set_warm_read.argtypes = [i32]
    f64, size = ctypes.c_double, ctypes.c_size_t
    p_drop = vp   # a zero_drop by reference, or NULL
    L.zero_embed.restype = i32
    L.zero_embed.argtypes = [vp, i32, i64, vp, i32, vp, i32, i64, f64, p_drop, vp, i32, i64, vp]
    L.zero_token_order_workspace_bytes.restype = size
    L.zero_token_order_workspace_bytes.argtypes = [i64, i64]
    L.zero_token_order.restype = i32
    L.zero_token_order.argtypes = [vp, i32, i64, i64, vp, vp, vp, size, vp]
    L.zero_embed_grad_workspace_bytes.restype = size
    L.zero_embed_grad_workspace_bytes.argtypes = [i64, i64]
    L.zero_embed_grad.restype = i32
    L.zero_embed_grad.argtypes = [vp, i32, i64, vp, vp, i64, vp, i32, i64, f64, p_drop, vp, i32, i32, i32, vp,
                                  size, vp]
    L.zero_dropout.restype = i32
    L.zero_dropout.argtypes = [vp, vp, vp, i64, i32, p_drop, vp]
    L.zero_token_logp_workspace_bytes.restype = size
    L.zero_token_logp_workspace_bytes.argtypes = [i64, i64]
    L.zero_token_logp.restype = i32
    L.zero_token_logp.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, size, vp]
    L.zero_preference_loss.restype = i32
    L.zero_preference_loss.argtypes = [i64, vp, i32, i64, vp, i32, i64, vp, vp, f64, f64, f64, vp, vp, vp, vp, vp]
    L.zero_token_logp_grad.restype = i32
    L.zero_token_logp_grad.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, i64, vp]
    _lib = L
    return L


def _check(status: int):
    if status != ZERO_OK:
        raise ZeroError(status, load().zero_last_error().decode(errors="replace"))


def _addr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


ESIZE = {ZERO_F32: 4, ZERO_F16: 2, ZERO_BF16: 2}


def _esize(dt: int) -> int:
    if dt not in ESIZE:
        raise ValueError(f"unknown dtype {dt}")
    return ESIZE[dt]


def _tensor_props(x, name: str, esize: int):
    """(element count, on a GPU) of tensor x after checking what does not
    depend on the plan: a contiguous tensor whose elements are esize bytes."""
    if not hasattr(x, "data_ptr") or not hasattr(x, "element_size"):
        raise TypeError(f"{name}: expected a torch tensor or an integer device address, got {type(x).__name__}")
    if x.element_size() != esize:
        raise ValueError(f"{name}: elements of {x.element_size()} bytes ({x.dtype}), expected {esize}")
    if not x.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return int(x.numel()), bool(x.is_cuda)


def _arg(x, name: str, esize: int, need: int, exact: bool = False) -> int:
    """Device address of x.  A tensor must be a contiguous GPU tensor holding
    at least `need` elements of esize bytes (exactly `need` with exact=True);
    None and integer addresses are passed through (the C side rejects a NULL
    it cannot accept)."""
    if x is None or isinstance(x, int):
        return _addr(x)
    n, on_gpu = _tensor_props(x, name, esize)
    if n < need or (exact and n != need):
        raise ValueError(f"{name} holds {n} elements, the plan needs {'exactly ' if exact else ''}{need}")
    if not on_gpu:
        raise ValueError(f"{name} is not on a GPU ({x.device})")
    return int(x.data_ptr())


def _arg_list(xs, name: str, count: int, esize: int, need: int, exact: bool = False) -> ctypes.Array:
    if xs is None:
        raise ValueError(f"{name} is None")
    xs = list(xs)
    if len(xs) != count:
        raise ValueError(f"{name} has {len(xs)} entries, the plan needs {count}")
    per = isinstance(need, (list, tuple))
    addrs = []
    for i, x in enumerate(xs):
        want = need[i] if per else need
        # Fast path for the common case (a contiguous GPU tensor of the right
        # element size and length); anything else goes through _arg, which
        # raises with the argument's name.
        try:
            if x.element_size() == esize and x.is_contiguous() and x.is_cuda:
                n = x.numel()
                if n == want or (n > want and not exact):
                    addrs.append(x.data_ptr())
                    continue
        except AttributeError:
            pass
        addrs.append(_arg(x, f"{name}[{i}]", esize, want, exact))
    return (ctypes.c_void_p * max(1, count))(*addrs)


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def zero_version() -> int:
    return int(load().zero_version())


WINDOW_AUTO = -1


def zero_set_write_window(period_ticks: int, open_ticks: int = 0) -> None:
    """Process-wide default store scheduling of the fused step and the
    reduction (results are identical): -1 automatic (default), 0 none, else a
    period of period_ticks real-time-counter ticks whose first open_ticks
    admit stores."""
    _check(load().zero_set_write_window(period_ticks, open_ticks))


WINDOW_INHERIT = -2


def zero_set_stream_write_window(stream, period_ticks: int, open_ticks: int = 0) -> None:
    """The same setting for launches on one stream only; -2 removes the
    stream's own setting so it follows the process-wide default again."""
    _check(load().zero_set_stream_write_window(_stream(stream), period_ticks, open_ticks))


def zero_set_warm_read(enable: bool) -> None:
    """Read up to 256 MiB of the fused step's own state just before each
    large fused step (process-wide; off by default)."""
    _check(load().zero_set_warm_read(1 if enable else 0))


def zero_last_error() -> str:
    return load().zero_last_error().decode(errors="replace")


class Plan:
    """Owner of a zero_plan_t handle, with its queries."""

    def __init__(self, handle: int, tensor_numel: Sequence[int]):
        self._h = ctypes.c_void_p(handle)
        self.tensor_numel = [int(n) for n in tensor_numel]
        self.n_tensors = len(self.tensor_numel)
        L = load()
        psi_pad, shard_total = ctypes.c_int64(), ctypes.c_int64()
        nb, nd = ctypes.c_int32(), ctypes.c_int32()
        _check(L.zero_plan_info(self._h, ctypes.byref(psi_pad), ctypes.byref(shard_total),
                                ctypes.byref(nb), ctypes.byref(nd)))
        self.psi_pad, self.shard_total = psi_pad.value, shard_total.value
        self.n_buckets, self.n_d = nb.value, nd.value

    @property
    def handle(self):
        return self._h

    def bucket(self, b: int):
        """(flat_off, numel, padded, shard_numel, shard_off) of bucket b."""
        vals = [ctypes.c_int64() for _ in range(5)]
        _check(load().zero_plan_bucket(self._h, b, *[ctypes.byref(v) for v in vals]))
        return tuple(v.value for v in vals)

    def tensor(self, t: int):
        """(bucket, flat_off) of tensor t."""
        b, off = ctypes.c_int32(), ctypes.c_int64()
        _check(load().zero_plan_tensor(self._h, t, ctypes.byref(b), ctypes.byref(off)))
        return b.value, off.value

    def buckets(self):
        return [self.bucket(b) for b in range(self.n_buckets)]

    def close(self):
        if self._h is not None and self._h.value:
            load().zero_plan_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def zero_plan(psi: int, n_d: int, tensor_numel: Sequence[int], bucket_cap: int = 0,
              shard_align: int = 64) -> Plan:
    n = len(tensor_numel)
    arr = (ctypes.c_int64 * max(1, n))(*tensor_numel)
    h = ctypes.c_void_p()
    _check(load().zero_plan(psi, n_d, arr, n, bucket_cap, shard_align, ctypes.byref(h)))
    return Plan(h.value, tensor_numel)


class GradSrc:
    """The N_d gradient contributions (zero_grad_src).  Tensors are checked
    here (16-bit elements, contiguous, on a GPU) and kept referenced; their
    sizes are compared with the plan at every call."""

    def __init__(self, dtype: int, ptrs: Sequence, is_full: Optional[Sequence[int]] = None):
        if dtype not in (ZERO_F16, ZERO_BF16):
            raise ValueError(f"gradient dtype {dtype} is not 16-bit")
        ptrs = list(ptrs)
        self.dtype = dtype
        self.n = len(ptrs)
        if is_full is not None and len(is_full) != self.n:
            raise ValueError(f"is_full has {len(is_full)} entries for {self.n} gradient buffers")
        self.is_full = [0] * self.n if is_full is None else [1 if f else 0 for f in is_full]
        self._keep = ptrs
        # Smallest tensor among the compact and among the full contributions
        # (plain addresses are not counted: the caller vouches for them).
        self.min_compact = self.min_full = None
        self.not_on_gpu = None   # name of the first tensor that is not on a GPU
        for q, x in enumerate(ptrs):
            if x is None or isinstance(x, int):
                continue
            n, on_gpu = _tensor_props(x, f"gradient of rank {q}", 2)
            if not on_gpu and self.not_on_gpu is None:
                self.not_on_gpu = f"gradient of rank {q} ({x.device})"
            if self.is_full[q]:
                self.min_full = n if self.min_full is None else min(self.min_full, n)
            else:
                self.min_compact = n if self.min_compact is None else min(self.min_compact, n)
        self._ptrs = (ctypes.c_void_p * max(1, self.n))(*[_addr(x) for x in ptrs])
        self._full = None if is_full is None else (ctypes.c_uint8 * max(1, self.n))(*self.is_full)
        self.c = _GradSrc(dtype, self.n, ctypes.cast(self._ptrs, ctypes.POINTER(ctypes.c_void_p)),
                          None if self._full is None else ctypes.cast(self._full, ctypes.POINTER(ctypes.c_uint8)))

    def check(self, plan: "Plan") -> None:
        if self.n != plan.n_d:
            raise ValueError(f"gradient source has {self.n} ranks, the plan has n_d={plan.n_d}")
        if self.min_compact is not None and self.min_compact < plan.shard_total:
            raise ValueError(f"a compact gradient slice holds {self.min_compact} elements, "
                             f"the plan needs {plan.shard_total}")
        if self.min_full is not None and self.min_full < plan.psi_pad:
            raise ValueError(f"a full gradient buffer holds {self.min_full} elements, the plan needs {plan.psi_pad}")
        if self.not_on_gpu is not None:
            raise ValueError(f"{self.not_on_gpu} is not on a GPU")


def zero_flatten_workspace_bytes(plan: Plan) -> int:
    return int(load().zero_flatten_workspace_bytes(plan.handle))


def zero_flatten(plan: Plan, tensors: Sequence, dt: int, flat, stream=None, workspace=None,
                 ws_bytes: int = 0) -> None:
    es = _esize(dt)
    arr = _arg_list(tensors, "tensors", plan.n_tensors, es, plan.tensor_numel, exact=True)
    out = _arg(flat, "flat", es, plan.psi_pad)
    ws = _addr(workspace)
    _check(load().zero_flatten(plan.handle, arr, dt, out, ws, ws_bytes, _stream(stream)))


def zero_shard_reduce(plan: Plan, rank: int, src: GradSrc, grad_scale: float, out, stream=None) -> None:
    src.check(plan)
    o = _arg(out, "out", 4, plan.shard_total)
    _check(load().zero_shard_reduce(plan.handle, rank, ctypes.byref(src.c), grad_scale, o, _stream(stream)))


def zero_adam_step(plan: Plan, rank: int, lr: float, beta1: float, beta2: float, eps: float,
                   grad_scale: float, t: int, slices: Optional[GradSrc], reduced, master, m, v,
                   param_dst, param_dt: int, dst_is_full: bool, stream=None) -> None:
    S = plan.shard_total
    if slices is not None:
        slices.check(plan)
        red = 0
    else:
        red = _arg(reduced, "reduced", 4, S)
    w_, m_, v_ = _arg(master, "master", 4, S), _arg(m, "m", 4, S), _arg(v, "v", 4, S)
    if param_dt not in (ZERO_F16, ZERO_BF16):
        raise ValueError(f"parameter dtype {param_dt} is not 16-bit")
    dst = _arg(param_dst, "param_dst", 2, plan.psi_pad if dst_is_full else S)
    hp = _AdamHyper(lr, beta1, beta2, eps, grad_scale)
    _check(load().zero_adam_step(plan.handle, rank, ctypes.byref(hp), t,
                                 None if slices is None else ctypes.byref(slices.c), red,
                                 w_, m_, v_, dst, param_dt, 1 if dst_is_full else 0, _stream(stream)))


def zero_gather_pack(plan: Plan, shards: Sequence, dt: int, full, stream=None) -> None:
    es = _esize(dt)
    arr = _arg_list(shards, "shards", plan.n_d, es, plan.shard_total)
    out = _arg(full, "full", es, plan.psi_pad)
    _check(load().zero_gather_pack(plan.handle, arr, dt, out, _stream(stream)))


def zero_reshard(src_plan: Plan, dst_plan: Plan, dst_rank: int, src_shards: Sequence, dt: int, dst_shard,
                 stream=None) -> None:
    es = _esize(dt)
    arr = _arg_list(src_shards, "src_shards", src_plan.n_d, es, src_plan.shard_total)
    out = _arg(dst_shard, "dst_shard", es, dst_plan.shard_total)
    _check(load().zero_reshard(src_plan.handle, dst_plan.handle, dst_rank, arr, dt, out, _stream(stream)))


# ---------------------------------------------------------------------------
# Operators at the two ends of the model (see include/zero.h)
# ---------------------------------------------------------------------------
#
# Tensors are checked as above.  2-D arguments may have rows further apart than
# they are wide (a slice of a wider activation); a contiguous tensor of any
# shape with n * width elements is taken as n rows.  A call whose tensors lie
# on another GPU than the current one is issued there, on that GPU's current
# stream unless a stream is passed.  Where addresses are passed as integers,
# the keyword arguments give what a tensor would tell.

class Drop:
    """Which elements a dropout keeps (zero_drop): the share dropped, and the
    numbers that the mask follows from.  step_dev, an int64 or uint64 tensor
    of one element on the GPU (or its address), is read when the kernel runs
    in place of step."""

    def __init__(self, p: float, seed: int, site: int = 0, step: int = 0, first: int = 0, step_dev=None):
        mask = (1 << 64) - 1
        self._keep = step_dev
        addr = None if step_dev is None else _arg(step_dev, "step_dev", 8, 1) or None
        self.c = _Drop(p, seed & mask, site & mask, step & mask, addr, first)
        self._ref = ctypes.byref(self.c)


# torch's current stream of a device as an integer, and its current device:
# the functions below torch.cuda's own, where torch has them, since a Stream
# object alone takes 2.8 us to build.
_raw_stream = _current_device = None


def _bind_torch() -> None:
    global _raw_stream, _current_device
    import torch
    torch.cuda.current_device()   # initialises torch's GPU side
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: int(torch.cuda.current_stream(d).cuda_stream))
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_ID_TYPES = {}       # torch integer types -> zero_itype


def _id_type(dtype):
    if not _ID_TYPES:
        import torch
        _ID_TYPES.update({torch.int32: ZERO_I32, torch.int64: ZERO_I64})
    return _ID_TYPES.get(dtype)


class _Call:
    """The device and stream of one call, gathered from its tensors."""

    __slots__ = ("stream", "device")

    def __init__(self, stream):
        self.stream, self.device = stream, None

    def see(self, x, name: str) -> None:
        if x is None or isinstance(x, int):
            return
        if not x.is_cuda:
            raise ValueError(f"{name} is not on a GPU ({x.device})")
        i = x.get_device()
        if self.device is None:
            self.device = i
        elif self.device != i:
            raise ValueError(f"{name} is on cuda:{i}, other arguments on cuda:{self.device}")

    def flat(self, x, name: str, esize: int, need: int, optional: bool = False) -> int:
        """Address of a contiguous buffer of at least need elements."""
        if x is None:
            if not optional and need > 0:
                raise ValueError(f"{name} is None")
            return 0
        try:   # the common case: a tensor that fits, on the call's device
            device = x.get_device()
            if (device >= 0 and (self.device is None or device == self.device) and x.numel() >= need
                    and x.element_size() == esize and x.is_contiguous()):
                self.device = device
                return x.data_ptr()
        except AttributeError:
            if isinstance(x, int):
                return x
        addr = _arg(x, name, esize, need)
        self.see(x, name)
        return addr

    def rows(self, x, name: str, esize: int, n: int, width: int, stride):
        """(address, row stride) of n rows of width elements."""
        if x is None:
            if n > 0:
                raise ValueError(f"{name} is None")
            return 0, width
        try:   # the common case, as above
            device = x.get_device()
            if (device >= 0 and (self.device is None or device == self.device) and x.numel() == n * width
                    and x.element_size() == esize and x.is_contiguous()):
                self.device = device
                return x.data_ptr(), width
        except AttributeError:
            if isinstance(x, int):
                return x, width if stride is None else stride
            raise TypeError(f"{name}: expected a torch tensor or an integer device address, got {type(x).__name__}")
        if x.element_size() != esize:
            raise ValueError(f"{name}: elements of {x.element_size()} bytes ({x.dtype}), expected {esize}")
        if x.numel() != n * width:
            raise ValueError(f"{name} holds {x.numel()} elements, expected {n} rows of {width}")
        self.see(x, name)
        if x.dim() != 2 or x.shape[1] != width or (width > 1 and x.stride(1) != 1) or (n > 1 and x.stride(0) < width):
            raise ValueError(f"{name}: rows must be contiguous (shape {tuple(x.shape)}, strides {x.stride()})")
        return x.data_ptr(), x.stride(0) if n > 1 else width

    def ids(self, x, name: str, n, it):
        """(address, integer type, count) of an id list."""
        try:   # the common case, as above
            device, kind = x.get_device(), _ID_TYPES.get(x.dtype)
            if (kind is not None and device >= 0 and (self.device is None or device == self.device)
                    and x.is_contiguous() and (n is None or n == x.numel())):
                self.device = device
                return x.data_ptr(), kind, x.numel()
        except AttributeError:
            if x is not None and not isinstance(x, int):
                raise TypeError(f"{name}: expected a torch tensor or an integer device address, got {type(x).__name__}")
            if n is None or it is None:
                raise ValueError(f"{name} is not a tensor: pass its count and integer type")
            return _addr(x), it, int(n)
        kind = _id_type(x.dtype)
        if kind is None:
            raise ValueError(f"{name} must be int32 or int64, got {x.dtype}")
        if not x.is_contiguous():
            raise ValueError(f"{name} is not contiguous")
        self.see(x, name)
        count = x.numel()
        if n is not None and int(n) != count:
            raise ValueError(f"{name} holds {count} elements, expected {n}")
        return x.data_ptr(), kind, count

    def workspace(self, x, need):
        """(address, bytes); an integer address is taken to hold the need()."""
        if x is None or isinstance(x, int):
            return _addr(x), need() if x else 0
        if not hasattr(x, "data_ptr") or not x.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor or an integer device address")
        self.see(x, "workspace")
        return x.data_ptr(), x.nbytes

    def drop(self, d):
        if d is None:
            return None
        if not isinstance(d, Drop):
            raise TypeError(f"drop: expected a Drop, got {type(d).__name__}")
        if d._keep is not None:
            self.see(d._keep, "step_dev")
        return d._ref

    def issue(self, fn, *args) -> None:
        """Calls fn with the stream, on the tensors' device."""
        device = self.device
        if device is None:
            status = fn(*args, _stream(self.stream))
        else:
            if _current_device is None:
                _bind_torch()
            stream = _raw_stream(device) if self.stream is None else _stream(self.stream)
            if _current_device() == device:
                status = fn(*args, stream)
            else:
                import torch
                with torch.cuda.device(device):
                    status = fn(*args, stream)
        if status != ZERO_OK:
            _check(status)


def zero_embed(plan: Plan, tensor: int, hidden: int, params, param_dt: int, tokens, scale: float, out, out_dt: int,
               drop: Optional[Drop] = None, stream=None, n: Optional[int] = None, token_it: Optional[int] = None,
               out_stride: Optional[int] = None) -> None:
    """out[i] = dropout(scale * table[tokens[i]]); the table is a tensor of the
    plan inside the full parameter buffer params.  Ids outside the table give
    rows of zeros."""
    c = _Call(stream)
    par = c.flat(params, "params", _esize(param_dt), plan.psi_pad)
    tok, it, n = c.ids(tokens, "tokens", n, token_it)
    o, ostride = c.rows(out, "out", _esize(out_dt), n, hidden, out_stride)
    keep = c.drop(drop)
    c.issue(load().zero_embed, plan.handle, tensor, hidden, par, param_dt, tok, it, n, scale, keep, o, out_dt,
            ostride)


def zero_token_order_workspace_bytes(n: int, rows: int) -> int:
    return int(load().zero_token_order_workspace_bytes(n, rows))


def zero_token_order(tokens, rows: int, sorted, order, workspace=None, stream=None, n: Optional[int] = None,
                     token_it: Optional[int] = None) -> None:
    """Positions of the tokens in token order (order, int32) and the tokens in
    that order (sorted, int32; padding ids last, as rows)."""
    c = _Call(stream)
    tok, it, n = c.ids(tokens, "tokens", n, token_it)
    s = c.flat(sorted, "sorted", 4, n)
    o = c.flat(order, "order", 4, n)
    ws, ws_bytes = c.workspace(workspace, lambda: zero_token_order_workspace_bytes(n, rows))
    c.issue(load().zero_token_order, tok, it, n, rows, s, o, ws, ws_bytes)


def zero_embed_grad_workspace_bytes(n: int, hidden: int) -> int:
    return int(load().zero_embed_grad_workspace_bytes(n, hidden))


def zero_embed_grad(plan: Plan, tensor: int, hidden: int, sorted, order, dy, dy_dt: int, scale: float, dst,
                    dst_dt: int, drop: Optional[Drop] = None, rank: int = -1, accumulate: bool = False,
                    workspace=None, stream=None, n: Optional[int] = None, dy_stride: Optional[int] = None) -> None:
    """Gradient of zero_embed's table into the full flat gradient buffer dst,
    or with rank >= 0 into the compact slice that this owner receives."""
    c = _Call(stream)
    if n is None:
        if sorted is None or isinstance(sorted, int):
            raise ValueError("sorted is not a tensor: pass n")
        n = int(sorted.numel())
    s = c.flat(sorted, "sorted", 4, n)
    o = c.flat(order, "order", 4, n)
    y, ystride = c.rows(dy, "dy", _esize(dy_dt), n, hidden, dy_stride)
    d = c.flat(dst, "dst", _esize(dst_dt), plan.psi_pad if rank < 0 else plan.shard_total)
    ws, ws_bytes = c.workspace(workspace, lambda: zero_embed_grad_workspace_bytes(n, hidden))
    keep = c.drop(drop)
    c.issue(load().zero_embed_grad, plan.handle, tensor, hidden, s, o, n, y, dy_dt, ystride, scale, keep, d,
            dst_dt, rank, 1 if accumulate else 0, ws, ws_bytes)


def zero_dropout(x, residual, out, dt: int, drop: Drop, stream=None, n: Optional[int] = None) -> None:
    """out = residual + dropout(x) (residual may be None; out may be x or the
    residual).  The backward pass is the same call on the gradient."""
    c = _Call(stream)
    if n is None:
        if x is None or isinstance(x, int):
            raise ValueError("x is not a tensor: pass n")
        n = int(x.numel())
    es = _esize(dt)
    xa = c.flat(x, "x", es, n)
    ra = c.flat(residual, "residual", es, n, optional=True)
    oa = c.flat(out, "out", es, n)
    keep = c.drop(drop)
    c.issue(load().zero_dropout, xa, ra, oa, n, dt, keep)


def zero_token_logp_workspace_bytes(n: int, vocab: int) -> int:
    return int(load().zero_token_logp_workspace_bytes(n, vocab))


def _vocab(logits, vocab: Optional[int]) -> int:
    if vocab is not None:
        return int(vocab)
    if logits is None or isinstance(logits, int):
        raise ValueError("logits is not a tensor: pass vocab")
    return int(logits.shape[-1])


def zero_token_logp(logits, dt: int, labels, logp, stats, workspace=None, stream=None, n: Optional[int] = None,
                    vocab: Optional[int] = None, stride: Optional[int] = None,
                    label_it: Optional[int] = None) -> None:
    """logp[t] = log softmax(logits[t])[labels[t]]; stats[2 t], stats[2 t + 1]
    are the row's maximum and the log of its sum relative to it.  Rows whose
    label lies outside the vocabulary are not scored (0)."""
    c = _Call(stream)
    v = _vocab(logits, vocab)
    lab, it, n = c.ids(labels, "labels", n, label_it)
    x, xstride = c.rows(logits, "logits", _esize(dt), n, v, stride)
    lp = c.flat(logp, "logp", 4, n)
    st = c.flat(stats, "stats", 4, 2 * n)
    ws, ws_bytes = c.workspace(workspace, lambda: zero_token_logp_workspace_bytes(n, v))
    c.issue(load().zero_token_logp, x, dt, n, v, xstride, lab, it, lp, st, ws, ws_bytes)


def zero_preference_loss(offsets, labels, vocab: int, logp, ref_logp, beta: float, smoothing: float,
                         grad_scale: float, loss, pair_loss, rewards, coef, stream=None,
                         n_pairs: Optional[int] = None, n: Optional[int] = None,
                         offset_it: Optional[int] = None, label_it: Optional[int] = None) -> None:
    """Paired preference loss of the sequences that offsets bounds (the chosen
    ones, then the rejected ones), and coef[t] = grad_scale * dloss/dlogp[t]."""
    c = _Call(stream)
    off, oit, n_off = c.ids(offsets, "offsets", None if n_pairs is None else 2 * n_pairs + 1, offset_it)
    if n_off % 2 == 0:
        raise ValueError(f"offsets holds {n_off} entries, expected 2 * n_pairs + 1")
    pairs = n_off // 2
    if n is None:
        if logp is None or isinstance(logp, int):
            raise ValueError("logp is not a tensor: pass n")
        n = int(logp.numel())
    if labels is None:
        lab, lit = 0, ZERO_I64
    else:
        lab, lit, _ = c.ids(labels, "labels", n, label_it)
    lp = c.flat(logp, "logp", 4, n)
    ref = c.flat(ref_logp, "ref_logp", 4, n, optional=True)
    lo = c.flat(loss, "loss", 4, 1)
    pl = c.flat(pair_loss, "pair_loss", 4, pairs)
    rw = c.flat(rewards, "rewards", 4, 2 * pairs)
    co = c.flat(coef, "coef", 4, n)
    c.issue(load().zero_preference_loss, pairs, off, oit, n, lab, lit, vocab, lp, ref, beta, smoothing, grad_scale, lo,
            pl, rw, co)


def zero_token_logp_grad(logits, dt: int, labels, stats, coef, dlogits, stream=None, n: Optional[int] = None,
                         vocab: Optional[int] = None, stride: Optional[int] = None,
                         dl_stride: Optional[int] = None, label_it: Optional[int] = None) -> None:
    """dlogits[t] = coef[t] * (onehot(labels[t]) - softmax(logits[t])); rows
    that are not scored are zero.  dlogits may be the logits themselves."""
    c = _Call(stream)
    v = _vocab(logits, vocab)
    lab, it, n = c.ids(labels, "labels", n, label_it)
    es = _esize(dt)
    x, xstride = c.rows(logits, "logits", es, n, v, stride)
    st = c.flat(stats, "stats", 4, 2 * n)
    co = c.flat(coef, "coef", 4, n)
    d, dstride = c.rows(dlogits, "dlogits", es, n, v, dl_stride)
    c.issue(load().zero_token_logp_grad, x, dt, n, v, xstride, lab, it, st, co, d, dstride)
