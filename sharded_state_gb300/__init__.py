"""Python binding of libshardstate (the GB300 sharded-state step, C ABI in
include/shardstate.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions keep the C names.  Tensors are passed as torch tensors (or
raw integer device addresses); torch supplies device memory and streams.

The library must have been built (``python sharded_state_gb300/build.py`` or
``__graft_entry__.build()``); importing this package raises if it is missing,
and there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libshardstate.so")

SS_OK = 0
SS_EINVAL = -1
SS_EALIGN = -2
SS_EOVERFLOW = -3
SS_ENOMEM = -4
SS_ECUDA = -5
SS_ENODEVICE = -6
SS_ESCRATCH = -7
SS_DDP_NOALLOC_TABLE_BYTES = 256 * 1024
SS_NORM_WORKSPACE_BYTES = 4 * 1024 * 1024

SS_FLAT_ORIG_FALSE = 0
SS_FLAT_ORIG_TRUE = 1
SS_PER_PARAM_DIM0 = 2
SS_PLAN_HOST_ONLY = 1
SS_LOSS_MEAN = 0
SS_LOSS_SUM = 1
SS_CE_GRADIENT = 1
SS_CE_STAGE_WEIGHT = 2
SS_MXFP4 = 0
SS_MXFP8 = 1
SS_MAX_WORLD = 64
SS_MAX_REPLICAS = 64

# every symbol include/shardstate.h declares
EXPORTED = ("fsdp_plan_create", "fsdp_plan_layout", "fsdp_plan_info", "fsdp_plan_param_offset",
            "fsdp_plan_group", "fsdp_plan_destroy", "fsdp_pack", "fsdp_init_master",
            "fsdp_reduce_scatter_adamw", "fsdp_all_gather_unpack", "ddp_bucket_pack_average",
            "ddp_bucket_assign", "ss_strerror", "ss_last_cuda_error", "ss_version",
            "ss_launch_count", "ddp_bucket_pack_average_noalloc", "fsdp_sharded_step",
            "fsdp_reduce_scatter_accumulate", "fsdp_plan_validate", "ss_grad_norm", "ss_clip_grads",
            "fsdp_reduce_scatter_norm", "fsdp_clip_adamw", "ss_linear_ce_workspace",
            "ss_linear_cross_entropy", "ss_linear_ce_expire_wait", "ss_dropout", "ss_rms_norm",
            "ss_rms_norm_workspace", "ss_rms_norm_backward", "ss_mx_bytes", "ss_mx_quantize", "ss_mx_dequantize",
            "ss_mx_matmul", "ss_mx_expire_wait")


class ShardStateError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({detail})")


class _PlanDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("world_size", ctypes.c_int), ("elem_bytes", ctypes.c_int),
                ("num_params", ctypes.c_int), ("dim0", ctypes.POINTER(ctypes.c_int64)),
                ("inner", ctypes.POINTER(ctypes.c_int64)), ("num_groups", ctypes.c_int),
                ("group_num_params", ctypes.POINTER(ctypes.c_int)), ("flags", ctypes.c_uint)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("shard_numel", ctypes.c_int64), ("total_numel", ctypes.c_int64),
                ("unpadded_numel", ctypes.c_int64), ("pad_numel", ctypes.c_int64),
                ("world_size", ctypes.c_int), ("elem_bytes", ctypes.c_int),
                ("num_params", ctypes.c_int), ("num_groups", ctypes.c_int), ("kind", ctypes.c_int),
                ("has_device_metadata", ctypes.c_int)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class AdamW(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64)]


class _Step(ctypes.Structure):
    _fields_ = [("rank_grads", ctypes.c_void_p), ("rank_param_grads", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("param_shards", ctypes.c_void_p),
                ("hp", ctypes.POINTER(AdamW)), ("reduced_grad_out", ctypes.c_void_p),
                ("params_out", ctypes.c_void_p), ("n_out", ctypes.c_int)]


class _LinearCE(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden_size", ctypes.c_int64),
                ("vocab_size", ctypes.c_int64), ("hidden", ctypes.c_void_p),
                ("hidden_stride", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("weight_stride", ctypes.c_int64), ("targets", ctypes.c_void_p),
                ("ignore_index", ctypes.c_int64), ("reduction", ctypes.c_int),
                ("grad_scale", ctypes.c_double), ("loss_out", ctypes.c_void_p),
                ("token_loss_out", ctypes.c_void_p), ("d_hidden", ctypes.c_void_p),
                ("d_hidden_stride", ctypes.c_int64), ("d_weight", ctypes.c_void_p),
                ("d_weight_stride", ctypes.c_int64), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


# The argument blocks of the calls that a small model makes many times a step are packed
# (a quarter of a ctypes structure's time): ss_norm, ss_norm_grad, ss_mx_quant and
# ss_mx_product as the C ABI lays them out, NULL as 0.
_NORM = struct.Struct("@qqiPqPqPddPPqPqPPP")
_NORM_GRAD = struct.Struct("@qqiPqPqPPPqdPPqPqPPN")
_MX_QUANT = struct.Struct("@qqiPqiPPPPP")
_MX_PRODUCT = struct.Struct("@qqqiPPPPPqi0q")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python sharded_state_gb300/build.py` "
                          "(nvcc, sm_103a); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    i64p = ctypes.POINTER(ctypes.c_int64)
    vpp = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "fsdp_plan_create": ([ctypes.POINTER(_PlanDesc), ctypes.POINTER(vp)], i32),
        "fsdp_plan_layout": ([i32, i32, i32, i32, i64p, i64p, ctypes.POINTER(vp)], i32),
        "fsdp_plan_info": ([vp, ctypes.POINTER(PlanInfo)], i32),
        "fsdp_plan_param_offset": ([vp, i32, i64p, i64p], i32),
        "fsdp_plan_group": ([vp, i32, i64p, i64p, ctypes.POINTER(i32), ctypes.POINTER(i32)], i32),
        "fsdp_plan_destroy": ([vp], None),
        "fsdp_plan_validate": ([vp], i32),
        "fsdp_pack": ([vp, vpp, vp, i32, vp], i32),
        "fsdp_init_master": ([vp, vp, vp, vp, vp, i32, vp], i32),
        "fsdp_reduce_scatter_adamw": ([vp, vpp, vp, vp, vp, vp, ctypes.POINTER(AdamW), vp, i32, vp],
                                      i32),
        "fsdp_all_gather_unpack": ([vp, vp, vpp, i32, i32, vp], i32),
        "ddp_bucket_pack_average": ([i32, i32, i64p, vpp, ctypes.c_size_t, vpp,
                                     ctypes.POINTER(i32), vp], i32),
        "ddp_bucket_pack_average_noalloc": ([i32, i32, i64p, vpp, ctypes.c_size_t, vpp,
                                             ctypes.POINTER(i32), vp], i32),
        "ddp_bucket_assign": ([i32, i64p, i32, ctypes.c_size_t, ctypes.POINTER(i32)], i32),
        "fsdp_sharded_step": ([vp, ctypes.POINTER(_Step), i32, vp], i32),
        "fsdp_reduce_scatter_accumulate": ([vp, vpp, vp, i32, i32, vp, vp, vp, vp,
                                            ctypes.POINTER(AdamW), vp, i32, vp], i32),
        "ss_grad_norm": ([i32, i64p, ctypes.POINTER(i32), vpp, vp, vp, ctypes.c_size_t, vp], i32),
        "ss_clip_grads": ([i32, i64p, ctypes.POINTER(i32), vpp, vpp, ctypes.c_double, vp, vp,
                           ctypes.c_size_t, vp], i32),
        "fsdp_reduce_scatter_norm": ([vp, vpp, vp, vp, vp, ctypes.c_size_t, i32, vp], i32),
        "fsdp_clip_adamw": ([vp, vp, vp, i32, ctypes.c_double, vp, vp, vp, vp, ctypes.POINTER(AdamW),
                             vp, i32, vp], i32),
        "ss_linear_ce_workspace": ([i64, i64, i64, ctypes.c_uint, ctypes.POINTER(ctypes.c_size_t)], i32),
        "ss_linear_cross_entropy": ([ctypes.POINTER(_LinearCE), vp], i32),
        "ss_linear_ce_expire_wait": ([i32], i32),
        "ss_dropout": ([i64, i64, i32, vp, i64, vp, i64, ctypes.c_double, vp, vp], i32),
        "ss_rms_norm": ([ctypes.c_char_p, vp], i32),
        "ss_rms_norm_workspace": ([i64, i64, ctypes.POINTER(ctypes.c_size_t)], i32),
        "ss_rms_norm_backward": ([ctypes.c_char_p, vp], i32),
        "ss_mx_bytes": ([i64, i64, i32, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)], i32),
        "ss_mx_quantize": ([ctypes.c_char_p, vp], i32),
        "ss_mx_dequantize": ([i64, i64, i32, vp, vp, vp, i64, i32, vp], i32),
        "ss_mx_matmul": ([ctypes.c_char_p, vp], i32),
        "ss_mx_expire_wait": ([i32], i32),
        "ss_strerror": ([i32], ctypes.c_char_p),
        "ss_last_cuda_error": ([], i32),
        "ss_version": ([], ctypes.c_char_p),
        "ss_launch_count": ([], ctypes.c_uint64),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def ss_strerror(status: int) -> str:
    return _lib.ss_strerror(status).decode()


def ss_last_cuda_error() -> int:
    return int(_lib.ss_last_cuda_error())


def ss_version() -> str:
    return _lib.ss_version().decode()


def ss_launch_count() -> int:
    return int(_lib.ss_launch_count())


def _check(fn: str, status: int) -> None:
    if status != SS_OK:
        detail = ss_strerror(status)
        if status == SS_ECUDA:
            detail += f", cudaError {ss_last_cuda_error()}"
        raise ShardStateError(fn, status, detail)


def _addr(x) -> Optional[int]:
    """Device address of a tensor (or an int / None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def ptr_array(xs: Sequence) -> ctypes.Array:
    """A host array of device pointers, built once and reusable across calls
    (every call that takes a list of tensors also accepts one of these)."""
    return _ptr_array(xs)


def _ptr_array(xs: Sequence) -> ctypes.Array:
    if isinstance(xs, ctypes.Array):
        return xs
    arr = (ctypes.c_void_p * max(1, len(xs)))()
    for k, x in enumerate(xs):
        arr[k] = _addr(x)
    return arr


def _current_stream() -> int:
    """The current stream's handle.  torch's own accessor of the raw handle, where it
    has one, costs a sixth of building a Stream object (0.5 against 2.9 us on a Grace
    core), which shows beside launches of a few microseconds."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if raw is None or device is None:
            return int(torch.cuda.current_stream().cuda_stream)
        torch.cuda.init()
        _raw_stream = lambda: raw(device())
    return _raw_stream()


_raw_stream = None


def _i64_array(xs: Sequence[int]):
    arr = (ctypes.c_int64 * max(1, len(xs)))()
    for k, x in enumerate(xs):
        arr[k] = int(x)
    return arr


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------

class Plan:
    """Owns an ss_plan*; destroyed with the object (or explicitly via destroy())."""

    def __init__(self, handle: int):
        self.handle = handle

    @property
    def _as_parameter_(self):
        return ctypes.c_void_p(self.handle)

    def info(self) -> PlanInfo:
        return fsdp_plan_info(self)

    def destroy(self) -> None:
        if self.handle:
            _lib.fsdp_plan_destroy(ctypes.c_void_p(self.handle))
            self.handle = 0

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def fsdp_plan_create(kind: int, world_size: int, elem_bytes: int, dim0: Sequence[int],
                     inner: Optional[Sequence[int]] = None,
                     group_num_params: Optional[Sequence[int]] = None,
                     host_only: bool = False) -> Plan:
    n = len(dim0)
    d0 = _i64_array(dim0)
    inn = _i64_array(inner) if inner is not None else None
    groups = None
    if group_num_params is not None:
        groups = (ctypes.c_int * max(1, len(group_num_params)))(*group_num_params)
    desc = _PlanDesc(kind, world_size, elem_bytes, n,
                     ctypes.cast(d0, ctypes.POINTER(ctypes.c_int64)),
                     ctypes.cast(inn, ctypes.POINTER(ctypes.c_int64)) if inn is not None else None,
                     len(group_num_params) if group_num_params is not None else 0,
                     ctypes.cast(groups, ctypes.POINTER(ctypes.c_int)) if groups is not None else None,
                     SS_PLAN_HOST_ONLY if host_only else 0)
    out = ctypes.c_void_p()
    _check("fsdp_plan_create", _lib.fsdp_plan_create(ctypes.byref(desc), ctypes.byref(out)))
    return Plan(out.value)


def fsdp_plan_layout(kind: int, world_size: int, elem_bytes: int, dim0: Sequence[int],
                     inner: Optional[Sequence[int]] = None) -> Plan:
    d0 = _i64_array(dim0)
    inn = _i64_array(inner) if inner is not None else None
    out = ctypes.c_void_p()
    _check("fsdp_plan_layout", _lib.fsdp_plan_layout(
        kind, world_size, elem_bytes, len(dim0), ctypes.cast(d0, ctypes.POINTER(ctypes.c_int64)),
        ctypes.cast(inn, ctypes.POINTER(ctypes.c_int64)) if inn is not None else None,
        ctypes.byref(out)))
    return Plan(out.value)


def fsdp_plan_info(plan: Plan) -> PlanInfo:
    info = PlanInfo()
    _check("fsdp_plan_info", _lib.fsdp_plan_info(plan, ctypes.byref(info)))
    return info


def fsdp_plan_param_offset(plan: Plan, param: int):
    off = ctypes.c_int64()
    rows = ctypes.c_int64()
    _check("fsdp_plan_param_offset",
           _lib.fsdp_plan_param_offset(plan, param, ctypes.byref(off), ctypes.byref(rows)))
    return off.value, rows.value


def fsdp_plan_group(plan: Plan, group: int):
    base, shard = ctypes.c_int64(), ctypes.c_int64()
    first, count = ctypes.c_int(), ctypes.c_int()
    _check("fsdp_plan_group", _lib.fsdp_plan_group(plan, group, ctypes.byref(base),
                                                   ctypes.byref(shard), ctypes.byref(first),
                                                   ctypes.byref(count)))
    return {"base": base.value, "shard_numel": shard.value, "first_param": first.value,
            "num_params": count.value}


def fsdp_plan_validate(plan: Plan) -> None:
    _check("fsdp_plan_validate", _lib.fsdp_plan_validate(plan))


def fsdp_plan_destroy(plan: Plan) -> None:
    plan.destroy()


# ---------------------------------------------------------------------------
# step
# ---------------------------------------------------------------------------

def fsdp_pack(plan: Plan, params: Sequence, packed, group: int = -1, stream=None) -> None:
    _check("fsdp_pack", _lib.fsdp_pack(plan, _ptr_array(params), _addr(packed), group,
                                       _stream(stream)))


def fsdp_init_master(plan: Plan, param_shards, master, exp_avg, exp_avg_sq, group: int = -1,
                     stream=None) -> None:
    _check("fsdp_init_master", _lib.fsdp_init_master(plan, _addr(param_shards), _addr(master),
                                                     _addr(exp_avg), _addr(exp_avg_sq), group,
                                                     _stream(stream)))


def adamw_params(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1) -> AdamW:
    return AdamW(lr, beta1, beta2, eps, weight_decay, step)


def fsdp_reduce_scatter_adamw(plan: Plan, rank_grads: Sequence, master, exp_avg, exp_avg_sq,
                              param_shards, hp: Optional[AdamW], reduced_grad_out=None,
                              group: int = -1, stream=None) -> None:
    _check("fsdp_reduce_scatter_adamw", _lib.fsdp_reduce_scatter_adamw(
        plan, _ptr_array(rank_grads), _addr(master), _addr(exp_avg), _addr(exp_avg_sq),
        _addr(param_shards), ctypes.byref(hp) if hp is not None else None, _addr(reduced_grad_out),
        group, _stream(stream)))


def fsdp_reduce_scatter_accumulate(plan: Plan, rank_grads: Sequence, accum, micro_step: int,
                                   num_micro: int, master=None, exp_avg=None, exp_avg_sq=None,
                                   param_shards=None, hp: Optional[AdamW] = None,
                                   reduced_grad_out=None, group: int = -1, stream=None) -> None:
    """Micro-batch `micro_step` of `num_micro`: accumulate the reduce-scatter in
    fp32, and on the last micro-batch run AdamW on the micro-batch mean."""
    _check("fsdp_reduce_scatter_accumulate", _lib.fsdp_reduce_scatter_accumulate(
        plan, _ptr_array(rank_grads), _addr(accum), micro_step, num_micro, _addr(master),
        _addr(exp_avg), _addr(exp_avg_sq), _addr(param_shards),
        ctypes.byref(hp) if hp is not None else None, _addr(reduced_grad_out), group,
        _stream(stream)))


def fsdp_all_gather_unpack(plan: Plan, param_shards, params_out: Sequence, n_out: int = 1,
                           group: int = -1, stream=None) -> None:
    """params_out: n_out * num_params tensors, replica-major."""
    _check("fsdp_all_gather_unpack", _lib.fsdp_all_gather_unpack(
        plan, _addr(param_shards), _ptr_array(params_out), n_out, group, _stream(stream)))


def fsdp_sharded_step(plan: Plan, master, exp_avg, exp_avg_sq, param_shards, hp: AdamW,
                      rank_grads: Optional[Sequence] = None,
                      rank_param_grads: Optional[Sequence] = None, params_out=None,
                      n_out: int = 0, reduced_grad_out=None, group: int = -1,
                      stream=None) -> None:
    """One-pass step: gradients from N packed buffers (rank_grads) or from N
    per-parameter gradient sets (rank_param_grads, rank-major: rank r's
    gradient of parameter i at r*num_params + i), reduce-scatter + AdamW, and
    optionally the n_out per-parameter outputs (replica-major)."""
    keep = []
    def arr(xs):
        if xs is None:
            return None
        a = _ptr_array(xs)
        keep.append(a)
        return ctypes.cast(a, ctypes.c_void_p)
    st = _Step(arr(rank_grads), arr(rank_param_grads), _addr(master), _addr(exp_avg),
               _addr(exp_avg_sq), _addr(param_shards), ctypes.pointer(hp), _addr(reduced_grad_out),
               arr(params_out) if n_out > 0 else None, n_out)
    _check("fsdp_sharded_step", _lib.fsdp_sharded_step(plan, ctypes.byref(st), group,
                                                       _stream(stream)))


class ShardedStep:
    """fsdp_sharded_step with every argument marshalled once, for loops whose
    steps are short enough that building the call each time shows: a call
    sets the AdamW step number (the other hyper-parameters are the ones given
    here) and runs the step on `stream`, an int handle (0: the legacy default
    stream) fixed here.  Keeps the pointer arrays alive; the tensors must stay
    alive and in place as long as the object is used."""

    def __init__(self, plan: Plan, master, exp_avg, exp_avg_sq, param_shards, hp: AdamW,
                 rank_grads: Optional[Sequence] = None,
                 rank_param_grads: Optional[Sequence] = None, params_out=None, n_out: int = 0,
                 reduced_grad_out=None, group: int = -1, stream=None):
        self._plan = plan  # keeps the plan alive
        self._pp = ctypes.c_void_p(plan.handle)
        self._hp = AdamW(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.step)
        self._keep = []

        def arr(xs):
            if xs is None:
                return None
            a = _ptr_array(xs)
            self._keep.append(a)
            return ctypes.cast(a, ctypes.c_void_p)
        self._st = _Step(arr(rank_grads), arr(rank_param_grads), _addr(master), _addr(exp_avg),
                         _addr(exp_avg_sq), _addr(param_shards), ctypes.pointer(self._hp),
                         _addr(reduced_grad_out), arr(params_out) if n_out > 0 else None, n_out)
        self._ref = ctypes.byref(self._st)
        self._group = group
        self._stream = _stream(stream)
        self._fn = _lib.fsdp_sharded_step

    def __call__(self, step: int) -> None:
        self._hp.step = step
        status = self._fn(self._pp, self._ref, self._group, self._stream)
        if status != SS_OK:
            _check("fsdp_sharded_step", status)


def ddp_bucket_pack_average(rank_grads: Sequence[Sequence], bucket_cap_bytes: int,
                            avg_out: Sequence, numels: Optional[Sequence[int]] = None,
                            stream=None) -> int:
    """rank_grads[r][t]: rank r's gradient of tensor t. Returns the bucket count."""
    N = len(rank_grads)
    T = len(avg_out)
    if numels is None:
        numels = [int(t.numel()) for t in avg_out]
    flat = [g for rank in rank_grads for g in rank]
    nb = ctypes.c_int()
    _check("ddp_bucket_pack_average", _lib.ddp_bucket_pack_average(
        N, T, _i64_array(numels), _ptr_array(flat), bucket_cap_bytes, _ptr_array(avg_out),
        ctypes.byref(nb), _stream(stream)))
    return nb.value


def ddp_bucket_pack_average_noalloc(rank_grads: Sequence[Sequence], bucket_cap_bytes: int,
                                    avg_out: Sequence, numels: Optional[Sequence[int]] = None,
                                    stream=None) -> int:
    """Same as ddp_bucket_pack_average, for callers that cannot allocate device
    memory: the library's fixed device array holds the per-call table (at most
    SS_DDP_NOALLOC_TABLE_BYTES; larger requests raise with SS_ESCRATCH).  Calls
    share that array, so calls that could overlap on the GPU must be ordered by
    the caller.  Returns the bucket count."""
    N = len(rank_grads)
    T = len(avg_out)
    if numels is None:
        numels = [int(t.numel()) for t in avg_out]
    flat = [g for rank in rank_grads for g in rank]
    nb = ctypes.c_int()
    _check("ddp_bucket_pack_average_noalloc", _lib.ddp_bucket_pack_average_noalloc(
        N, T, _i64_array(numels), _ptr_array(flat), bucket_cap_bytes, _ptr_array(avg_out),
        ctypes.byref(nb), _stream(stream)))
    return nb.value


def ddp_bucket_assign(numels: Sequence[int], elem_bytes: int, bucket_cap_bytes: int):
    T = len(numels)
    out = (ctypes.c_int * max(1, T))()
    nb = _lib.ddp_bucket_assign(T, _i64_array(numels), elem_bytes, bucket_cap_bytes, out)
    if nb < 0:
        _check("ddp_bucket_assign", nb)
    return [int(out[t]) for t in range(T)], int(nb)


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------

def _want(fn: str, t, dtype: str, what: str, numel: int = 0) -> int:
    """Address of a tensor whose place, type and size the C ABI cannot check."""
    if not t.is_cuda or t.dtype != _dtype(dtype) or not t.is_contiguous() or t.numel() < numel:
        raise ShardStateError(fn, SS_EINVAL, f"{what}: contiguous {dtype} on the GPU, at least {numel} elements")
    return t.data_ptr()


def _workspace(fn: str, t):
    """Address and bytes of a workspace tensor of any type."""
    if not t.is_cuda or not t.is_contiguous():
        raise ShardStateError(fn, SS_EINVAL, "workspace: a contiguous tensor on the GPU")
    return t.data_ptr(), t.nbytes


_dtypes = {}


def _dtype(name: str):
    if name not in _dtypes:
        import torch
        _dtypes[name] = getattr(torch, name)
    return _dtypes[name]


def _grad_list(fn: str, grads: Sequence, out: Optional[Sequence]):
    """numels, element sizes and pointers of a list of contiguous bf16 / fp32 tensors."""
    kinds = (_dtype("bfloat16"), _dtype("float32"))
    for k, g in enumerate(grads):
        if not g.is_cuda or g.dtype not in kinds or not g.is_contiguous():
            raise ShardStateError(fn, SS_EINVAL, f"tensor {k}: contiguous bf16 or fp32 on the GPU is wanted")
    if out is not None:
        if len(out) != len(grads):
            raise ShardStateError(fn, SS_EINVAL, "out: one tensor for each gradient is wanted")
        for k, (g, o) in enumerate(zip(grads, out)):
            if not o.is_cuda or o.dtype != g.dtype or o.numel() != g.numel() or not o.is_contiguous():
                raise ShardStateError(fn, SS_EINVAL, f"out {k}: its gradient's type and size are wanted")
    eb = (ctypes.c_int * max(1, len(grads)))(*[g.element_size() for g in grads])
    return (len(grads), _i64_array([g.numel() for g in grads]), eb, _ptr_array(grads),
            _ptr_array(out) if out is not None else None)


def ss_grad_norm(grads: Sequence, norm_out, workspace, stream=None) -> None:
    """norm_out (2 floats on the device) = {global norm of the tensors, 1}."""
    fn = "ss_grad_norm"
    norm = _want(fn, norm_out, "float32", "norm_out", 2)
    ws, nbytes = _workspace(fn, workspace)
    n, numels, eb, ptrs, _ = _grad_list(fn, grads, None)
    _check(fn, _lib.ss_grad_norm(n, numels, eb, ptrs, norm, ws, nbytes, _stream(stream)))


def ss_clip_grads(grads: Sequence, max_norm: float, norm_out, workspace, out: Optional[Sequence] = None,
                  stream=None) -> None:
    """Scale the tensors (into `out`, or in place) by min(1, max_norm / (norm + 1e-6));
    norm_out = {global norm, that factor}."""
    GradClip(grads, max_norm, norm_out, workspace, out=out, stream=_stream(stream))()


class GradClip:
    """ss_clip_grads with every argument marshalled once, for a loop whose
    gradients stay in place; called with nothing, it clips on `stream` (by
    default the stream that is current at the call).  The tensors must stay
    alive as long as the object is used."""

    def __init__(self, grads: Sequence, max_norm: float, norm_out, workspace,
                 out: Optional[Sequence] = None, stream=None):
        fn = "ss_clip_grads"
        norm = _want(fn, norm_out, "float32", "norm_out", 2)
        ws, nbytes = _workspace(fn, workspace)
        n, numels, eb, ptrs, outs = _grad_list(fn, grads, out)
        self._args = (n, numels, eb, ptrs, outs, ctypes.c_double(max_norm), ctypes.c_void_p(norm),
                      ctypes.c_void_p(ws), ctypes.c_size_t(nbytes))
        self._keep = (norm_out, workspace)
        self._stream = None if stream is None else _stream(stream)
        self._fn = _lib.ss_clip_grads

    def __call__(self) -> None:
        stream = _stream(None) if self._stream is None else self._stream
        status = self._fn(*self._args, stream)
        if status != SS_OK:
            _check("ss_clip_grads", status)


def fsdp_reduce_scatter_norm(plan: Plan, rank_grads: Sequence, reduced_grad, sq_out, workspace,
                             group: int = -1, stream=None) -> None:
    """reduced_grad = the ranks' mean; sq_out (1 fp64 element) = its sum of squares."""
    fn = "fsdp_reduce_scatter_norm"
    sq = _want(fn, sq_out, "float64", "sq_out", 1)
    ws, nbytes = _workspace(fn, workspace)
    _check(fn, _lib.fsdp_reduce_scatter_norm(plan, _ptr_array(rank_grads), _addr(reduced_grad), sq, ws, nbytes,
                                             group, _stream(stream)))


def fsdp_clip_adamw(plan: Plan, reduced_grad, sq_sums, max_norm: float, master, exp_avg, exp_avg_sq,
                    param_shards, hp: AdamW, norm_out, group: int = -1, stream=None) -> None:
    """AdamW on reduced_grad scaled by min(1, max_norm / (norm + 1e-6)), the norm
    being the root of the sum of sq_sums (fp64, one element per
    fsdp_reduce_scatter_norm call the norm spans); norm_out = {norm, factor}."""
    fn = "fsdp_clip_adamw"
    sq = _want(fn, sq_sums, "float64", "sq_sums", 1)
    norm = _want(fn, norm_out, "float32", "norm_out", 2)
    _check(fn, _lib.fsdp_clip_adamw(plan, _addr(reduced_grad), sq, sq_sums.numel(), max_norm, _addr(master),
                                    _addr(exp_avg), _addr(exp_avg_sq), _addr(param_shards), ctypes.byref(hp), norm,
                                    group, _stream(stream)))


# ---------------------------------------------------------------------------
# the loss at the head of the model
# ---------------------------------------------------------------------------

def ss_linear_ce_workspace(num_tokens: int, hidden_size: int, vocab_size: int, gradient: bool,
                           stage_weight: bool = False) -> int:
    """Bytes of workspace ss_linear_cross_entropy takes: with `gradient`, to write
    d_hidden or d_weight; with `stage_weight`, for a weight whose rows do not
    start on 16-byte boundaries (assumed when hidden_size % 8 != 0)."""
    out = ctypes.c_size_t()
    flags = (SS_CE_GRADIENT if gradient else 0) | (SS_CE_STAGE_WEIGHT if stage_weight else 0)
    _check("ss_linear_ce_workspace", _lib.ss_linear_ce_workspace(num_tokens, hidden_size, vocab_size, flags,
                                                                 ctypes.byref(out)))
    return out.value


def _matrix(fn: str, t, what: str, rows: int, cols: int):
    """Address and row stride of a bf16 matrix (NULL, 0 for None)."""
    if t is None:
        return None, 0
    if not t.is_cuda or t.dtype != _dtype("bfloat16") or t.shape != (rows, cols) or (cols > 1 and t.stride(1) != 1):
        raise ShardStateError(fn, SS_EINVAL,
                              f"{what}: bf16 [{rows}, {cols}] on the GPU with unit column stride is wanted")
    stride = t.stride(0)
    return t.data_ptr(), stride if rows > 1 or stride > cols else cols


def ss_linear_ce_expire_wait(launch: int) -> None:
    """Diagnostics: a wait of the next ss_linear_cross_entropy call runs out, in its tensor-core
    launch number `launch` (0: the statistics, from 1 on the gradients; -1: none)."""
    _check("ss_linear_ce_expire_wait", _lib.ss_linear_ce_expire_wait(launch))


def ss_linear_cross_entropy(hidden, weight, targets, loss_out, workspace, token_loss_out=None, d_hidden=None,
                            d_weight=None, ignore_index: int = -100, reduction: str = "mean",
                            grad_scale: float = 1.0, stream=None) -> None:
    """Cross entropy of softmax(hidden @ weight.T) against targets, with no logits
    kept: hidden [T, D] and weight [V, D] bf16 (rows may be strided), targets [T]
    int64 -> loss_out (1 float; "mean" or "sum" over the targets that are not
    ignore_index), token_loss_out [T], and grad_scale times the gradients in
    d_hidden [T, D] and d_weight [V, D]; the last three are optional."""
    fn = "ss_linear_cross_entropy"
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ShardStateError(fn, SS_EINVAL, "hidden and weight: matrices are wanted")
    T, D = hidden.shape
    V = weight.shape[0]
    if reduction not in ("mean", "sum"):
        raise ShardStateError(fn, SS_EINVAL, "reduction: mean or sum")
    y = _want(fn, targets, "int64", "targets", T)
    loss = _want(fn, loss_out, "float32", "loss_out", 1)
    ws, nbytes = _workspace(fn, workspace)
    token_loss = None if token_loss_out is None else _want(fn, token_loss_out, "float32", "token_loss_out", T)
    h, ldh = _matrix(fn, hidden, "hidden", T, D)
    w, ldw = _matrix(fn, weight, "weight", V, D)
    dh, ld_dh = _matrix(fn, d_hidden, "d_hidden", T, D)
    dw, ld_dw = _matrix(fn, d_weight, "d_weight", V, D)
    args = _LinearCE(T, D, V, h, ldh, w, ldw, y, ignore_index,
                     SS_LOSS_MEAN if reduction == "mean" else SS_LOSS_SUM, grad_scale, loss, token_loss, dh, ld_dh, dw,
                     ld_dw, ws, nbytes)
    _check(fn, _lib.ss_linear_cross_entropy(ctypes.byref(args), _stream(stream)))


# ---------------------------------------------------------------------------
# the residual stream between two layers
# ---------------------------------------------------------------------------

def _device() -> int:
    """The current device, by torch's own accessor where it has one (see _current_stream)."""
    global _get_device
    if _get_device is None:
        import torch
        torch.cuda.current_device()  # initialises CUDA
        _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _get_device()


_get_device = None


def _row_dtype(fn: str, t, what: str):
    """The type and shape of the bf16 or fp32 matrix that gives a call its sizes."""
    dtype, shape = t.dtype, t.shape
    if len(shape) != 2 or (dtype is not _dtype("bfloat16") and dtype is not _dtype("float32")):
        raise ShardStateError(fn, SS_EINVAL, f"{what}: a bf16 or fp32 matrix is wanted")
    return dtype, shape


def _rows(fn: str, t, what: str, shape, dtype, device: int):
    """Address and row stride of a matrix of that type on the current device (0, 0 for None)."""
    if t is None:
        return 0, 0
    if t.get_device() == device and t.dtype is dtype and t.shape == shape:
        stride, unit = t.stride()
        rows, cols = shape
        if unit == 1 or cols <= 1:
            return t.data_ptr(), stride if rows > 1 or stride > cols else cols
    raise ShardStateError(fn, SS_EINVAL, f"{what}: {dtype} {list(shape)} on the current GPU with unit column stride "
                                         "is wanted")


def _flat(fn: str, t, what: str, dtype, numel: int, device: int) -> int:
    """Address of a contiguous tensor of at least numel elements on the current device (0 for None)."""
    if t is None:
        return 0
    if t.get_device() != device or t.dtype is not dtype or t.numel() < numel or not t.is_contiguous():
        raise ShardStateError(fn, SS_EINVAL, f"{what}: contiguous {dtype} on the current GPU, at least {numel} elements")
    return t.data_ptr()


def ss_dropout(x, out, p: float, rng, stream=None) -> None:
    """out = dropout(x) with probability p (in steps of 2^-16), for bf16 or fp32
    matrices (rows may be strided; out may be x): the mask follows from rng (2 int64 on
    the device: seed, offset) and from each element's place, and the same call on a
    gradient is the backward pass."""
    fn = "ss_dropout"
    (dtype, shape), dev = _row_dtype(fn, x, "x"), _device()
    rows, cols = shape
    ax, ldx = _rows(fn, x, "x", shape, dtype, dev)
    ao, ldo = _rows(fn, out, "out", shape, dtype, dev)
    status = _lib.ss_dropout(rows, cols, dtype.itemsize, ax, ldx, ao, ldo, p,
                             _flat(fn, rng, "rng", _dtype("int64"), 2, dev), _stream(stream))
    if status != SS_OK:
        _check(fn, status)


def ss_rms_norm(x, weight, eps: float, out=None, residual=None, sum_out=None, rstd_out=None, mx_data=None,
                mx_scales=None, dropout: float = 0.0, rng=None, stream=None) -> None:
    """h = dropout(x) + residual (into sum_out), out = h * rstd * weight with
    rstd = 1 / sqrt(mean(h^2) + eps) of each row (into rstd_out [rows], fp32); x,
    residual, sum_out and out are bf16 or fp32 matrices of one type (rows may be
    strided; sum_out may be x or residual, out may be x), weight [cols] too.  mx_data
    and mx_scales get out as SS_MXFP8 (buffers of ss_mx_bytes).  At least one output is
    wanted; residual and dropout are optional."""
    fn = "ss_rms_norm"
    (dtype, shape), dev = _row_dtype(fn, x, "x"), _device()
    rows, cols = shape
    ax, ldx = _rows(fn, x, "x", shape, dtype, dev)
    ar, ldr = _rows(fn, residual, "residual", shape, dtype, dev)
    ah, ldh = _rows(fn, sum_out, "sum_out", shape, dtype, dev)
    ao, ldo = _rows(fn, out, "out", shape, dtype, dev)
    if weight is None or weight.numel() != cols:
        raise ShardStateError(fn, SS_EINVAL, f"weight: {cols} elements are wanted")
    md, ms = _mx_buffers(fn, mx_data, mx_scales, "mx", rows, cols, SS_MXFP8, dev)
    args = _NORM.pack(rows, cols, dtype.itemsize, ax, ldx, ar, ldr, _flat(fn, weight, "weight", dtype, cols, dev), eps,
                 dropout, _flat(fn, rng, "rng", _dtype("int64"), 2, dev), ah, ldh, ao, ldo,
                 _flat(fn, rstd_out, "rstd_out", _dtype("float32"), rows, dev), md, ms)
    status = _lib.ss_rms_norm(args, _stream(stream))
    if status != SS_OK:
        _check(fn, status)


def ss_rms_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace ss_rms_norm_backward takes on the current device."""
    out = ctypes.c_size_t()
    _check("ss_rms_norm_workspace", _lib.ss_rms_norm_workspace(rows, cols, ctypes.byref(out)))
    return out.value


def ss_rms_norm_backward(d_out, h, weight, rstd, d_h, workspace, d_sum=None, d_x=None, d_weight=None,
                         dropout: float = 0.0, rng=None, stream=None) -> None:
    """Gradients of ss_rms_norm from what it left (h, its sum_out, and rstd): d_h is the
    gradient of the sum, d_sum included (the part that reaches h from elsewhere); d_x that
    of x behind the forward pass's dropout; d_weight [cols] that of the weight.  d_h (which
    may be d_out or d_sum), d_x and d_weight are optional; the workspace
    (ss_rms_norm_workspace bytes) is for d_weight."""
    fn = "ss_rms_norm_backward"
    (dtype, shape), dev = _row_dtype(fn, h, "h"), _device()
    rows, cols = shape
    ay, ldy = _rows(fn, d_out, "d_out", shape, dtype, dev)
    ah, ldh = _rows(fn, h, "h", shape, dtype, dev)
    as_, lds = _rows(fn, d_sum, "d_sum", shape, dtype, dev)
    ag, ldg = _rows(fn, d_h, "d_h", shape, dtype, dev)
    ax, ldx = _rows(fn, d_x, "d_x", shape, dtype, dev)
    for name, t in (("weight", weight), ("d_weight", d_weight)):
        if t is not None and t.numel() != cols:
            raise ShardStateError(fn, SS_EINVAL, f"{name}: {cols} elements are wanted")
    ws, nbytes = (0, 0) if workspace is None else _workspace(fn, workspace)
    args = _NORM_GRAD.pack(rows, cols, dtype.itemsize, ay, ldy, ah, ldh, _flat(fn, weight, "weight", dtype, cols, dev),
                     _flat(fn, rstd, "rstd", _dtype("float32"), rows, dev), as_, lds, dropout,
                     _flat(fn, rng, "rng", _dtype("int64"), 2, dev), ag, ldg, ax, ldx,
                     _flat(fn, d_weight, "d_weight", dtype, cols, dev), ws, nbytes)
    status = _lib.ss_rms_norm_backward(args, _stream(stream))
    if status != SS_OK:
        _check(fn, status)


# ---------------------------------------------------------------------------
# matrices in few bits
# ---------------------------------------------------------------------------

def ss_mx_bytes(rows: int, cols: int, format: int):
    """(bytes of data, bytes of scales) of a [rows, cols] matrix in SS_MXFP4 or SS_MXFP8."""
    data, scales = ctypes.c_size_t(), ctypes.c_size_t()
    _check("ss_mx_bytes", _lib.ss_mx_bytes(rows, cols, format, ctypes.byref(data), ctypes.byref(scales)))
    return data.value, scales.value


def _mx_buffers(fn: str, data, scales, what: str, rows: int, cols: int, format: int, device: int):
    """Addresses of a quantised matrix's buffers, uint8 and large enough (0, 0 for None, None)."""
    if data is None and scales is None:
        return 0, 0
    if data is None or scales is None:
        raise ShardStateError(fn, SS_EINVAL, f"{what}: data and scales are wanted together")
    wide = -(-cols // 128)
    byte = _dtype("uint8")
    return (_flat(fn, data, what + " data", byte, rows * wide * (64 if format == SS_MXFP4 else 128), device),
            _flat(fn, scales, what + " scales", byte, -(-rows // 128) * wide * 512, device))


def _mx_format(fn: str, format: int) -> None:
    if format not in (SS_MXFP4, SS_MXFP8):
        raise ShardStateError(fn, SS_EINVAL, "format: SS_MXFP4 or SS_MXFP8")


def ss_mx_quantize(x, format: int, data=None, scales=None, t_data=None, t_scales=None, rng=None, stream=None) -> None:
    """Quantise a bf16 or fp32 matrix x [R, C] (rows may be strided) to SS_MXFP4 or
    SS_MXFP8: along its rows into data and scales, along its columns (x.T, [C, R]) into
    t_data and t_scales, either or both from one read; uint8 buffers of ss_mx_bytes.  To
    the nearest, or stochastically with rng (2 int64 on the device: seed, offset); elements
    beyond the format's largest are cut to it either way."""
    fn = "ss_mx_quantize"
    (dtype, shape), dev = _row_dtype(fn, x, "x"), _device()
    _mx_format(fn, format)
    rows, cols = shape
    ax, ldx = _rows(fn, x, "x", shape, dtype, dev)
    d, s = _mx_buffers(fn, data, scales, "quantised", rows, cols, format, dev)
    td, ts = _mx_buffers(fn, t_data, t_scales, "transposed", cols, rows, format, dev)
    args = _MX_QUANT.pack(rows, cols, dtype.itemsize, ax, ldx, format, d, s, td, ts,
                    _flat(fn, rng, "rng", _dtype("int64"), 2, dev))
    status = _lib.ss_mx_quantize(args, _stream(stream))
    if status != SS_OK:
        _check(fn, status)


def ss_mx_dequantize(data, scales, format: int, out, stream=None) -> None:
    """The values of a quantised matrix into out [R, C], bf16 or fp32 (rows may be strided)."""
    fn = "ss_mx_dequantize"
    (dtype, shape), dev = _row_dtype(fn, out, "out"), _device()
    _mx_format(fn, format)
    rows, cols = shape
    ao, ldo = _rows(fn, out, "out", shape, dtype, dev)
    d, s = _mx_buffers(fn, data, scales, "quantised", rows, cols, format, dev)
    status = _lib.ss_mx_dequantize(rows, cols, format, d, s, ao, ldo, dtype.itemsize, _stream(stream))
    if status != SS_OK:
        _check(fn, status)


def ss_mx_expire_wait(on: bool) -> None:
    """Diagnostics: a wait of the next ss_mx_matmul call that launches runs out."""
    _check("ss_mx_expire_wait", _lib.ss_mx_expire_wait(int(on)))


def ss_mx_matmul(a_data, a_scales, b_data, b_scales, K: int, format: int, out, stream=None) -> None:
    """out [M, N] (bf16 or fp32, rows may be strided) = A B^T of two quantised matrices
    of one format, A [M, K] and B [N, K]: a linear layer whose weight is B, and with the
    transposes of ss_mx_quantize both of its gradients."""
    fn = "ss_mx_matmul"
    (dtype, shape), dev = _row_dtype(fn, out, "out"), _device()
    _mx_format(fn, format)
    M, N = shape
    ao, ldo = _rows(fn, out, "out", shape, dtype, dev)
    ad, as_ = _mx_buffers(fn, a_data, a_scales, "A", M, K, format, dev)
    bd, bs = _mx_buffers(fn, b_data, b_scales, "B", N, K, format, dev)
    args = _MX_PRODUCT.pack(M, N, K, format, ad, as_, bd, bs, ao, ldo, dtype.itemsize)
    status = _lib.ss_mx_matmul(args, _stream(stream))
    if status != SS_OK:
        _check(fn, status)
