"""Python binding of the B200 MuonAdamW library (ctypes over ``lib/libmuonadamw.so``).

Argument marshalling only: every step of the optimizer runs in the library's
CUDA kernels. PyTorch supplies device memory and streams. The functions keep
the C names (``ma_partition``, ``muon_step_batched``, ``adamw_step_fused``,
``muonadamw_step``, ...). A missing or unloadable library raises
``LibraryMissing``. There is no fallback of any kind.
"""
from __future__ import annotations

import array
import contextlib
import importlib.machinery
import importlib.util
import ctypes
import math
import os
import sysconfig
from typing import Sequence

__all__ = [
    "LibraryMissing", "MAError", "lib", "MuonHParams", "AdamWHParams", "Group", "Tensor",
    "MA_OK", "MA_F32", "MA_BF16", "MA_MUON", "MA_ADAMW", "ROLE_HIDDEN", "ROLE_EMBED", "ROLE_UNEMBED",
    "ROLE_FORCE_ADAMW", "ShardSlot", "ShardBucket", "SHARD_ALIGN", "ma_partition", "ma_assign_owners",
    "ma_shard_layout", "muon_workspace_bytes", "muon_step_batched",
    "muon_step_batched_noalloc", "STATIC_SCRATCH_BYTES", "ns_iterate_workspace_bytes", "ns_iterate_bf16",
    "adamw_step_fused", "ma_plan_create", "muonadamw_step", "muonadamw_step_graph", "muonadamw_step_from_host",
    "ma_plan_describe", "ma_plan_destroy", "ma_plan_status", "ma_device_status", "ma_device_status_async",
    "ma_set_wait_limit_ns", "ma_set_momentum_overlap", "ma_debug_build", "MA_ERR_BOUNDS",
    "ma_selftest_wait_timeout", "ma_profile_enable", "ma_profile_collect", "PROF_CLASSES", "group_table", "Plan",
    "MuonAdamW", "muon_hparams", "adamw_hparams", "CLIP_BYTES", "clip_buffer", "ma_grad_norm", "ma_grad_clip",
    "ma_clip_finalize", "ma_plan_set_clip", "GradClip", "MA_I32", "MA_I64", "embedding_lookup",
    "embed_grad_workspace_bytes", "embedding_grad", "embedding", "qk_max_logit", "qk_clip",
]

HERE = os.path.dirname(os.path.abspath(__file__))
# The release library, or (MA_LIBRARY=debug) the build with guarded device
# indexing, lib/libmuonadamw_debug.so; both are compiled by build.py.
LIB_PATH = os.path.join(HERE, "lib", "libmuonadamw_debug.so" if os.environ.get("MA_LIBRARY") == "debug"
                        else "libmuonadamw.so")

MA_OK, MA_ERR_NULL, MA_ERR_SHAPE, MA_ERR_DTYPE, MA_ERR_ALIGN, MA_ERR_WORKSPACE = 0, 1, 2, 3, 4, 5
MA_ERR_UNSUPPORTED, MA_ERR_CUDA, MA_ERR_TIMEOUT, MA_ERR_ARG, MA_ERR_BOUNDS = 6, 7, 8, 9, 10
MA_F32, MA_BF16, MA_I32, MA_I64 = 0, 1, 2, 3
MA_MUON, MA_ADAMW = 0, 1
ROLE_HIDDEN, ROLE_EMBED, ROLE_UNEMBED, ROLE_FORCE_ADAMW = 0, 1, 2, 3
MAX_NS_STEPS = 16
MAX_GROUPS = 32
MAX_BATCH = 256


class LibraryMissing(RuntimeError):
    """The compiled library is absent or cannot be loaded (there is no CPU fallback)."""


class MAError(RuntimeError):
    """A C entry point returned a nonzero status; ``code`` holds it."""
    def __init__(self, code: int, what: str = ""):
        self.code = int(code)
        msg = _lib_status_string(code)
        super().__init__(f"{what}: {msg} (status {code})" if what else f"{msg} (status {code})")


# ---------------------------------------------------------------------------- structs (mirror muonadamw.h)

class MuonHParams(ctypes.Structure):
    """ma_muon_hparams_t: Muon hyperparameters (lr, beta, weight decay, eps, Nesterov,
    Newton-Schulz schedule, scale mode, heads, precision, cautious decay)."""
    _fields_ = [("lr", ctypes.c_float), ("beta", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("eps", ctypes.c_float), ("nesterov", ctypes.c_int32), ("ns_steps", ctypes.c_int32),
                ("n_coeffs", ctypes.c_int32), ("coeffs", (ctypes.c_float * 3) * MAX_NS_STEPS),
                ("scale_mode", ctypes.c_int32), ("heads", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("cautious", ctypes.c_int32)]


class AdamWHParams(ctypes.Structure):
    """ma_adamw_hparams_t: AdamW hyperparameters and the 1-based step being taken."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int64)]


class Group(ctypes.Structure):
    """ma_group_t: one parameter group, Muon or AdamW by ``kind``."""
    _fields_ = [("kind", ctypes.c_int32), ("muon", MuonHParams), ("adamw", AdamWHParams)]


class Tensor(ctypes.Structure):
    """ma_tensor_t: one tensor of the table (device pointers, gradient dtype, shape, role, group)."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32),
                ("state0", ctypes.c_void_p), ("state1", ctypes.c_void_p), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 2), ("role", ctypes.c_int32), ("group", ctypes.c_int32)]


class ShardSlot(ctypes.Structure):
    """ma_shard_slot_t: where a tensor sits in the flat buffers of a sharded step."""
    _fields_ = [("bucket", ctypes.c_int32), ("owner", ctypes.c_int32), ("offset", ctypes.c_int64)]


class ShardBucket(ctypes.Structure):
    """ma_shard_bucket_t: one bucket of a sharded step (kind, tensors, start, per-rank segment)."""
    _fields_ = [("kind", ctypes.c_int32), ("count", ctypes.c_int32), ("start", ctypes.c_int64),
                ("seg", ctypes.c_int64)]


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library. Raises LibraryMissing when it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise LibraryMissing(f"{LIB_PATH} is missing: build it with `python -m adamw_hybrid_optimizer_muon_b200.build`")
    try:
        L = ctypes.CDLL(LIB_PATH)
    except OSError as e:
        raise LibraryMissing(f"cannot load {LIB_PATH}: {e}") from e
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    pp = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "ma_status_string": (ctypes.c_char_p, [i32]),
        "ma_version": (i32, []),
        "ma_struct_size": (sz, [i32]),
        "ma_partition": (i32, [ctypes.POINTER(Tensor), i32, ctypes.POINTER(ctypes.c_int32)]),
        "ma_assign_owners": (i32, [ctypes.POINTER(Tensor), i32, ctypes.POINTER(Group), i32, i32,
                                   ctypes.POINTER(ctypes.c_int32)]),
        "ma_shard_layout": (i32, [ctypes.POINTER(Tensor), i32, ctypes.POINTER(Group), i32, i32, i64,
                                  ctypes.POINTER(ShardSlot), ctypes.POINTER(ShardBucket), ctypes.POINTER(i32),
                                  ctypes.POINTER(i64)]),
        "muon_workspace_bytes": (sz, [i32, i64, i64, ctypes.POINTER(MuonHParams)]),
        "muon_step_batched": (i32, [i32, i64, i64, pp, pp, i32, pp, ctypes.POINTER(MuonHParams), vp, sz, vp]),
        "ns_iterate_workspace_bytes": (sz, [i32, i64, i64]),
        "ns_iterate_bf16": (i32, [i32, i64, i64, vp, vp, ctypes.POINTER(ctypes.c_float), i32, i32, vp, sz, vp]),
        "ma_grad_norm": (i32, [i32, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp]),
        "ma_grad_clip": (i32, [i32, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp]),
        "ma_clip_finalize": (i32, [ctypes.c_float, ctypes.c_float, vp, vp]),
        "adamw_step_fused_clipped": (i32, [i32, pp, pp, i32, pp, pp, ctypes.POINTER(ctypes.c_int64),
                                           ctypes.POINTER(AdamWHParams), vp, vp]),
        "muon_step_batched_clipped": (i32, [i32, i64, i64, pp, pp, i32, pp, ctypes.POINTER(MuonHParams), vp, vp, sz,
                                            vp]),
        "ma_embed_lookup": (i32, [i64, vp, i32, i64, i64, vp, i32, i64, ctypes.c_float, i64, vp, i32, i64, vp]),
        "ma_embed_grad_workspace_bytes": (sz, [i64, i64, i64]),
        "ma_embed_grad": (i32, [i64, vp, i32, i64, i64, vp, i32, i64, ctypes.c_float, i64, i32, vp, i32, i64, vp, sz,
                                vp]),
        "ma_qk_max_logit": (i32, [i64, i64, i64, i32, i32, i32, vp, i64, i64, i64, vp, i64, i64, i64, vp, ctypes.c_float,
                                  i32, i32, i32, vp, vp]),
        "ma_qk_clip": (i32, [i32, i32, i64, i64, i64, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp]),
        "ma_plan_set_clip": (i32, [vp, i32, ctypes.c_float, ctypes.c_float, vp]),
        "adamw_step_fused": (i32, [i32, pp, pp, i32, pp, pp, ctypes.POINTER(ctypes.c_int64),
                                   ctypes.POINTER(AdamWHParams), vp]),
        "ma_plan_create": (i32, [ctypes.POINTER(Tensor), i32, ctypes.POINTER(Group), i32, ctypes.POINTER(vp),
                                 ctypes.POINTER(sz)]),
        "muonadamw_step": (i32, [vp, ctypes.POINTER(Group), vp, sz, vp]),
        "muonadamw_step_from_host": (i32, [vp, ctypes.POINTER(Group), pp, vp, sz, vp, vp]),
        "ma_plan_last_launches": (i32, [vp]),
        "muonadamw_step_graph": (i32, [vp, ctypes.POINTER(Group), vp, sz, vp]),
        "ma_plan_graph_captures": (i32, [vp]),
        "ma_plan_describe": (i32, [vp, ctypes.POINTER(Group), ctypes.c_char_p, sz]),
        "ma_plan_destroy": (None, [vp]),
        "ma_device_status": (i32, [vp, i32]),
        "ma_device_status_async": (i32, [vp, vp]),
        "ma_plan_status": (i32, [vp, vp]),
        "ma_set_wait_limit_ns": (i32, [i64]),
        "ma_set_momentum_overlap": (i32, [i32]),
        "ma_debug_build": (i32, []),
        "ma_selftest_wait_timeout": (i32, [i64, vp]),
        "muon_step_batched_noalloc": (i32, [i32, i64, i64, pp, pp, i32, pp, ctypes.POINTER(MuonHParams), vp]),
        "ma_profile_enable": (i32, [i32]),
        "ma_profile_collect": (i32, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64),
                                     ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    for which, cls in enumerate((Tensor, Group, MuonHParams, AdamWHParams, ShardSlot, ShardBucket)):
        if L.ma_struct_size(which) != ctypes.sizeof(cls):
            raise LibraryMissing(f"ABI mismatch for {cls.__name__}: C {L.ma_struct_size(which)} "
                                 f"vs Python {ctypes.sizeof(cls)}")
    _LIB = L
    return L


def _lib_status_string(code: int) -> str:
    try:
        return lib().ma_status_string(int(code)).decode()
    except LibraryMissing:
        return "status"


def _check(code: int, what: str) -> None:
    if code != MA_OK:
        raise MAError(code, what)


# ---------------------------------------------------------------------------- marshalling helpers

def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _ptr_array(xs) -> ctypes.Array:
    try:
        ptrs = _marshal().pointers(xs)
    except TypeError:  # plain addresses, or None, among them
        ptrs = bytearray(array.array("Q", map(_ptr, xs)))
    return (ctypes.c_void_p * max(1, len(ptrs) // 8)).from_buffer(ptrs or bytearray(8))


def _numel_array(xs) -> ctypes.Array:
    """Element counts of tensors."""
    try:
        counts = _marshal().numels(xs)
    except TypeError:
        counts = bytearray(array.array("q", [int(x.numel()) for x in xs]))
    return (ctypes.c_int64 * max(1, len(counts) // 8)).from_buffer(counts or bytearray(8))


class _Methods:
    """What the extension module does, through the tensors' methods."""

    @staticmethod
    def pointers(xs):
        return bytearray(array.array("Q", map(_torch().Tensor.data_ptr, xs)))

    @staticmethod
    def numels(xs):
        return bytearray(array.array("q", map(_torch().Tensor.numel, xs)))

    @classmethod
    def unchanged(cls, xs, ptrs, counts):
        return cls.pointers(xs) == ptrs and cls.numels(xs) == counts


class _Addresses:
    """The same where torch is not installed: the items are addresses, or have the methods."""

    @staticmethod
    def pointers(xs):
        return bytearray(array.array("Q", map(_ptr, xs)))

    @staticmethod
    def numels(xs):
        return bytearray(array.array("q", [int(x.numel()) for x in xs]))


def _marshal_path(torch) -> str:
    """Where the extension module for this Python and this torch is, or would be. It was compiled with the layout of
    that torch's tensors, which another torch need not share although it has every symbol: so the name tells."""
    abi = sysconfig.get_config_var("SOABI")
    return os.path.join(os.path.dirname(LIB_PATH), f"_marshal.{abi}.torch-{torch.__version__}.so")


_MARSHAL = None


def _marshal():
    """The extension module that reads lists of tensors, or what stands in its place."""
    global _MARSHAL
    if _MARSHAL is None:
        try:
            path = _marshal_path(_torch())  # whose libraries it is linked to
        except ImportError:
            _MARSHAL = _Addresses
            return _MARSHAL
        try:
            loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_marshal", path, loader=loader))
            loader.exec_module(module)
            _MARSHAL = module
        except ImportError:  # not built for this Python and torch
            _MARSHAL = _Methods
    return _MARSHAL


_TORCH = None


def _torch():
    """The torch module, imported on first use."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(stream) -> int:
    if stream is None:
        torch = _torch()
        if torch.cuda.is_initialized():  # the handle itself, without a Stream object around it
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _stream_object(handle: int, index: int | None = None):
    """The torch stream of a handle. (ExternalStream takes the default stream's, 0, for none given, and hands out a
    stream of torch's pool.)"""
    cuda = _torch().cuda
    return cuda.ExternalStream(handle, device=index) if handle else cuda.default_stream(index)


def _dtype_code(t) -> int:
    torch = _torch()
    dt = t.dtype
    if dt is torch.bfloat16:
        return MA_BF16
    if dt is torch.float32:
        return MA_F32
    raise MAError(MA_ERR_DTYPE, f"unsupported gradient dtype {dt}")


def muon_hparams(lr=0.02, beta=0.95, weight_decay=0.01, eps=1e-7, nesterov=True, ns_steps=5,
                 coeffs=((1.5, -0.5, 0.0),), scale_mode=0, heads=1, precision=0, cautious=False) -> MuonHParams:
    """Build Muon hyperparameters; ``coeffs`` is one (a, b, c) triple for every iteration or one per iteration."""
    hp = MuonHParams()
    hp.lr, hp.beta, hp.weight_decay, hp.eps = lr, beta, weight_decay, eps
    hp.nesterov, hp.ns_steps, hp.n_coeffs = int(bool(nesterov)), int(ns_steps), len(coeffs)
    if len(coeffs) > MAX_NS_STEPS:
        raise MAError(MA_ERR_ARG, "too many coefficient triples")
    for k, (a, b, c) in enumerate(coeffs):
        hp.coeffs[k][0], hp.coeffs[k][1], hp.coeffs[k][2] = a, b, c
    hp.scale_mode, hp.heads, hp.precision = int(scale_mode), int(heads), int(precision)
    hp.cautious = int(bool(cautious))
    return hp


def adamw_hparams(lr=0.02, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01, step=1) -> AdamWHParams:
    """Build AdamW hyperparameters."""
    hp = AdamWHParams()
    hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, hp.step = lr, beta1, beta2, eps, weight_decay, int(step)
    return hp


# ---------------------------------------------------------------------------- entry points

def ma_partition(tensors: Sequence[Tensor]) -> list:
    """Kind (MA_MUON or MA_ADAMW) of each tensor descriptor, by rank and role (host-only)."""
    n = len(tensors)
    arr = (Tensor * max(1, n))(*tensors)
    out = (ctypes.c_int32 * max(1, n))()
    _check(lib().ma_partition(arr, n, out), "ma_partition")
    return [int(out[i]) for i in range(n)]


def ma_assign_owners(tensors: Sequence[Tensor], groups: Sequence[Group], world_size: int) -> list:
    """Owner rank of each tensor for a sharded data-parallel step over ``world_size`` ranks (host-only)."""
    n = len(tensors)
    arr = (Tensor * max(1, n))(*tensors)
    garr = (Group * max(1, len(groups)))(*groups)
    out = (ctypes.c_int32 * max(1, n))()
    _check(lib().ma_assign_owners(arr, n, garr, len(groups), int(world_size), out), "ma_assign_owners")
    return [int(out[i]) for i in range(n)]


SHARD_ALIGN = 64  # MA_SHARD_ALIGN


def ma_shard_layout(tensors: Sequence[Tensor], groups: Sequence[Group], world_size: int, seg_cap: int):
    """Flat-buffer layout of a sharded data-parallel step (host-only).

    Returns (slots, buckets, total): per tensor a (bucket, owner, offset) tuple
    (owner -1 for AdamW tensors, which are split by element range), per bucket
    a (kind, count, start, seg) tuple, and the flat buffers' length in elements.
    """
    n = len(tensors)
    arr = (Tensor * max(1, n))(*tensors)
    garr = (Group * max(1, len(groups)))(*groups)
    slots = (ShardSlot * max(1, n))()
    buckets = (ShardBucket * max(1, n))()
    nb, total = ctypes.c_int(0), ctypes.c_int64(0)
    _check(lib().ma_shard_layout(arr, n, garr, len(groups), int(world_size), int(seg_cap), slots, buckets,
                                 ctypes.byref(nb), ctypes.byref(total)), "ma_shard_layout")
    return ([(int(s.bucket), int(s.owner), int(s.offset)) for s in slots[:n]],
            [(int(b.kind), int(b.count), int(b.start), int(b.seg)) for b in buckets[:nb.value]],
            int(total.value))


def muon_workspace_bytes(batch: int, R: int, C: int, hp: MuonHParams) -> int:
    """Workspace bytes muon_step_batched needs for ``batch`` R x C matrices."""
    v = lib().muon_workspace_bytes(int(batch), int(R), int(C), ctypes.byref(hp))
    if v == ctypes.c_size_t(-1).value:
        raise MAError(MA_ERR_ARG, "muon_workspace_bytes")
    return int(v)


def muon_step_batched(W, G, M, hp: MuonHParams, ws, ws_bytes: int | None = None, stream=None,
                      gdt: int | None = None, shape=None, clip=None) -> None:
    """One Muon step on same-shape matrices. W, G, M: sequences of torch tensors (or device pointers).
    clip: a clip buffer whose coefficient multiplies the gradients as they are read (see ma_grad_norm)."""
    batch = len(W)
    if shape is None:
        R, C = (int(W[0].shape[0]), int(W[0].shape[1])) if batch else (0, 0)
    else:
        R, C = int(shape[0]), int(shape[1])
    if gdt is None:
        gdt = _dtype_code(G[0]) if batch else MA_F32
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    coef = _clip_ptr("muon_step_batched", clip, CLIP_HEAD_BYTES, _on_current_gpu)
    _check(lib().muon_step_batched_clipped(batch, R, C, _ptr_array(W), _ptr_array(G), int(gdt), _ptr_array(M),
                                           ctypes.byref(hp), coef, _ptr(ws), int(ws_bytes), _stream(stream)),
           "muon_step_batched")


STATIC_SCRATCH_BYTES = 64 << 20  # MA_STATIC_SCRATCH_BYTES


def muon_step_batched_noalloc(W, G, M, hp: MuonHParams, stream=None, gdt: int | None = None, shape=None) -> None:
    """muon_step_batched without a workspace argument: for callers that cannot
    allocate device memory. Its scratch is the library's fixed device array of
    STATIC_SCRATCH_BYTES per GPU, shared by every call: calls that overlap on
    the GPU race. The first call on a device looks up the array's address and
    should come before any stream capture. Raises MAError(MA_ERR_WORKSPACE)
    when the step needs more scratch than the array holds."""
    batch = len(W)
    if shape is None:
        R, C = (int(W[0].shape[0]), int(W[0].shape[1])) if batch else (0, 0)
    else:
        R, C = int(shape[0]), int(shape[1])
    if gdt is None:
        gdt = _dtype_code(G[0]) if batch else MA_F32
    _check(lib().muon_step_batched_noalloc(batch, R, C, _ptr_array(W), _ptr_array(G), int(gdt), _ptr_array(M),
                                           ctypes.byref(hp), _stream(stream)), "muon_step_batched_noalloc")


def ns_iterate_workspace_bytes(batch: int, m: int, n: int) -> int:
    """Workspace bytes ns_iterate_bf16 needs for ``batch`` m x n matrices."""
    return int(lib().ns_iterate_workspace_bytes(int(batch), int(m), int(n)))


def ns_iterate_bf16(X_in, X_out, coeffs, steps: int, ws, ws_bytes: int | None = None, stream=None) -> None:
    """Newton-Schulz iterations (no normalisation) on a [batch, m, n] bf16 tensor with m <= n."""
    batch, m, n = (int(s) for s in X_in.shape)
    flat = [float(x) for c in coeffs for x in c]
    carr = (ctypes.c_float * len(flat))(*flat)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().ns_iterate_bf16(batch, m, n, _ptr(X_in), _ptr(X_out), carr, len(coeffs), int(steps), _ptr(ws),
                                 int(ws_bytes), _stream(stream)), "ns_iterate_bf16")


def adamw_step_fused(P, G, M, V, hp: AdamWHParams, stream=None, gdt: int | None = None, numel=None,
                     clip=None) -> None:
    """One multi-tensor AdamW step over parallel lists of fp32 params, gradients, exp_avg and exp_avg_sq.
    clip: a clip buffer whose coefficient multiplies the gradients as they are read (see ma_grad_norm)."""
    n = len(P)
    if gdt is None:
        gdt = _dtype_code(G[0]) if n else MA_F32
    nar = _numel_array(P) if numel is None else (ctypes.c_int64 * max(1, n))(*numel)
    coef = _clip_ptr("adamw_step_fused", clip, CLIP_HEAD_BYTES, _on_current_gpu)
    _check(lib().adamw_step_fused_clipped(n, _ptr_array(P), _ptr_array(G), int(gdt), _ptr_array(M), _ptr_array(V),
                                          nar, ctypes.byref(hp), coef, _stream(stream)), "adamw_step_fused")


CLIP_BYTES = 16640  # MA_CLIP_BYTES


def clip_buffer(device=None):
    """A clip buffer (fp32 tensor of CLIP_BYTES): element 0 is the norm, 1 the coefficient, and elements 2..3 hold
    the sum of squares as one double. It needs no initial value."""
    import torch
    return torch.empty(CLIP_BYTES // 4, dtype=torch.float32, device=device or "cuda")


def _on_current_gpu(what: str, *tensors) -> None:
    """Refuse tensors that are not on the current CUDA device (the one the launch goes to)."""
    current = None
    for t in tensors:
        if t is None:
            continue
        on = t.get_device()
        if current is None and on >= 0:
            current = _torch()._C._cuda_getDevice()
        if on != current or on < 0:
            raise MAError(MA_ERR_ARG, f"{what}: tensor on {t.device}, not on the current CUDA device")


def _on_gpu(what: str, *tensors) -> None:
    """Refuse tensors that are not on a GPU."""
    for t in tensors:
        if not t.is_cuda:
            raise MAError(MA_ERR_ARG, f"{what}: tensor on {t.device}, not on a GPU")


CLIP_HEAD_BYTES = 16  # norm, coefficient and sum of squares: all that is read of a buffer that is not filled


def _clip_ptr(what: str, clip, nbytes: int, on_gpu) -> int:
    """Address of a clip buffer of which ``nbytes`` are read or written (a plain address, or None, is taken as it is)."""
    if clip is None or isinstance(clip, int):
        return clip or 0
    on_gpu(what, clip)
    if clip.nbytes < nbytes or not clip.is_contiguous():
        raise MAError(MA_ERR_WORKSPACE, f"{what}: a clip buffer has {CLIP_BYTES} contiguous bytes")
    return clip.data_ptr()


def _grad_tables(G):
    """Pointer, dtype and element-count arrays of a list of gradients (contiguous tensors)."""
    n = len(G)
    for g in G:
        if not g.is_contiguous():
            raise MAError(MA_ERR_SHAPE, "gradients must be contiguous")
    return n, _ptr_array(G), (ctypes.c_int32 * max(1, n))(*[_dtype_code(g) for g in G]), _numel_array(G)


def ma_grad_norm(G, clip, max_norm: float = math.inf, scale: float = 1.0, stream=None) -> None:
    """Global norm of a list of gradients (fp32 or bf16, any mix) into the clip buffer: norm = scale * sqrt(sum g^2)
    and coef = scale * min(1, max_norm / norm), 0 when the sum of squares (in fp64) is not finite. A norm beyond fp32
    reads infinite, with the coef of its fp64 value. The gradients are left alone:
    adamw_step_fused, muon_step_batched and the plan's steps take them times coef."""
    _on_current_gpu("ma_grad_norm", *G)
    buf = _clip_ptr("ma_grad_norm", clip, CLIP_BYTES, _on_current_gpu)
    _check(lib().ma_grad_norm(*_grad_tables(G), float(scale), float(max_norm), buf, _stream(stream)), "ma_grad_norm")


def ma_grad_clip(G, clip, max_norm: float, scale: float = 1.0, stream=None) -> None:
    """ma_grad_norm, then every gradient times coef, in place (zero, whatever it holds, where coef is 0)."""
    _on_current_gpu("ma_grad_clip", *G)
    buf = _clip_ptr("ma_grad_clip", clip, CLIP_BYTES, _on_current_gpu)
    _check(lib().ma_grad_clip(*_grad_tables(G), float(scale), float(max_norm), buf, _stream(stream)), "ma_grad_clip")


def ma_clip_finalize(clip, max_norm: float = math.inf, scale: float = 1.0, stream=None) -> None:
    """Norm and coef again from the buffer's sum of squares (after the sums of several ranks were added)."""
    buf = _clip_ptr("ma_clip_finalize", clip, CLIP_HEAD_BYTES, _on_current_gpu)
    _check(lib().ma_clip_finalize(float(scale), float(max_norm), buf, _stream(stream)), "ma_clip_finalize")


def ma_plan_set_clip(plan, clip, max_norm: float = math.inf, scale: float = 1.0, measure: bool = True) -> None:
    """Clip the gradients of the plan's later steps by their global norm, through this buffer (None: off again).
    measure=False: the steps take the coefficient the buffer holds by then, and fill nothing."""
    buf = _clip_ptr("ma_plan_set_clip", clip, CLIP_BYTES if measure else CLIP_HEAD_BYTES, _on_gpu)
    _check(lib().ma_plan_set_clip(plan, int(bool(measure)), float(scale), float(max_norm), buf), "ma_plan_set_clip")


NO_PADDING = -(1 << 63)


def _ids(ids, stream):
    """Contiguous token ids and their dtype code."""
    torch = _torch()
    if ids.dtype is torch.int64:
        idt = MA_I64
    elif ids.dtype is torch.int32:
        idt = MA_I32
    else:
        raise MAError(MA_ERR_DTYPE, f"token ids must be int32 or int64, not {ids.dtype}")
    if not ids.is_contiguous():
        with _on_stream(stream):
            ids = ids.contiguous()
    return ids, idt


def _rows(t, what: str):
    """(tensor as rows x dim, row stride): the last dimension contiguous, the others evenly strided."""
    if t.is_contiguous():
        return t, max(1, t.shape[-1])
    if t.dim() != 2:
        try:
            t = t.view(math.prod(t.shape[:-1]), t.shape[-1])
        except RuntimeError as e:
            raise MAError(MA_ERR_SHAPE, f"{what}: rows are not evenly strided") from e
    rows, dim = t.shape
    if dim > 1 and t.stride(1) != 1:
        raise MAError(MA_ERR_SHAPE, f"{what}: rows must be contiguous")
    return t, (int(t.stride(0)) if rows > 1 else max(1, int(dim)))


_HERE = contextlib.nullcontext()


def _on_stream(stream):
    """A context in which torch allocates for ``stream`` (None: the current one)."""
    if stream is None:
        return _HERE
    torch = _torch()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else _stream_object(_stream(stream)))


def _new(like, shape, dtype, stream):
    """An uninitialised tensor on ``like``'s device, allocated for ``stream``."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on_stream(stream):
        return like.new_empty(shape, dtype=dtype)


def embedding_lookup(ids, table, scale: float = 1.0, padding: int | None = None, out=None, dtype=None, stream=None):
    """Rows of an embedding table by token: out[...] = scale * table[ids[...]], rounded once to ``dtype`` (fp32 or
    bf16; default: the table's), or into ``out`` (shape ids.shape + (dim,)). An id outside the table gives zeros and
    records MA_ERR_BOUNDS in the status word, except ``padding`` (-1, say), which only gives zeros."""
    _on_current_gpu("embedding_lookup", ids, table, out)
    ids, idt = _ids(ids, stream)
    if table.dim() != 2:
        raise MAError(MA_ERR_SHAPE, "embedding_lookup: the table must be 2-D")
    V, D = table.shape
    tab, ldt = _rows(table, "embedding_lookup: table")
    if out is None:
        out = _new(table, (*ids.shape, D), dtype or table.dtype, stream)
    elif out.shape != ids.shape + (D,) or (dtype is not None and out.dtype != dtype):
        raise MAError(MA_ERR_SHAPE, "embedding_lookup: out has another shape or dtype")
    rows, ldo = _rows(out, "embedding_lookup: out")
    _check(lib().ma_embed_lookup(ids.numel(), _ptr(ids), idt, V, D, _ptr(tab), _dtype_code(table), ldt, float(scale),
                                 NO_PADDING if padding is None else int(padding), _ptr(rows), _dtype_code(out), ldo,
                                 _stream(stream)), "embedding_lookup")
    return out


def embed_grad_workspace_bytes(n: int, rows: int, dim: int) -> int:
    """Workspace bytes embedding_grad needs for n tokens and a rows x dim table."""
    v = lib().ma_embed_grad_workspace_bytes(int(n), int(rows), int(dim))
    if v == ctypes.c_size_t(-1).value:
        raise MAError(MA_ERR_ARG, "embed_grad_workspace_bytes")
    return int(v)


def embedding_grad(ids, grad_rows, grad, scale: float = 1.0, padding: int | None = None, accumulate: bool = False,
                   ws=None, stream=None):
    """Gradient of a table from those of the rows looked up, by sorted tokens: grad[v] = scale * sum of grad_rows
    over the tokens that are v. Every row of ``grad`` (fp32 or bf16, the table's shape: the buffer the optimizer
    reads) is written, zeros where no token points; with ``accumulate`` the sums are added to the rows that have
    tokens. fp32 sums in token order, no atomics: the same inputs give the same bits. Tokens equal to ``padding``
    add nothing. ws: workspace (embed_grad_workspace_bytes; allocated here when None). Returns ``grad``."""
    _on_current_gpu("embedding_grad", ids, grad_rows, grad, ws)
    ids, idt = _ids(ids, stream)
    if grad.dim() != 2 or grad_rows.shape != ids.shape + (grad.shape[1],):
        raise MAError(MA_ERR_SHAPE, "embedding_grad: grad must be rows x dim, grad_rows ids.shape + (dim,)")
    V, D = grad.shape
    g, ldg = _rows(grad, "embedding_grad: grad")
    y, ldy = _rows(grad_rows, "embedding_grad: grad_rows")
    n = ids.numel()
    if ws is None:
        ws_bytes = embed_grad_workspace_bytes(n, V, D)
        if ws_bytes:
            ws = _new(grad, ws_bytes, _torch().uint8, stream)
    else:
        if not ws.is_contiguous():
            raise MAError(MA_ERR_WORKSPACE, "embedding_grad: ws must be contiguous")
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().ma_embed_grad(n, _ptr(ids), idt, V, D, _ptr(y), _dtype_code(grad_rows), ldy, float(scale),
                               NO_PADDING if padding is None else int(padding), int(bool(accumulate)), _ptr(g),
                               _dtype_code(grad), ldg, _ptr(ws), ws_bytes, _stream(stream)), "embedding_grad")
    return grad


_SUM_STREAMS = {}  # per device: stream objects, by handle, of lookups whose gradients go to buffers
_LAST_SUM = {}     # per device: stream, backward pass and capture of the last such sum, and the event after it


def _sum_stream(index: int) -> int:
    """The handle of device ``index``'s current stream, which is from now on among those of lookups into buffers."""
    stream = _torch()._C._cuda_getCurrentRawStream(index)
    known = _SUM_STREAMS.get(index)
    if known is None or stream not in known:
        _SUM_STREAMS[index] = {**(known or {}), stream: _stream_object(stream, index)}
    return stream


def _sum_in_turn(index: int, add) -> None:
    """add(), a sum into a gradient buffer of device ``index`` within a backward pass, after the one before it.

    Autograd runs each lookup's backward on the stream of its forward, and joins streams along the edges of the
    graph; two lookups that add to one buffer have no edge between them. So each sum waits for the last one on this
    device when that ran on another stream (whatever its buffer: two views may be one). An event and a wait belong
    to one capture or to none: a captured sum waits for those of its own backward pass, which is captured whole, an
    eager one for any eager one.

    While all lookups were on one stream there is nothing to wait for, and no event is recorded (7 us of the host's
    time a sum in a backward pass). A sum from that time is waited for by what is left: its stream as it is then,
    where the pass is the same, so that the stream is there, else the device."""
    torch = _torch()
    stream, task = _sum_stream(index), torch._C._current_graph_task_id()
    known, last = _SUM_STREAMS[index], _LAST_SUM.get(index)
    if len(known) == 1:
        add()
        _LAST_SUM[index] = stream, task, False, None
        return
    captured = torch._C._cuda_isCurrentStreamCapturing()
    if last is not None and stream != last[0]:
        if last[3] is not None:
            if task == last[1] or not (captured or last[2]):
                known[stream].wait_event(last[3])
        elif task == last[1]:
            known[stream].wait_stream(known[last[0]])
        elif not captured:
            torch.cuda.synchronize(index)
    add()
    event = torch.cuda.Event() if captured or last is None or last[2] or last[3] is None else last[3]
    event.record(known[stream])
    _LAST_SUM[index] = stream, task, captured, event


_EMBEDDING = None


def _embedding_function():
    """The autograd function behind :func:`embedding` (made on first use: torch is imported lazily)."""
    global _EMBEDDING
    if _EMBEDDING is not None:
        return _EMBEDDING
    import torch
    from torch.autograd.function import once_differentiable

    class Embedding(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ids, table, scale, padding, dtype, grad, anchor):
            ctx.save_for_backward(ids)
            ctx.args = scale, padding, grad, table.shape, table.dtype, table.device
            return embedding_lookup(ids, table, scale, padding, dtype=dtype)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            (ids,) = ctx.saved_tensors
            scale, padding, grad, shape, dtype, device = ctx.args
            dy = dy.contiguous()
            if grad is not None:
                _sum_in_turn(grad.get_device(),
                             lambda: embedding_grad(ids, dy, grad, scale, padding, accumulate=True))
                return (None,) * 7
            out = torch.empty(shape, dtype=dtype, device=device)
            return None, embedding_grad(ids, dy, out, scale, padding), None, None, None, None, None

    _EMBEDDING = Embedding
    return Embedding


def embedding(ids, table, scale: float = 1.0, padding: int | None = None, dtype=None, grad=None):
    """embedding_lookup with a gradient for the table (embedding_grad; not differentiable twice, and without a forward
    mode, vmap or the transforms of torch.func).

    ``grad``: a fp32 or bf16 buffer of the shape of the table (which requires
    grad) that backward adds the gradient to, in place of returning one: the buffer the optimizer reads can
    then be filled over several micro-batches, and no table-sized gradient is
    made and added. The caller zeroes it, and it is complete when backward is.
    Lookups of one pass may run on several streams: their sums into buffers are
    ordered. What else writes to the buffer in that pass (the table's own
    ``.grad``, say, when the table is used elsewhere too) has to be on the same
    stream as they are. Autograd does not see this gradient: hooks on the table
    (register_hook, register_post_accumulate_grad_hook, a wrapper that reduces
    gradients in one) do not run for it, and torch.autograd.grad finds no path
    to the table.

    A backward pass captured into a CUDA graph: with ``grad``, at any time;
    without, as with any operator of torch, only while no output of an earlier
    uncaptured call on the table is still alive (torch refuses the capture)."""
    if grad is None:
        return _embedding_function().apply(ids, table, float(scale), padding, dtype, None, None)
    if tuple(grad.shape) != tuple(table.shape):
        raise MAError(MA_ERR_SHAPE, "embedding: grad must have the table's shape")
    # Autograd calls backward for a leaf of this call alone: torch binds a leaf to the stream of its first use, and
    # the table's would tie a captured pass to the stream of an eager one.
    torch = _torch()
    if table.is_cuda:
        _sum_stream(table.get_device())
    needed = table.requires_grad and torch.is_grad_enabled()
    anchor = torch.empty(0, device=table.device, requires_grad=True) if needed else None
    return _embedding_function().apply(ids, table.detach(), float(scale), padding, dtype, grad, anchor)


def qk_max_logit(q, k, scale: float | None = None, causal: bool = True, offsets=None, max_len: int | None = None,
                 absolute: bool = False, out=None, accumulate: bool = False, stream=None):
    """Largest attention logit of each query head: max over sequences and visible pairs of scale * q_i . k_j (with
    ``absolute``, of its magnitude), as ``heads`` floats on the device.

    q: bf16, sequences x tokens x heads x dim, or tokens x heads x dim with
    ``offsets`` (int32 on the device, sequences + 1 positions of sequences laid
    end to end, none longer than ``max_len``; default: all tokens). k: the same
    with a number of heads that divides q's. dim: a multiple of 8 up to 256;
    strides multiples of 8. scale: default dim ** -0.5. ``accumulate`` takes the
    maximum with what ``out`` holds. Without a visible pair: -inf; a NaN logit, or one that ``out`` holds: NaN."""
    torch = _torch()
    _on_current_gpu("qk_max_logit", q, k, offsets, out)
    nd = 3 if offsets is not None else 4
    if q.dim() != nd or k.dim() != nd or q.shape[:-2] != k.shape[:-2] or q.shape[-1] != k.shape[-1]:
        raise MAError(MA_ERR_SHAPE, "qk_max_logit: q and k must be (sequences x) tokens x heads x dim")
    if q.dtype is not torch.bfloat16 or k.dtype is not torch.bfloat16:
        raise MAError(MA_ERR_DTYPE, "qk_max_logit: q and k must be bf16")
    qt, kt = q.stride(), k.stride()
    H, KV, D = q.shape[-2], k.shape[-2], q.shape[-1]
    if (qt[-1] != 1 or kt[-1] != 1) and q.numel():
        raise MAError(MA_ERR_SHAPE, "qk_max_logit: dim must be contiguous")
    if accumulate and out is None:
        raise MAError(MA_ERR_NULL, "qk_max_logit: accumulate needs out")
    if out is None:
        out = _new(q, H, torch.float32, stream)
    elif out.shape != (H,) or out.dtype != torch.float32 or not out.is_contiguous():
        raise MAError(MA_ERR_SHAPE, "qk_max_logit: out must be heads contiguous fp32 values")
    if offsets is not None:
        if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 1 or not offsets.is_contiguous():
            raise MAError(MA_ERR_SHAPE, "qk_max_logit: offsets must be sequences + 1 contiguous int32 positions")
        S, total = offsets.numel() - 1, q.shape[0]
        T, qs, ks = total if max_len is None else int(max_len), 0, 0
    else:
        S, T, total = q.shape[0], q.shape[1], 0
        qs, ks = qt[0], kt[0]
    _check(lib().ma_qk_max_logit(S, T, total, H, KV, D, _ptr(q), qs, qt[-3], qt[-2], _ptr(k), ks, kt[-3], kt[-2],
                                 _ptr(offsets),
                                 D ** -0.5 if scale is None else float(scale), int(bool(causal)), int(bool(absolute)),
                                 int(bool(accumulate)), _ptr(out), _stream(stream)), "qk_max_logit")
    return out


def qk_clip(wq, wk, max_logit, tau: float = 100.0, alpha: float = 0.5, kv_heads: int | None = None, stream=None) -> None:
    """QK-Clip of the query and key weights, in place: heads whose largest logit (``max_logit``, one fp32 value per
    query head, as qk_max_logit gives it) exceeds ``tau`` are scaled so that it becomes tau. wq: (heads * q_rows) x
    cols, wk: (kv_heads * k_rows) x cols, fp32, contiguous (kv_heads: default heads). The query weights take the
    factor to the power alpha, the key weights the rest; a key head shared by several query heads takes what the
    one furthest over needs, and its query heads' weights make up for it, so that each head's logits scale by its
    own factor: those of heads within tau, or whose maximum is not finite, by one. The weights of such a head are not
    touched unless it shares its key head with one over tau (its query weights then grow by what its keys lose).

    Weights replicated over data-parallel ranks: each rank has the maximum of its own batch, and the ranks' weights
    part unless all clip by the same one. Reduce it first: ``dist.all_reduce(max_logit, dist.ReduceOp.MAX)``."""
    torch = _torch()
    _on_current_gpu("qk_clip", wq, wk, max_logit)
    for t in (wq, wk, max_logit):
        if t.dtype != torch.float32:
            raise MAError(MA_ERR_DTYPE, "qk_clip: weights and maxima must be fp32")
        if not t.is_contiguous():
            raise MAError(MA_ERR_SHAPE, "qk_clip: weights and maxima must be contiguous")
    H = max_logit.numel()
    KV = H if kv_heads is None else int(kv_heads)
    if wq.dim() != 2 or wk.dim() != 2 or wq.shape[1] != wk.shape[1] or H < 1 or KV < 1 or wq.shape[0] % H or \
            wk.shape[0] % KV:
        raise MAError(MA_ERR_SHAPE, "qk_clip: weights must be (heads * rows) x cols")
    _check(lib().ma_qk_clip(H, KV, int(wq.shape[0]) // H, int(wk.shape[0]) // KV, int(wq.shape[1]), _ptr(wq), _ptr(wk),
                            _ptr(max_logit), float(tau), float(alpha), _stream(stream)), "qk_clip")


def ma_plan_create(tensors: Sequence[Tensor], groups: Sequence[Group], ws_cap: int = 0):
    """Plan a parameter table; returns (plan handle, workspace bytes the step needs)."""
    n = len(tensors)
    arr = (Tensor * max(1, n))(*tensors)
    garr = (Group * max(1, len(groups)))(*groups)
    plan = ctypes.c_void_p()
    ws = ctypes.c_size_t(int(ws_cap))
    _check(lib().ma_plan_create(arr, n, garr, len(groups), ctypes.byref(plan), ctypes.byref(ws)), "ma_plan_create")
    return plan, int(ws.value)


def muonadamw_step(plan, groups: Sequence[Group], ws, ws_bytes: int, stream=None) -> None:
    """One MuonAdamW step over the planned table, gradients already on the device."""
    garr = (Group * max(1, len(groups)))(*groups)
    _check(lib().muonadamw_step(plan, garr, _ptr(ws), int(ws_bytes), _stream(stream)), "muonadamw_step")


def ma_plan_describe(plan, groups: Sequence[Group]) -> str:
    """Text description of the plan's buckets, sub-batches and launch segments (host-only)."""
    garr = (Group * max(1, len(groups)))(*groups)
    size = 1 << 14
    while True:
        buf = ctypes.create_string_buffer(size)
        rc = lib().ma_plan_describe(plan, garr, buf, size)
        if rc != MA_ERR_SHAPE or size >= 1 << 24:
            _check(rc, "ma_plan_describe")
            return buf.value.decode()
        size *= 4


def muonadamw_step_graph(plan, groups: Sequence[Group], ws, ws_bytes: int, stream=None) -> None:
    """muonadamw_step replayed from a CUDA graph the plan captures and keeps."""
    garr = (Group * max(1, len(groups)))(*groups)
    _check(lib().muonadamw_step_graph(plan, garr, _ptr(ws), int(ws_bytes), _stream(stream)), "muonadamw_step_graph")


def muonadamw_step_from_host(plan, groups: Sequence[Group], host_grads, ws, ws_bytes: int, stream=None,
                             copy_stream=None) -> None:
    """One step whose gradients are copied from host memory (pinned tensors or host pointers) on copy_stream,
    overlapped with the compute on stream."""
    garr = (Group * max(1, len(groups)))(*groups)
    _check(lib().muonadamw_step_from_host(plan, garr, _ptr_array(host_grads), _ptr(ws), int(ws_bytes),
                                          _stream(stream), _stream(copy_stream) if copy_stream is not None
                                          else _stream(stream)), "muonadamw_step_from_host")


def ma_plan_destroy(plan) -> None:
    """Free a plan (and its CUDA graph, if one was captured)."""
    lib().ma_plan_destroy(plan)


def ma_device_status(stream=None, reset: bool = True) -> int:
    """Wait for ``stream``, then read (and by default reset) this device's status word."""
    return int(lib().ma_device_status(_stream(stream), int(bool(reset))))


def ma_plan_status(plan, stream=None) -> int:
    """Wait for ``stream``, then read and clear the status word of the device the plan's steps ran on."""
    return int(lib().ma_plan_status(plan, _stream(stream)))


def ma_device_status_async(host_dst, stream=None) -> None:
    """Enqueue a copy of the device status word into host_dst (a pinned int32 tensor element or address)."""
    _check(lib().ma_device_status_async(_ptr(host_dst), _stream(stream)), "ma_device_status_async")


def ma_set_wait_limit_ns(limit_ns: int) -> None:
    """Time limit of the kernels' bounded waits, in nanoseconds (default 2 s)."""
    _check(lib().ma_set_wait_limit_ns(int(limit_ns)), "ma_set_wait_limit_ns")


def ma_debug_build() -> bool:
    """Whether the loaded library is the build with guarded device indexing."""
    return bool(lib().ma_debug_build())


def ma_set_momentum_overlap(on: bool) -> None:
    """Momentum passes under the previous sub-batch's chain, on a side stream, for plans created
    after the call (default off: slower on a B200, see the header)."""
    _check(lib().ma_set_momentum_overlap(1 if on else 0), "ma_set_momentum_overlap")


def ma_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch a block whose wait can only time out; the status word must then read MA_ERR_TIMEOUT."""
    _check(lib().ma_selftest_wait_timeout(int(limit_ns), _stream(stream)), "ma_selftest_wait_timeout")


PROF_CLASSES = ("adamw", "momentum", "finalize", "ns_gram", "ns_apply", "ns_gramsq", "ns_final", "momentum_side",
                "ns_q1", "clip", "embed", "qk")


def ma_profile_enable(on: bool) -> None:
    """Bracket every later launch of this thread with CUDA events (ma_profile_collect reads them)."""
    _check(lib().ma_profile_enable(int(bool(on))), "ma_profile_enable")


def ma_profile_collect() -> dict:
    """Per kernel class: {"ms", "launches", "flops", "bytes"} summed since the last collect."""
    k = len(PROF_CLASSES)
    ms, cnt = (ctypes.c_double * k)(), (ctypes.c_int64 * k)()
    fl, by = (ctypes.c_double * k)(), (ctypes.c_double * k)()
    _check(lib().ma_profile_collect(ms, cnt, fl, by), "ma_profile_collect")
    return {name: {"ms": ms[i], "launches": int(cnt[i]), "flops": fl[i], "bytes": by[i]}
            for i, name in enumerate(PROF_CLASSES)}


# ---------------------------------------------------------------------------- user-level wrappers

def group_table(groups) -> list:
    """ma_group_t entries from ("muon", MuonHParams) / ("adamw", AdamWHParams) pairs."""
    table = []
    for kind, hp in groups:
        g = Group()
        g.kind = MA_MUON if kind == "muon" else MA_ADAMW
        if g.kind == MA_MUON:
            g.muon = hp
        else:
            g.adamw = hp
        table.append(g)
    return table


class GradClip:
    """Global norm and clipping of a fixed list of gradients (contiguous fp32 or bf16 tensors on one GPU).

    Keeps the pointer tables, so that a call costs a few microseconds of host
    time, and the clip ``buffer`` that the steps take. It clips the tensors it
    was given, wherever their memory is by then, and keeps them alive: they
    have to stay the parameters' gradients. After ``zero_grad()`` they are not,
    since that drops them (``set_to_none=True`` is torch's default); zero them
    in place (``set_to_none=False``), or make another object. Calls that
    overlap on the GPU need an object each.
    """

    def __init__(self, grads):
        self.grads = list(grads)
        self._read_gradients()
        self.buffer = clip_buffer()
        self._norm = self.buffer[0]
        self._ptr = _ptr(self.buffer)
        self._device = self.buffer.get_device()

    def _read_gradients(self):
        _on_current_gpu("GradClip", *self.grads)
        self._tables = _grad_tables(self.grads)
        self._args = (self._tables[0], *[ctypes.addressof(a) for a in self._tables[1:]])
        self._read = (self.grads, _marshal().pointers(self.grads), _marshal().numels(self.grads))
        self._unchanged = _marshal().unchanged
        self._get_device = _torch()._C._cuda_getDevice
        self._get_stream = _torch()._C._cuda_getCurrentRawStream

    def _ready(self, what: str, stream) -> int:
        """Before a call: the device is the buffer's, and the tables are those of the gradients as they are. The
        stream's handle."""
        if self._get_device() != self._device:
            _on_current_gpu(what, self.buffer)
        if not self._unchanged(*self._read):
            self._read_gradients()
        return self._get_stream(self._device) if stream is None else _stream(stream)

    def norm(self, max_norm: float = math.inf, scale: float = 1.0, stream=None):
        """Fill ``buffer``; the norm (times scale) as a 0-d view of it, on the device. The next call overwrites it."""
        at = self._ready("GradClip.norm", stream)
        _check(lib().ma_grad_norm(*self._args, scale, max_norm, self._ptr, at), "ma_grad_norm")
        return self._norm

    def clip(self, max_norm: float, scale: float = 1.0, stream=None):
        """Scale and clip the gradients in place; returns their norm before clipping, as :meth:`norm` does."""
        at = self._ready("GradClip.clip", stream)
        _check(lib().ma_grad_clip(*self._args, scale, max_norm, self._ptr, at), "ma_grad_clip")
        return self._norm


class Plan:
    """Owns an ma_plan_t and its device workspace (a torch uint8 buffer)."""

    def __init__(self, tensors: Sequence[Tensor], groups: Sequence[Group], ws_cap: int = 0, device=None):
        import torch
        self.tensors = list(tensors)
        self.groups = list(groups)
        self.handle, self.ws_bytes = ma_plan_create(self.tensors, self.groups, ws_cap)
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=device or "cuda")

    def step(self, groups: Sequence[Group] | None = None, stream=None, graph: bool = False) -> None:
        fn = muonadamw_step_graph if graph else muonadamw_step
        fn(self.handle, groups if groups is not None else self.groups, self.ws, self.ws.numel(), stream)

    def step_from_host(self, host_grads, groups: Sequence[Group] | None = None, stream=None,
                       copy_stream=None) -> None:
        muonadamw_step_from_host(self.handle, groups if groups is not None else self.groups, host_grads, self.ws,
                                 self.ws.numel(), stream, copy_stream)

    def set_clip(self, clip, max_norm: float = math.inf, scale: float = 1.0) -> None:
        """Clip the gradients of later steps by their global norm, through a clip buffer (None: off)."""
        ma_plan_set_clip(self.handle, clip, max_norm, scale)
        self.clip = clip  # keeps the buffer alive

    @property
    def launches(self) -> int:
        return int(lib().ma_plan_last_launches(self.handle))

    @property
    def graph_captures(self) -> int:
        return int(lib().ma_plan_graph_captures(self.handle))

    def status(self, stream=None) -> int:
        """Wait for ``stream``; MA_OK or the first device-side error of the steps since the last read."""
        return ma_plan_status(self.handle, stream)

    def describe(self, groups: Sequence[Group] | None = None) -> str:
        """What a step runs: workspace, buckets, sub-batches and shared launches."""
        return ma_plan_describe(self.handle, groups if groups is not None else self.groups)

    def close(self) -> None:
        if self.handle is not None and self.handle.value:
            ma_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MuonAdamW:
    """Torch-facing optimizer over (param, role, group) entries.

    ``params``: list of (tensor, role, group_index). The fp32 params live on the
    GPU. Gradients are read from ``param.grad`` (fp32 or bf16), or from the
    ``grads`` list given to :meth:`step`. ``groups``: list of
    ("muon", MuonHParams) or ("adamw", AdamWHParams). State buffers are
    allocated here, zero-initialised, and owned by this object. The AdamW
    step counter advances on every call.
    """

    def __init__(self, params, groups, ws_cap: int = 0):
        import torch
        self.entries = list(params)
        self.groups = group_table(groups)
        self.state = []
        self.step_count = 0
        self._ws_cap = ws_cap
        self._plan = None
        self._grad_ptrs = None
        self._clip = None
        kinds = ma_partition([self._desc(p, role, grp, None) for p, role, grp in self.entries])
        for (p, role, grp), kind in zip(self.entries, kinds):
            s0 = torch.zeros_like(p)
            s1 = torch.zeros_like(p) if kind == MA_ADAMW else None
            self.state.append((s0, s1))

    @staticmethod
    def _desc(p, role, grp, g, s0=None, s1=None) -> Tensor:
        t = Tensor()
        t.param = _ptr(p)
        t.grad = _ptr(g)
        t.grad_dtype = _dtype_code(g) if g is not None else MA_F32
        t.state0 = _ptr(s0)
        t.state1 = _ptr(s1)
        t.ndim = p.dim()
        for d in range(min(2, p.dim())):
            t.shape[d] = int(p.shape[d])
        t.role = int(role)
        t.group = int(grp)
        return t

    def _ensure_plan(self, grads):
        ptrs = tuple(_ptr(g) for g in grads)
        if self._plan is not None and ptrs == self._grad_ptrs:
            return
        if self._plan is not None:
            self._plan.close()
        descs = [self._desc(p, role, grp, g, s0, s1)
                 for (p, role, grp), g, (s0, s1) in zip(self.entries, grads, self.state)]
        self._plan = Plan(descs, self.groups, self._ws_cap, device=self.entries[0][0].device)
        self._grad_ptrs = ptrs

    def _advance(self):
        self.step_count += 1
        for g in self.groups:
            if g.kind == MA_ADAMW:
                g.adamw.step = self.step_count

    def _set_clip(self, max_norm, grad_scale):
        if max_norm is None and grad_scale == 1.0:
            self._plan.set_clip(None)
            return
        if self._clip is None:
            self._clip = clip_buffer(self.entries[0][0].device)
        self._plan.set_clip(self._clip, math.inf if max_norm is None else max_norm, grad_scale)

    @property
    def grad_norm(self):
        """Global gradient norm (times grad_scale) of the last step that had one, as a 0-d device tensor that the
        next such step overwrites. NaN or infinite where a gradient was (that step took every gradient as zero), and
        infinite too where finite gradients have a norm beyond fp32 (that step clipped them): grad_coef tells."""
        if self._clip is None:
            raise RuntimeError("no step with max_norm or grad_scale yet")
        return self._clip[0]

    @property
    def grad_coef(self):
        """What the last step with max_norm or grad_scale multiplied the gradients by, as a 0-d device tensor that
        the next such step overwrites. 0 where max_norm is above it: a gradient was not finite, and that step took
        every one as zero."""
        if self._clip is None:
            raise RuntimeError("no step with max_norm or grad_scale yet")
        return self._clip[1]

    def step(self, grads=None, stream=None, graph: bool = False, max_norm: float | None = None,
             grad_scale: float = 1.0) -> None:
        """One step. max_norm: clip the gradients to this global norm; grad_scale: what they have to be multiplied by
        first (1 / loss scale). Both are applied as the step reads the gradients, which stay as they are; a gradient
        that is not finite makes it a step with zero gradients (grad_coef is then 0). graph=True replays the step from
        a CUDA graph that the plan captures on first use (same results; one launch instead of one per kernel).
        A plan, and with it the graph, belongs to one set of gradient buffers:
        keep them at fixed addresses (as persistent ``.grad`` tensors are)."""
        if grads is None:
            grads = [p.grad for p, _, _ in self.entries]
        self._ensure_plan(grads)
        self._set_clip(max_norm, grad_scale)
        self._advance()
        self._plan.step(self.groups, stream, graph)

    def step_from_host(self, host_grads, device_grads, stream=None, copy_stream=None,
                       max_norm: float | None = None, grad_scale: float = 1.0) -> None:
        """One step whose gradients arrive from host memory. With max_norm or grad_scale (as in step) the
        updates start after the last copy, since the norm needs every gradient.

        host_grads: pinned CPU tensors (or host pointers), one per entry.
        device_grads: the device buffers that receive them (same shapes and
        dtypes); the library copies each group of gradients on copy_stream
        (default: a stream owned by this optimizer) and overlaps the copies
        with the compute on stream.

        The call returns before the copies have read host_grads: do not write
        to them until ``host_copies_done`` (a CUDA event recorded on the copy
        stream after the last copy) has completed, e.g.
        ``opt.host_copies_done.synchronize()``.
        """
        import torch
        self._ensure_plan(device_grads)
        if copy_stream is None:
            if getattr(self, "_copy_stream", None) is None:
                self._copy_stream = torch.cuda.Stream(device=self.entries[0][0].device)
            copy_stream = self._copy_stream
        self._set_clip(max_norm, grad_scale)
        self._advance()
        self._plan.step_from_host(host_grads, self.groups, stream, copy_stream)
        cs = copy_stream if isinstance(copy_stream, torch.cuda.Stream) else _stream_object(int(copy_stream))
        self.host_copies_done = torch.cuda.Event()
        self.host_copies_done.record(cs)

    def state_dict(self) -> dict:
        """The step count and the state buffers (the tensors themselves, not
        copies): per entry (momentum, None) for Muon, (exp_avg, exp_avg_sq)
        for AdamW."""
        return {"step": self.step_count, "state": list(self.state)}

    def load_state_dict(self, sd: dict) -> None:
        """Copy a state_dict of an optimizer over the same table into this one."""
        if len(sd["state"]) != len(self.state):
            raise ValueError("state of another parameter table")
        for (a0, a1), (b0, b1) in zip(self.state, sd["state"]):
            if a0.shape != b0.shape or (a1 is None) != (b1 is None):
                raise ValueError("state of another parameter table")
            a0.copy_(b0)
            if a1 is not None:
                a1.copy_(b1)
        self.step_count = int(sd["step"])

    @property
    def launches(self) -> int:
        return self._plan.launches if self._plan is not None else 0

    @property
    def graph_captures(self) -> int:
        """How many times the plan captured its CUDA graph (graph steps only)."""
        return self._plan.graph_captures if self._plan is not None else 0

    def describe(self) -> str:
        """What a step runs (buckets, sub-batches, shared launches); needs one step first."""
        if self._plan is None:
            raise RuntimeError("no plan yet: the plan is built on the first step")
        return self._plan.describe(self.groups)
