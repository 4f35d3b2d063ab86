"""GB300 ring attention -- forward, backward and the context-parallel variants:
the Python binding of libra.so (include/ra.h).

The functions keep the C names (``ra_plan``, ``ra_plan_window``, ``ra_plan_tile_counts``, ``ra_fwd``,
``ra_fwd_static``, ``ra_fwd_static_status``, ``ra_merge_partials``, ``ra_layout_perm``, ``ra_layout_index``,
``ra_fwd_step``, ``ra_ring_rotate``, ``ra_ring_fwd``, ``ra_bwd``,
``ra_bwd_scratch_size``, ``ra_allgather_kv``, ``ra_fwd_gathered``,
``ra_ulysses_a2a``, ``ra_sync_status``, ``ra_wait_selftest``, ``ra_last_error``;
``ra_kv4_plan``, ``ra_kv4_cache_size``, ``ra_kv4_write``, ``ra_kv4_read``,
``ra_kv4_attend``, ``ra_kv4_attend_scratch_size``, ``ra_kv4_sync_status``;
``ra_rope_plan``, ``ra_rope``, ``ra_rope_bwd``;
``ra_paged_plan``, ``ra_paged_append``, ``ra_paged_attend``, ``ra_paged_attend_scratch_size``,
``ra_paged_weigh``, ``ra_paged_weigh_scratch_size``, ``ra_paged_evict``, ``ra_paged_sync_status``).
This module only marshals arguments: PyTorch supplies device memory and the
current stream (outputs and scratch made for a call with a ``stream`` of its own belong to
that stream), every step of the computation runs in the library's CUDA kernels, and there is
no fallback -- if libra.so is missing or cannot be loaded, every call raises.  Because the library sees only pointers, every tensor a caller
passes (outputs and scratch included) is checked here for its exact shape, dtype,
contiguity and device before anything is launched.

Tensors are ``[B, H, S, d]`` contiguous with S in layout order (shard p owns rows
[p*S/N, (p+1)*S/N)); ``ra_layout_perm`` moves natural order <-> layout order.  The rotations
take them with any strides, and the paged cache takes packed tensors ``[tokens, H, d]``.

With RA_LIBRARY_VARIANT=debug in the environment the binding loads libra_debug.so
instead: the same library with the kernels' bounds checks compiled in, which
``ra_sync_status`` reports as RaError(RA_ERR_BOUNDS).
"""

import contextlib
import ctypes
import os

import numpy as np

__all__ = [
    "RaError", "Plan", "LAYOUTS",
    "ra_plan", "ra_plan_window", "ra_plan_destroy", "ra_plan_tile_counts", "ra_fwd", "ra_merge_partials",
    "ra_layout_perm", "ra_layout_index", "ra_sync_status", "ra_last_error", "ra_fwd_static",
    "ra_fwd_static_status", "ra_fwd_step", "ra_ring_rotate", "ra_ring_fwd", "ra_bwd", "ra_bwd_scratch_size",
    "ra_allgather_kv", "ra_fwd_gathered", "ra_ulysses_a2a", "ra_wait_selftest",
    "Kv4", "ra_kv4_plan", "ra_kv4_destroy", "ra_kv4_cache_size", "ra_kv4_write", "ra_kv4_read", "ra_kv4_attend",
    "ra_kv4_attend_scratch_size", "ra_kv4_sync_status",
    "Rope", "ROPE_SCALINGS", "ra_rope_plan", "ra_rope_destroy", "ra_rope", "ra_rope_bwd",
    "Paged", "ra_paged_plan", "ra_paged_destroy", "ra_paged_cache_shape", "ra_paged_append", "ra_paged_attend",
    "ra_paged_attend_scratch_size", "ra_paged_weigh", "ra_paged_weigh_scratch_size", "ra_paged_evict",
    "ra_paged_sync_status",
    "library_path", "load_library", "EXPORTED",
]

LAYOUTS = {"contiguous": 0, "striped": 1, "zigzag": 2}
DTYPES = {"f32": 0, "bf16": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}
_STATUS = {0: "RA_OK", 1: "RA_ERR_INVALID_ARG", 2: "RA_ERR_UNSUPPORTED", 3: "RA_ERR_CUDA",
           4: "RA_ERR_TIMEOUT", 5: "RA_ERR_NO_DEVICE", 6: "RA_ERR_BOUNDS"}
EXPORTED = ("ra_plan", "ra_plan_window", "ra_plan_destroy", "ra_plan_tile_counts", "ra_fwd", "ra_merge_partials",
            "ra_layout_perm", "ra_layout_index", "ra_sync_status", "ra_last_error", "ra_fwd_static",
            "ra_fwd_static_status", "ra_fwd_step", "ra_ring_rotate", "ra_ring_fwd", "ra_bwd", "ra_bwd_scratch_size",
            "ra_allgather_kv", "ra_fwd_gathered", "ra_ulysses_a2a", "ra_wait_selftest",
            "ra_kv4_plan", "ra_kv4_destroy", "ra_kv4_cache_size", "ra_kv4_write", "ra_kv4_read", "ra_kv4_attend",
            "ra_kv4_attend_scratch_size", "ra_kv4_sync_status",
            "ra_rope_plan", "ra_rope_destroy", "ra_rope", "ra_rope_bwd",
            "ra_paged_plan", "ra_paged_destroy", "ra_paged_append", "ra_paged_attend", "ra_paged_attend_scratch_size",
            "ra_paged_weigh", "ra_paged_weigh_scratch_size", "ra_paged_evict", "ra_paged_sync_status")

_TORCH = None
_NO_CONTEXT = contextlib.nullcontext()


def _torch():
    """The torch module, imported at the first call that needs it (the helpers below run several
    times a call, where an import statement costs more than the check it is for)."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class RaError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        self.name = _STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {message}")


class _Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seq", ctypes.c_int64), ("heads_q", ctypes.c_int32),
                ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("n_shards", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("causal", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _Kv4Problem(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("page_rows", ctypes.c_int32), ("heads_q", ctypes.c_int32),
                ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("scale", ctypes.c_float)]


class _RopeProblem(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("base", ctypes.c_double), ("scaling", ctypes.c_int32),
                ("factor", ctypes.c_double), ("original", ctypes.c_int64), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class _PagedProblem(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("page_rows", ctypes.c_int32), ("heads_q", ctypes.c_int32),
                ("heads_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("scale", ctypes.c_float)]


def library_path():
    """libra.so, or with RA_LIBRARY_VARIANT=debug in the environment libra_debug.so: the same
    library with the kernels' bounds checks compiled in (built by build.build_all())."""
    name = "libra_debug.so" if os.environ.get("RA_LIBRARY_VARIANT") == "debug" else "libra.so"
    return os.path.join(_HERE, name)


def load_library():
    """Load libra.so (built in-tree by ``build.build()``); raises if it is absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run context_ring_attention_gb300.build.build_all()")
    lib = ctypes.CDLL(path)
    P, I32, I64, VP = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    sig = {
        "ra_plan": ([ctypes.POINTER(_Problem), ctypes.POINTER(P)], I32),
        "ra_plan_window": ([ctypes.POINTER(_Problem), I64, I64, ctypes.POINTER(P)], I32),
        "ra_plan_destroy": ([P], I32),
        "ra_plan_tile_counts": ([P, VP, VP, VP], I32),
        "ra_fwd": ([P, VP, VP, VP, VP, VP, VP, VP, VP], I32),
        "ra_merge_partials": ([I32, I64, I32, VP, VP, VP, I32, VP, VP], I32),
        "ra_layout_perm": ([I32, I64, I32, I32, I64, I32, VP, VP, VP], I32),
        "ra_layout_index": ([I32, I64, I32, VP], I32),
        "ra_sync_status": ([P, VP], I32),
        "ra_last_error": ([], ctypes.c_char_p),
        "ra_fwd_static": ([ctypes.POINTER(_Problem), VP, VP, VP, VP, VP, VP], I32),
        "ra_fwd_static_status": ([VP], I32),
        "ra_fwd_step": ([P, I32, VP, VP, VP, VP, VP, VP], I32),
        "ra_ring_rotate": ([P, VP, VP, VP, VP, VP], I32),
        "ra_ring_fwd": ([P, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP], I32),
        "ra_bwd": ([P, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP], I32),
        "ra_bwd_scratch_size": ([P, VP], I32),
        "ra_allgather_kv": ([P, VP, VP, VP, VP, VP], I32),
        "ra_fwd_gathered": ([P, VP, VP, VP, VP, VP, VP], I32),
        "ra_ulysses_a2a": ([I32, I32, I64, I32, I64, I32, I32, VP, VP, VP], I32),
        "ra_wait_selftest": ([VP], I32),
        "ra_kv4_plan": ([ctypes.POINTER(_Kv4Problem), ctypes.POINTER(P)], I32),
        "ra_kv4_destroy": ([P], I32),
        "ra_kv4_cache_size": ([P, VP], I32),
        "ra_kv4_write": ([P, VP, I64, I64, VP, VP, VP, I64, VP, VP, VP], I32),
        "ra_kv4_read": ([P, VP, I64, I64, VP, I64, VP, VP, I32, VP, VP, VP], I32),
        "ra_kv4_attend": ([P, VP, I64, I64, VP, VP, I64, VP, VP, VP, VP, VP], I32),
        "ra_kv4_attend_scratch_size": ([P, I64, I64, I64, VP], I32),
        "ra_kv4_sync_status": ([P, VP], I32),
        "ra_rope_plan": ([ctypes.POINTER(_RopeProblem), ctypes.POINTER(P)], I32),
        "ra_rope_destroy": ([P], I32),
        "ra_rope": ([P, I64, I64, I32, I32, I32, I32, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP], I32),
        "ra_rope_bwd": ([P, I64, I64, I32, I32, I32, I32, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP], I32),
        "ra_paged_plan": ([ctypes.POINTER(_PagedProblem), ctypes.POINTER(P)], I32),
        "ra_paged_destroy": ([P], I32),
        "ra_paged_append": ([P, P, VP, I64, I64, VP, VP, VP, VP, VP, VP, VP, VP, VP, I64, VP, VP, VP, VP], I32),
        "ra_paged_attend": ([P, VP, I64, I64, VP, VP, VP, I64, VP, VP, VP, VP, VP, VP, VP], I32),
        "ra_paged_attend_scratch_size": ([P, I64, I64, I64, VP], I32),
        "ra_paged_weigh": ([P, VP, I64, I64, VP, VP, VP, VP, I64, VP, VP, VP, VP, I64, VP, VP], I32),
        "ra_paged_weigh_scratch_size": ([P, I64, I64, I64, VP], I32),
        "ra_paged_evict": ([P, VP, I64, VP, I64, VP, VP, VP, I64, I64, I64, I64, VP, I64, VP, VP, VP], I32),
        "ra_paged_sync_status": ([P, VP], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = lib
    return lib


def ra_last_error():
    return load_library().ra_last_error().decode()


def _check(status):
    if status != 0:
        raise RaError(status, ra_last_error())


def _layout(layout):
    return LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    torch = _TORCH or _torch()
    if stream is None:
        # (the raw handle: building a Stream object for it takes longer than a launch)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    cur = torch.cuda.current_device()
    if stream.device.index != cur:
        raise ValueError(f"the stream belongs to {stream.device}; the library launches on the current device "
                         f"cuda:{cur}")
    return stream.cuda_stream


def _alloc_on(stream):
    """Context in which buffers made for a call belong to the stream the call runs on, so that
    the allocator does not hand them on while its kernels may still use them."""
    torch = _TORCH or _torch()
    if stream is None:
        return _NO_CONTEXT
    if isinstance(stream, int):  # (1 is the runtime's name of the default stream)
        stream = torch.cuda.ExternalStream(0 if stream == 1 else stream)
    return torch.cuda.stream(stream)


def _on_current_device(name, t):
    """The kernels run on the current CUDA device: every buffer must live there."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = (_TORCH or _torch())._C._cuda_getDevice()  # (a CUDA tensor exists: the runtime is up)
    if t.get_device() != cur:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur} "
                         f"(make its device current, e.g. with torch.cuda.device)")


class Plan:
    """Owns an ``ra_plan_t``; the problem it was built for is ``self.problem``."""

    def __init__(self, handle, problem):
        self._h = handle
        self.problem = problem
        self._bwd_scratch = None  # bytes of ra_bwd's scratch

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load_library().ra_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _make_plan(batch, seq, heads_q, heads_kv, head_dim, n_shards, layout, causal, dtype, scale, create):
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    prob = _Problem(int(batch), int(seq), int(heads_q), int(heads_kv), int(head_dim), int(n_shards),
                    _layout(layout), int(bool(causal)), dt, float(scale or 0.0))
    h = ctypes.c_void_p()
    _check(create(prob, h))
    info = dict(batch=int(batch), seq=int(seq), heads_q=int(heads_q), heads_kv=int(heads_kv),
                head_dim=int(head_dim), n_shards=int(n_shards), layout=_layout(layout),
                causal=bool(causal), dtype=dt, scale=float(scale or 0.0))
    return Plan(h, info)


def ra_plan(batch, seq, heads_q, heads_kv, head_dim, n_shards, layout="contiguous",
            causal=False, dtype="bf16", scale=0.0):
    """Validate a problem and build its ring schedule (see include/ra.h)."""
    lib = load_library()
    return _make_plan(batch, seq, heads_q, heads_kv, head_dim, n_shards, layout, causal, dtype, scale,
                      lambda prob, h: lib.ra_plan(ctypes.byref(prob), ctypes.byref(h)))


def ra_plan_window(batch, seq, heads_q, heads_kv, head_dim, n_shards, window, sinks=0, layout="contiguous",
                   dtype="bf16", scale=0.0):
    """A causal plan in which a query sees its last ``window`` keys and the first ``sinks`` keys.

    Key j is visible to query i (natural positions) when j <= i and (j > i - window or
    j < sinks).  The plan works with every call that takes one: ``ra_fwd``,
    ``ra_fwd_step``, ``ra_ring_fwd``, ``ra_fwd_gathered`` and ``ra_bwd``.
    """
    lib = load_library()
    plan = _make_plan(batch, seq, heads_q, heads_kv, head_dim, n_shards, layout, True, dtype, scale,
                      lambda prob, h: lib.ra_plan_window(ctypes.byref(prob), int(window), int(sinks), ctypes.byref(h)))
    plan.problem.update(window=int(window), sinks=int(sinks))
    return plan


def ra_plan_destroy(plan):
    plan.close()


def ra_plan_tile_counts(plan):
    """Per-shard (FULL, PARTIAL, SKIP) tile counts of one (batch, query head)."""
    n = plan.problem["n_shards"]
    full, part, skip = (np.zeros(n, np.int64) for _ in range(3))
    _check(load_library().ra_plan_tile_counts(plan.handle, full.ctypes.data, part.ctypes.data,
                                              skip.ctypes.data))
    return full, part, skip


def _check_qkv(plan, **tensors):
    """Shape/dtype/contiguity of q ([B, Hq, S, d]) and K/V-like ([B, Hkv, S, d]) arguments, all
    on the current device."""
    torch = _TORCH or _torch()
    pb = plan.problem
    B, S, d = pb["batch"], pb["seq"], pb["head_dim"]
    dt = torch.bfloat16 if pb["dtype"] == 1 else torch.float32
    for name, t in tensors.items():
        shape = (B, pb["heads_q"] if name == "q" else pb["heads_kv"], S, d)
        if t.shape != shape or t.dtype != dt or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor of shape {shape}")
        _on_current_device(name, t)


def _need_like(name, t, shape, dtype, device):
    """``t`` must be a contiguous tensor of exactly this shape and dtype on ``device``, a device
    that was checked already."""
    if (not isinstance(t, (_TORCH or _torch()).Tensor) or t.shape != tuple(shape) or t.dtype != dtype or t.device != device
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _need(name, t, shape, dtype, device):
    """``t`` must be a contiguous tensor of exactly this shape and dtype on ``device``, which
    must be the current device: the library sees only its pointer, so a smaller buffer would
    be overrun."""
    _need_like(name, t, shape, dtype, device)
    _on_current_device(name, t)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def ra_fwd(plan, q, k, v, o=None, lse=None, partials=False, o_parts=None, lse_parts=None,
           stream=None):
    """Ring-attention forward.  Fused: returns (O, LSE).  partials=True: (O_parts, LSE_parts)."""
    torch = _TORCH or _torch()
    pb = plan.problem
    B, Hq, S, d, N = pb["batch"], pb["heads_q"], pb["seq"], pb["head_dim"], pb["n_shards"]
    _check_qkv(plan, q=q, k=k, v=v)
    lib = load_library()
    if partials:
        with _alloc_on(stream):
            if o_parts is None:
                o_parts = torch.empty((N, B, Hq, S, d), dtype=torch.float32, device=q.device)
            if lse_parts is None:
                lse_parts = torch.empty((N, B, Hq, S), dtype=torch.float32, device=q.device)
        _need("o_parts", o_parts, (N, B, Hq, S, d), torch.float32, q.device)
        _need("lse_parts", lse_parts, (N, B, Hq, S), torch.float32, q.device)
        _check(lib.ra_fwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), None, None, _ptr(o_parts),
                          _ptr(lse_parts), _stream(stream)))
        return o_parts, lse_parts
    if o is not None:
        _need_like("o", o, q.shape, q.dtype, q.device)
    if lse is not None:
        _need_like("lse", lse, (B, Hq, S), torch.float32, q.device)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    _check(lib.ra_fwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), None, None,
                      _stream(stream)))
    return o, lse


def ra_merge_partials(o_parts, lse_parts, out_dtype=None, o=None, lse=None, stream=None):
    """Merge [n, ..., d] partial outputs with their [n, ...] LSEs -> (O, LSE)."""
    import torch
    n, d = o_parts.shape[0], o_parts.shape[-1]
    rows = lse_parts[0].numel()
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise ValueError("partials must be float32")
    if not (o_parts.is_contiguous() and lse_parts.is_contiguous()):
        raise ValueError("partials must be contiguous")
    if tuple(lse_parts.shape) != tuple(o_parts.shape[:-1]):
        raise ValueError("lse_parts must have the shape of o_parts without its last axis")
    _on_current_device("o_parts", o_parts)
    _same_device(o_parts.device, lse_parts=lse_parts)
    out_dtype = out_dtype or torch.float32
    with _alloc_on(stream):
        if o is None:
            o = torch.empty(o_parts.shape[1:], dtype=out_dtype, device=o_parts.device)
        if lse is None:
            lse = torch.empty(lse_parts.shape[1:], dtype=torch.float32, device=o_parts.device)
    if o.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("o must be float32 or bfloat16")
    _need("o", o, o_parts.shape[1:], o.dtype, o_parts.device)
    _need("lse", lse, lse_parts.shape[1:], torch.float32, o_parts.device)
    code = 1 if o.dtype == torch.bfloat16 else 0
    _check(load_library().ra_merge_partials(n, rows, d, _ptr(o_parts), _ptr(lse_parts), _ptr(o), code,
                                            _ptr(lse), _stream(stream)))
    return o, lse


def ra_layout_perm(x, layout, n_shards, inverse=False, seq_dim=None, out=None, stream=None):
    """Natural -> layout order (inverse=False) or back, along ``seq_dim``.

    ``seq_dim`` defaults to 2, the sequence axis of the library's [B, H, S, d] and
    [B, H, S] tensors.  Everything after the sequence axis moves as one row.
    """
    import torch
    if not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous CUDA tensor")
    seq_dim = (2 if seq_dim is None else seq_dim) % x.dim()
    seq = x.shape[seq_dim]
    outer = int(np.prod(x.shape[:seq_dim], dtype=np.int64)) if seq_dim else 1
    row_bytes = int(np.prod(x.shape[seq_dim + 1:], dtype=np.int64)) * x.element_size()
    if out is None:
        with _alloc_on(stream):
            out = torch.empty_like(x)
    _need("out", out, x.shape, x.dtype, x.device)
    _check(load_library().ra_layout_perm(_layout(layout), seq, int(n_shards), int(bool(inverse)), outer,
                                         row_bytes, _ptr(x), _ptr(out), _stream(stream)))
    return out


def ra_layout_index(layout, seq, n_shards):
    """Natural position of every layout-ordered row (host helper)."""
    pos = np.zeros(int(seq), np.int64)
    _check(load_library().ra_layout_index(_layout(layout), int(seq), int(n_shards), pos.ctypes.data))
    return pos


def ra_wait_selftest():
    """Run the tensor-core kernels' bounded wait against a barrier nothing completes
    (about one second); returns the status word it left (2: it gave up as designed)."""
    word = ctypes.c_uint32(0)
    _check(load_library().ra_wait_selftest(ctypes.addressof(word)))
    return word.value


def ra_sync_status(plan, stream=None):
    """Synchronize the stream and raise RaError if a device wait of this plan timed out."""
    _check(load_library().ra_sync_status(plan.handle, _stream(stream)))


def ra_fwd_static(batch, seq, heads_q, heads_kv, n_shards, layout, causal, q, k, v, o=None, lse=None,
                  scale=0.0, stream=None):
    """Fused bf16 forward without a plan and without allocating device memory.

    For callers that must not allocate device memory at run time (the library's
    static scratch array holds the work list).  Returns (O, LSE); pass ``o`` and
    ``lse`` to avoid the two torch allocations this wrapper otherwise makes.
    """
    import torch
    _need("q", q, (batch, heads_q, seq, 128), torch.bfloat16, q.device)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    _need("k", k, (batch, heads_kv, seq, 128), torch.bfloat16, q.device)
    _need("v", v, (batch, heads_kv, seq, 128), torch.bfloat16, q.device)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((batch, heads_q, seq), dtype=torch.float32, device=q.device)
    _need("o", o, q.shape, q.dtype, q.device)
    _need("lse", lse, (batch, heads_q, seq), torch.float32, q.device)
    prob = _Problem(int(batch), int(seq), int(heads_q), int(heads_kv), 128, int(n_shards), _layout(layout),
                    int(bool(causal)), 1, float(scale or 0.0))
    _check(load_library().ra_fwd_static(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                        _stream(stream)))
    return o, lse


def ra_fwd_static_status(stream=None):
    """Raise RaError (RA_ERR_TIMEOUT) if the latest ra_fwd_static call on the current
    device gave up on a device-side wait; synchronizes ``stream`` first."""
    _check(load_library().ra_fwd_static_status(_stream(stream)))


def ra_fwd_step(plan, step, q, k_blk, v_blk, o_part=None, lse_part=None, stream=None):
    """One ring step for every shard over the blocks the shards hold -> (O_t, LSE_t) in float32.

    ``k_blk``/``v_blk`` hold, in the rows of shard p, the block shard p holds at this
    step (K/V themselves at step 0; ``ra_ring_rotate`` passes them on).
    """
    import torch
    pb = plan.problem
    B, Hq, S, d = pb["batch"], pb["heads_q"], pb["seq"], pb["head_dim"]
    _check_qkv(plan, q=q, k_blk=k_blk, v_blk=v_blk)
    _same_device(q.device, k_blk=k_blk, v_blk=v_blk)
    with _alloc_on(stream):
        if o_part is None:
            o_part = torch.empty((B, Hq, S, d), dtype=torch.float32, device=q.device)
        if lse_part is None:
            lse_part = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
    _need("o_part", o_part, (B, Hq, S, d), torch.float32, q.device)
    _need("lse_part", lse_part, (B, Hq, S), torch.float32, q.device)
    _check(load_library().ra_fwd_step(plan.handle, int(step), _ptr(q), _ptr(k_blk), _ptr(v_blk), _ptr(o_part),
                                      _ptr(lse_part), _stream(stream)))
    return o_part, lse_part


def ra_ring_rotate(plan, k_src, v_src, k_dst=None, v_dst=None, stream=None):
    """Pass every shard's K/V block on to the next shard -> (k_dst, v_dst)."""
    import torch
    _check_qkv(plan, k_src=k_src, v_src=v_src)
    with _alloc_on(stream):
        if k_dst is None:
            k_dst = torch.empty_like(k_src)
        if v_dst is None:
            v_dst = torch.empty_like(v_src)
    _check_qkv(plan, k_dst=k_dst, v_dst=v_dst)
    _same_device(k_src.device, v_src=v_src, k_dst=k_dst, v_dst=v_dst)
    _check(load_library().ra_ring_rotate(plan.handle, _ptr(k_src), _ptr(v_src), _ptr(k_dst), _ptr(v_dst),
                                         _stream(stream)))
    return k_dst, v_dst


def ra_ring_fwd(plan, q, k, v, o=None, lse=None, k_buf=None, v_buf=None, o_parts=None, lse_parts=None,
                stream=None, comm_stream=None):
    """Explicit ring driver: N per-step launches, K/V passed on on ``comm_stream``, then a merge.

    Returns (O, LSE).  Scratch (two receive buffers for K and V, the N float32
    partials) is allocated here unless passed in; ``comm_stream`` defaults to a
    new stream (pass the compute stream itself to run without overlap).
    """
    import torch
    pb = plan.problem
    B, Hq, S, d, N = pb["batch"], pb["heads_q"], pb["seq"], pb["head_dim"], pb["n_shards"]
    _check_qkv(plan, q=q, k=k, v=v)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, S), dtype=torch.float32, device=q.device)
        if N > 1:
            if k_buf is None:
                k_buf = torch.empty((2,) + tuple(k.shape), dtype=k.dtype, device=k.device)
            if v_buf is None:
                v_buf = torch.empty((2,) + tuple(v.shape), dtype=v.dtype, device=v.device)
        if o_parts is None:
            o_parts = torch.empty((N, B, Hq, S, d), dtype=torch.float32, device=q.device)
        if lse_parts is None:
            lse_parts = torch.empty((N, B, Hq, S), dtype=torch.float32, device=q.device)
    _same_device(q.device, k=k, v=v)
    _need("o", o, q.shape, q.dtype, q.device)
    _need("lse", lse, (B, Hq, S), torch.float32, q.device)
    if N > 1:
        _need("k_buf", k_buf, (2,) + tuple(k.shape), k.dtype, q.device)
        _need("v_buf", v_buf, (2,) + tuple(v.shape), v.dtype, q.device)
    _need("o_parts", o_parts, (N, B, Hq, S, d), torch.float32, q.device)
    _need("lse_parts", lse_parts, (N, B, Hq, S), torch.float32, q.device)
    if comm_stream is None:
        comm_stream = torch.cuda.Stream(device=q.device)
    _check(load_library().ra_ring_fwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(k_buf),
                                      _ptr(v_buf), _ptr(o_parts), _ptr(lse_parts), _stream(stream),
                                      _stream(comm_stream)))
    return o, lse


def ra_bwd(plan, q, k, v, o, lse, dout, dq=None, dk=None, dv=None, scratch=None, stream=None):
    """Gradients (dQ, dK, dV) of the forward for the upstream gradient ``dout``.

    ``o`` and ``lse`` are the forward's outputs for the same q, k, v; ``scratch``
    (``ra_bwd_scratch_size`` bytes, float32) is allocated here unless passed in.
    """
    torch = _TORCH or _torch()
    pb = plan.problem
    B, Hq, S = pb["batch"], pb["heads_q"], pb["seq"]
    _check_qkv(plan, q=q, k=k, v=v)
    _check_qkv(plan, q=o)
    _check_qkv(plan, q=dout)
    if dq is not None:
        _need_like("dq", dq, q.shape, q.dtype, q.device)
    if dk is not None:
        _need_like("dk", dk, k.shape, k.dtype, k.device)
    if dv is not None:
        _need_like("dv", dv, v.shape, v.dtype, v.device)
    if scratch is not None and (scratch.numel() * scratch.element_size() < ra_bwd_scratch_size(plan)
                                or scratch.dtype != torch.float32 or not scratch.is_contiguous()
                                or scratch.device != q.device):
        raise ValueError("scratch must be a contiguous float32 tensor of at least ra_bwd_scratch_size(plan) "
                         "bytes on the device of q")
    with _alloc_on(stream):
        if dq is None:
            dq = torch.empty_like(q)
        if dk is None:
            dk = torch.empty_like(k)
        if dv is None:
            dv = torch.empty_like(v)
        if scratch is None:
            scratch = torch.empty(ra_bwd_scratch_size(plan) // 4, dtype=torch.float32, device=q.device)
    _need_like("lse", lse, (B, Hq, S), torch.float32, q.device)
    _check(load_library().ra_bwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                 _ptr(dq), _ptr(dk), _ptr(dv), _ptr(scratch), _stream(stream)))
    return dq, dk, dv


def ra_bwd_scratch_size(plan):
    """Bytes of the float32 scratch buffer ra_bwd needs for this plan."""
    if plan._bwd_scratch is None:
        n = ctypes.c_int64()
        _check(load_library().ra_bwd_scratch_size(plan.handle, ctypes.byref(n)))
        plan._bwd_scratch = n.value
    return plan._bwd_scratch


def ra_allgather_kv(plan, k, v, k_all=None, v_all=None, stream=None):
    """Gather every shard's K/V block into one natural-order copy -> (k_all, v_all)."""
    import torch
    _check_qkv(plan, k=k, v=v)
    with _alloc_on(stream):
        if k_all is None:
            k_all = torch.empty_like(k)
        if v_all is None:
            v_all = torch.empty_like(v)
    _check_qkv(plan, k_all=k_all, v_all=v_all)
    _same_device(k.device, v=v, k_all=k_all, v_all=v_all)
    _check(load_library().ra_allgather_kv(plan.handle, _ptr(k), _ptr(v), _ptr(k_all), _ptr(v_all),
                                          _stream(stream)))
    return k_all, v_all


def ra_fwd_gathered(plan, q, k_all, v_all, o=None, lse=None, stream=None):
    """Forward of the all-gather variant: layout-order q against natural-order K/V -> (O, LSE)."""
    import torch
    pb = plan.problem
    _check_qkv(plan, q=q, k_all=k_all, v_all=v_all)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((pb["batch"], pb["heads_q"], pb["seq"]), dtype=torch.float32, device=q.device)
    _same_device(q.device, k_all=k_all, v_all=v_all)
    _need("o", o, q.shape, q.dtype, q.device)
    _need("lse", lse, (pb["batch"], pb["heads_q"], pb["seq"]), torch.float32, q.device)
    _check(load_library().ra_fwd_gathered(plan.handle, _ptr(q), _ptr(k_all), _ptr(v_all), _ptr(o), _ptr(lse),
                                          _stream(stream)))
    return o, lse


def ra_ulysses_a2a(x, layout, n_shards, direction, out=None, stream=None):
    """Ulysses' exchange.  direction 0: [B, H, S, ...] layout order -> [N, B, H/N, S, ...];
    direction 1: back.  Rows are d = 128 bf16 ([..., 128]) or one float32 ([...])."""
    import torch
    if not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous CUDA tensor")
    N = int(n_shards)
    if direction == 0:
        B, H, S = x.shape[:3]
        if N < 1 or H % N:
            raise ValueError("the head count must be a multiple of n_shards")
        out_shape = (N, B, H // N, S) + tuple(x.shape[3:])
    else:
        n_, B, hl, S = x.shape[:4]
        if n_ != N:
            raise ValueError(f"x must have n_shards = {N} head shards on its first axis")
        H = hl * N
        out_shape = (B, H, S) + tuple(x.shape[4:])
    row_bytes = int(np.prod(x.shape[3 if direction == 0 else 4:], dtype=np.int64)) * x.element_size()
    if out is None:
        with _alloc_on(stream):
            out = torch.empty(out_shape, dtype=x.dtype, device=x.device)
    _need("out", out, out_shape, x.dtype, x.device)
    _check(load_library().ra_ulysses_a2a(int(direction), _layout(layout), int(S), N, int(B), int(H), row_bytes,
                                         _ptr(x), _ptr(out), _stream(stream)))
    return out


class Kv4:
    """Owns an ``ra_kv4_t``; the cache it was described for is ``self.problem``."""

    def __init__(self, handle, problem):
        self._h = handle
        self.problem = problem
        self._bytes = None    # of the cache
        self._scratch = (None, 0)  # (batch, rows, table width) of the last attention call, its bytes of scratch

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load_library().ra_kv4_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ra_kv4_plan(pages, page_rows, heads_q, heads_kv, head_dim, dtype="bf16", window=0, sinks=0, scale=0.0):
    """Describe a paged 4-bit key/value cache and the attention over it (see include/ra.h)."""
    lib = load_library()
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    prob = _Kv4Problem(int(pages), int(page_rows), int(heads_q), int(heads_kv), int(head_dim), dt, int(window),
                       int(sinks), float(scale or 0.0))
    h = ctypes.c_void_p()
    _check(lib.ra_kv4_plan(ctypes.byref(prob), ctypes.byref(h)))
    info = dict(pages=int(pages), page_rows=int(page_rows), heads_q=int(heads_q), heads_kv=int(heads_kv),
                head_dim=int(head_dim), dtype=dt, window=int(window), sinks=int(sinks), scale=float(scale or 0.0))
    return Kv4(h, info)


def ra_kv4_destroy(kv):
    kv.close()


def ra_kv4_cache_size(kv):
    """Bytes of the cache buffer (a contiguous uint8 CUDA tensor of the caller's)."""
    if kv._bytes is None:
        n = ctypes.c_int64()
        _check(load_library().ra_kv4_cache_size(kv.handle, ctypes.byref(n)))
        kv._bytes = n.value
    return kv._bytes


def _kv4_dtype(kv):
    torch = _TORCH or _torch()
    return torch.bfloat16 if kv.problem["dtype"] == 1 else torch.float32


def _kv4_tables(kv, cache, batch, page_table, name, table, count=None):
    """The cache, the page table and the [batch] int32 tables of a call, all on one device, which
    is returned."""
    torch = _TORCH or _torch()
    device, i32 = cache.device, torch.int32
    _need("cache", cache, (kv._bytes or ra_kv4_cache_size(kv),), torch.uint8, device)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError(f"page_table must be an int32 tensor of shape ({batch}, pages of a sequence)")
    _need_like("page_table", page_table, page_table.shape, i32, device)
    _need_like(name, table, (batch,), i32, device)
    if count is not None:
        _need_like("count", count, (batch,), i32, device)
    return device


def ra_kv4_write(kv, cache, k, v, page_table, first, count=None, stream=None):
    """Quantise rows k, v [B, Hkv, T, d] into the cache at positions first[b] + t, t < count[b]."""
    pb = kv.problem
    B, T = (k.shape[0], k.shape[2]) if k.dim() == 4 else (0, 0)
    device, dtype = _kv4_tables(kv, cache, B, page_table, "first", first, count), _kv4_dtype(kv)
    shape = (B, pb["heads_kv"], T, pb["head_dim"])
    _need_like("k", k, shape, dtype, device)
    _need_like("v", v, shape, dtype, device)
    _check(load_library().ra_kv4_write(kv.handle, _ptr(cache), B, T, _ptr(k), _ptr(v), _ptr(page_table),
                                       page_table.shape[1], _ptr(first), _ptr(count), _stream(stream)))


def ra_kv4_read(kv, cache, page_table, first, rows, count=None, k=None, v=None, stream=None):
    """Rows [B, Hkv, rows, d] of the cache as the values they stand for -> (k, v).

    Rows from count[b] on stay as they were in k and v that are passed in (both or
    neither); they are zeros where k and v are allocated here.
    """
    torch = _TORCH or _torch()
    pb = kv.problem
    B, T = page_table.shape[0], int(rows)
    device, dtype = _kv4_tables(kv, cache, B, page_table, "first", first, count), _kv4_dtype(kv)
    shape = (B, pb["heads_kv"], T, pb["head_dim"])
    if (k is None) != (v is None):
        raise ValueError("pass both k and v, or neither")
    own = k is None
    if own:
        with _alloc_on(stream):
            k = torch.empty(shape, dtype=dtype, device=device)
            v = torch.empty_like(k)
    else:
        _need_like("k", k, shape, dtype, device)
        _need_like("v", v, shape, dtype, device)
    _check(load_library().ra_kv4_read(kv.handle, _ptr(cache), B, T, _ptr(page_table), page_table.shape[1],
                                      _ptr(first), _ptr(count), int(own), _ptr(k), _ptr(v), _stream(stream)))
    return k, v


def ra_kv4_attend_scratch_size(kv, batch, rows, table_width):
    """Bytes of the float32 scratch buffer ra_kv4_attend needs for these sizes (0: none)."""
    key = (int(batch), int(rows), int(table_width))
    if kv._scratch[0] != key:
        n = ctypes.c_int64()
        _check(load_library().ra_kv4_attend_scratch_size(kv.handle, *key, ctypes.byref(n)))
        kv._scratch = (key, n.value)
    return kv._scratch[1]


def ra_kv4_attend(kv, cache, q, page_table, length, o=None, lse=None, scratch=None, stream=None):
    """Attention of the last T tokens q [B, Hq, T, d] of every sequence over the cache -> (O, LSE).

    length[b] counts the tokens of sequence b in the cache, the T new ones among them.
    ``scratch`` (``ra_kv4_attend_scratch_size`` bytes, float32) is allocated here unless
    passed in.
    """
    torch = _TORCH or _torch()
    pb = kv.problem
    if q.dim() != 4:
        raise ValueError("q must have the shape [B, Hq, T, d]")
    B, Hq, T, d = q.shape
    device = _kv4_tables(kv, cache, B, page_table, "length", length)
    _need_like("q", q, (B, pb["heads_q"], T, pb["head_dim"]), _kv4_dtype(kv), device)
    need = ra_kv4_attend_scratch_size(kv, B, T, page_table.shape[1]) // 4
    if scratch is not None and (scratch.numel() < need or scratch.dtype != torch.float32
                                  or not scratch.is_contiguous() or scratch.device != device):
        raise ValueError("scratch must be a contiguous float32 tensor of at least ra_kv4_attend_scratch_size(...) "
                         "bytes on the device of q")
    if o is not None:
        _need_like("o", o, q.shape, q.dtype, device)
    if lse is not None:
        _need_like("lse", lse, (B, Hq, T), torch.float32, device)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, Hq, T), dtype=torch.float32, device=device)
        if scratch is None and need:
            scratch = torch.empty(need, dtype=torch.float32, device=device)
    _check(load_library().ra_kv4_attend(kv.handle, _ptr(cache), B, T, _ptr(q), _ptr(page_table), page_table.shape[1],
                                        _ptr(length), _ptr(o), _ptr(lse), _ptr(scratch), _stream(stream)))
    return o, lse


def ra_kv4_sync_status(kv, stream=None):
    """Synchronize the stream and raise RaError if a call met a page index, position, length
    or count out of range."""
    _check(load_library().ra_kv4_sync_status(kv.handle, _stream(stream)))


class Rope:
    """Owns an ``ra_rope_t``; the rotation it was described for is ``self.problem``."""

    def __init__(self, handle, problem):
        self._h = handle
        self.problem = problem
        self.dtype = _torch().bfloat16 if problem["dtype"] == 1 else _torch().float32

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load_library().ra_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ra_rope_plan(head_dim, rotary_dim=0, base=10000.0, interleaved=False, scaling="none", factor=1.0, original=0,
                 low=1.0, high=4.0, amplitude=1.0, dtype="bf16"):
    """Describe a rotation by positions (see include/ra.h); rotary_dim 0 is the whole head.

    ``scaling``: "none", "linear", "base", "bands" or "ramp", for contexts ``factor`` times
    longer than the ``original`` tokens; ``low`` and ``high`` are turns within those.
    """
    lib = load_library()
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    kind = ROPE_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    if not amplitude > 0:
        raise ValueError("amplitude must be > 0")
    prob = _RopeProblem(int(head_dim), int(rotary_dim) or int(head_dim), int(bool(interleaved)), dt, float(base), kind,
                        float(factor), int(original), float(low), float(high), float(amplitude))
    h = ctypes.c_void_p()
    _check(lib.ra_rope_plan(ctypes.byref(prob), ctypes.byref(h)))
    info = dict(head_dim=prob.head_dim, rotary_dim=prob.rotary_dim, interleaved=bool(interleaved), dtype=dt,
                base=float(base), scaling=kind, factor=float(factor), original=int(original), low=float(low),
                high=float(high), amplitude=float(amplitude))
    return Rope(h, info)


def ra_rope_destroy(rope):
    rope.close()


_ARRAYS = {}  # strides -> the host array that the library takes


def _array(*strides):
    a = _ARRAYS.get(strides)
    if a is None:
        if len(_ARRAYS) > 4096:
            _ARRAYS.clear()
        a = _ARRAYS[strides] = (ctypes.c_int64 * len(strides))(*strides)
    return a


def _new_like(t):
    """A contiguous tensor of t's shape and type."""
    return _TORCH.empty_like(t, memory_format=_TORCH.contiguous_format)


def _bad_rows(name, shape, dtype, device):
    return ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}, contiguous along its last axis")


def _rows4(name, t, shape, dtype, device):
    """Strides of ``t`` along its first three axes as a host array (0 along an axis of one), once it
    is a tensor of this shape, dtype and device (checked already), its last axis contiguous."""
    if not isinstance(t, _TORCH.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device:
        raise _bad_rows(name, shape, dtype, device)
    a, b, c, e = t.stride()
    if e != 1 and shape[3] > 1:
        raise _bad_rows(name, shape, dtype, device)
    return _array(a if shape[0] > 1 else 0, b if shape[1] > 1 else 0, c if shape[2] > 1 else 0)


def _rows3(name, t, shape, dtype, device):
    """As _rows4, of a packed tensor."""
    if not isinstance(t, _TORCH.Tensor) or t.shape != shape or t.dtype != dtype or t.device != device:
        raise _bad_rows(name, shape, dtype, device)
    a, b, e = t.stride()
    if e != 1 and shape[2] > 1:
        raise _bad_rows(name, shape, dtype, device)
    return _array(a if shape[0] > 1 else 0, b if shape[1] > 1 else 0)


def _rope_call(call, rope, q, k, layout, n_shards, position, q_out, k_out, stream):
    torch = _TORCH or _torch()
    d, dtype = rope.problem["head_dim"], rope.dtype
    if q.dim() != 4:
        raise ValueError("q must have the shape [B, Hq, S, d]")
    B, Hq, S, _ = q.shape
    device, shape = q.device, (B, Hq, S, d)
    qs = _rows4("q", q, shape, dtype, device)
    _on_current_device("q", q)
    if position is not None:
        _need_like("position", position, (B, S), torch.int32, device)
    if q_out is None:
        with _alloc_on(stream):
            q_out = _new_like(q)
        qos = _array(Hq * S * d, S * d, d)
    else:
        qos = _rows4("q_out", q_out, shape, dtype, device)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        _check(call(rope.handle, B, S, Hq, 0, _layout(layout), int(n_shards), _ptr(position), q.data_ptr(), qs, None, None,
                    q_out.data_ptr(), qos, None, None, _stream(stream)))
        return q_out
    Hk = k.shape[1] if k.dim() == 4 else 0
    shape = (B, Hk, S, d)
    ks = _rows4("k", k, shape, dtype, device)
    if k_out is None:
        with _alloc_on(stream):
            k_out = _new_like(k)
        kos = _array(Hk * S * d, S * d, d)
    else:
        kos = _rows4("k_out", k_out, shape, dtype, device)
    _check(call(rope.handle, B, S, Hq, Hk, _layout(layout), int(n_shards), _ptr(position), q.data_ptr(), qs, k.data_ptr(), ks,
                q_out.data_ptr(), qos, k_out.data_ptr(), kos, _stream(stream)))
    return q_out, k_out


def ra_rope(rope, q, k=None, layout="contiguous", n_shards=1, position=None, q_out=None, k_out=None, stream=None):
    """Rotate q [B, Hq, S, d] and k [B, Hkv, S, d] by their positions -> (q_out, k_out), or q_out without k.

    Row i of shard p stands at its natural position of the layout, unless ``position``
    [B, S] int32 gives them.  All tensors may have strides of their own; the outputs are
    contiguous unless passed in, and may be the inputs themselves.
    """
    return _rope_call(load_library().ra_rope, rope, q, k, layout, n_shards, position, q_out, k_out, stream)


def ra_rope_bwd(rope, dq, dk=None, layout="contiguous", n_shards=1, position=None, q_out=None, k_out=None, stream=None):
    """Gradients with respect to ra_rope's inputs from those with respect to its outputs."""
    return _rope_call(load_library().ra_rope_bwd, rope, dq, dk, layout, n_shards, position, q_out, k_out, stream)


class Paged:
    """Owns an ``ra_paged_t``; the cache it was described for is ``self.problem``."""

    def __init__(self, handle, problem):
        self._h = handle
        self.problem = problem
        pb = problem
        self.dtype = _torch().bfloat16 if pb["dtype"] == 1 else _torch().float32
        self._shape = (pb["pages"], 2, pb["heads_kv"], pb["page_rows"], pb["head_dim"])
        # (batch, tokens, table width) of the last call, its bytes of scratch: attention's, the weights'
        self._scratch, self._weigh_scratch = (None, 0), (None, 0)

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            load_library().ra_paged_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def ra_paged_plan(pages, page_rows, heads_q, heads_kv, head_dim, dtype="bf16", window=0, sinks=0, scale=0.0):
    """Describe a paged key/value cache and the attention over it (see include/ra.h)."""
    lib = load_library()
    dt = DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    prob = _PagedProblem(int(pages), int(page_rows), int(heads_q), int(heads_kv), int(head_dim), dt, int(window),
                         int(sinks), float(scale or 0.0))
    h = ctypes.c_void_p()
    _check(lib.ra_paged_plan(ctypes.byref(prob), ctypes.byref(h)))
    info = dict(pages=int(pages), page_rows=int(page_rows), heads_q=int(heads_q), heads_kv=int(heads_kv),
                head_dim=int(head_dim), dtype=dt, window=int(window), sinks=int(sinks), scale=float(scale or 0.0))
    return Paged(h, info)


def ra_paged_destroy(kv):
    kv.close()


def ra_paged_cache_shape(kv):
    """Shape of the cache, a contiguous CUDA tensor of the caller's in the handle's dtype:
    [pages, keys and values, Hkv, page_rows, d]."""
    return kv._shape


def _paged_tables(kv, cache, page_table, length, offset=None):
    """The cache and the int32 tables of a call, all on one device -> (dtype, device, batch)."""
    torch = _TORCH or _torch()
    dtype, device, i32 = kv.dtype, cache.device, torch.int32
    _need("cache", cache, kv._shape, dtype, device)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 tensor of shape (sequences, pages of a sequence)")
    batch, width = page_table.shape
    _need_like("page_table", page_table, (batch, width), i32, device)
    _need_like("length", length, (batch,), i32, device)
    if offset is not None:
        _need_like("offset", offset, (batch + 1,), i32, device)
    return dtype, device, batch, width


def ra_paged_append(kv, cache, k, v, page_table, offset, length, rope=None, position=None, q=None, q_out=None,
                    stream=None):
    """New tokens' keys and values k, v [tokens, Hkv, d] into the cache -> q_out (None without q).

    Sequence b has the tokens offset[b] .. offset[b+1]-1 and length[b] slots in use, those
    among them.  With ``rope`` the keys, and the queries q [tokens, Hq, d], are rotated by
    ``position`` [tokens] (default: the tokens' slots) on the way.
    """
    torch = _TORCH or _torch()
    pb = kv.problem
    dtype, device, batch, width = _paged_tables(kv, cache, page_table, length, offset)
    T, d = k.shape[0] if k.dim() == 3 else 0, pb["head_dim"]
    shape = (T, pb["heads_kv"], d)
    ks, vs = _rows3("k", k, shape, dtype, device), _rows3("v", v, shape, dtype, device)
    if position is not None:
        _need_like("position", position, (T,), torch.int32, device)
    qs = qos = None
    if q is not None:
        shape = (T, pb["heads_q"], d)
        qs = _rows3("q", q, shape, dtype, device)
        if q_out is None:
            with _alloc_on(stream):
                q_out = _new_like(q)
        qos = _rows3("q_out", q_out, shape, dtype, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check(load_library().ra_paged_append(
        kv.handle, None if rope is None else rope.handle, cache.data_ptr(), batch, T, k.data_ptr(), ks, v.data_ptr(), vs,
        _ptr(q), qs, _ptr(q_out), qos, page_table.data_ptr(), width, offset.data_ptr(), length.data_ptr(), _ptr(position),
        _stream(stream)))
    return q_out


def ra_paged_attend_scratch_size(kv, batch, tokens, table_width):
    """Bytes of the float32 scratch buffer ra_paged_attend needs for these sizes (0: none)."""
    key = (int(batch), int(tokens), int(table_width))
    if kv._scratch[0] != key:
        n = ctypes.c_int64()
        _check(load_library().ra_paged_attend_scratch_size(kv.handle, *key, ctypes.byref(n)))
        kv._scratch = (key, n.value)
    return kv._scratch[1]


def ra_paged_attend(kv, cache, q, page_table, offset, length, o=None, lse=None, scratch=None, stream=None):
    """Attention of the new tokens q [tokens, Hq, d] over their sequences' slots -> (O, LSE [tokens, Hq]).

    ``scratch`` (``ra_paged_attend_scratch_size`` bytes, float32) is allocated here unless
    passed in.  Rows of no sequence stay as they were (in tensors made here: undefined).
    """
    torch = _TORCH or _torch()
    pb = kv.problem
    dtype, device, batch, width = _paged_tables(kv, cache, page_table, length, offset)
    T = q.shape[0] if q.dim() == 3 else 0
    shape = (T, pb["heads_q"], pb["head_dim"])
    qs = _rows3("q", q, shape, dtype, device)
    need = ra_paged_attend_scratch_size(kv, batch, T, width) // 4
    if scratch is not None:
        _need_scratch("ra_paged_attend_scratch_size", scratch, need, device)
    if lse is not None:
        _need_like("lse", lse, (T, pb["heads_q"]), torch.float32, device)
    with _alloc_on(stream):
        if o is None:
            o = _new_like(q)
        if lse is None:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=device)
        if scratch is None and need:
            scratch = torch.empty(need, dtype=torch.float32, device=device)
    os = _rows3("o", o, shape, dtype, device)
    _check(load_library().ra_paged_attend(kv.handle, cache.data_ptr(), batch, T, q.data_ptr(), qs, page_table.data_ptr(), width,
                                          offset.data_ptr(), length.data_ptr(), o.data_ptr(), os, lse.data_ptr(),
                                          _ptr(scratch), _stream(stream)))
    return o, lse


def _need_weights(name, t, kv, batch, device):
    torch = _TORCH or _torch()
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a float32 tensor of shape (sequences, Hkv, slots)")
    _need_like(name, t, (batch, kv.problem["heads_kv"], t.shape[2]), torch.float32, device)


def ra_paged_weigh_scratch_size(kv, batch, tokens, table_width):
    """Bytes of the float32 scratch buffer ra_paged_weigh needs for these sizes (0: none)."""
    key = (int(batch), int(tokens), int(table_width))
    if kv._weigh_scratch[0] != key:
        n = ctypes.c_int64()
        _check(load_library().ra_paged_weigh_scratch_size(kv.handle, *key, ctypes.byref(n)))
        kv._weigh_scratch = (key, n.value)
    return kv._weigh_scratch[1]


def _need_scratch(name, scratch, need, device):
    if (scratch.numel() < need or scratch.dtype != (_TORCH or _torch()).float32 or not scratch.is_contiguous()
            or scratch.device != device):
        raise ValueError(f"scratch must be a contiguous float32 tensor of at least {name}(...) bytes on {device}")


def ra_paged_weigh(kv, cache, q, lse, page_table, offset, length, weight, weight_in=None, scratch=None, stream=None):
    """Attention weight of every slot from the new tokens, added to ``weight_in`` (default: zeros) -> weight.

    weight, weight_in: [sequences, Hkv, slots] float32, and may be one tensor; the slots of the
    call's own tokens start from zero.  lse: what ra_paged_attend returned for q.
    """
    torch = _TORCH or _torch()
    pb = kv.problem
    dtype, device, batch, width = _paged_tables(kv, cache, page_table, length, offset)
    T = q.shape[0] if q.dim() == 3 else 0
    qs = _rows3("q", q, (T, pb["heads_q"], pb["head_dim"]), dtype, device)
    _need_like("lse", lse, (T, pb["heads_q"]), torch.float32, device)
    _need_weights("weight", weight, kv, batch, device)
    if weight_in is not None:
        _need_like("weight_in", weight_in, weight.shape, torch.float32, device)
    need = ra_paged_weigh_scratch_size(kv, batch, T, width) // 4
    if scratch is not None:
        _need_scratch("ra_paged_weigh_scratch_size", scratch, need, device)
    elif need:
        with _alloc_on(stream):
            scratch = torch.empty(need, dtype=torch.float32, device=device)
    _check(load_library().ra_paged_weigh(kv.handle, cache.data_ptr(), batch, T, q.data_ptr(), qs, lse.data_ptr(),
                                         page_table.data_ptr(), width, offset.data_ptr(), length.data_ptr(), _ptr(weight_in),
                                         weight.data_ptr(), weight.shape[2], _ptr(scratch), _stream(stream)))
    return weight


def ra_paged_evict(kv, cache, page_table, length, weight, keep, first=0, recent=0, new_table=None, weight_out=None,
                   kept=None, new_length=None, stream=None):
    """Keep ``keep`` slots of every sequence and head: the first, the most recent, the heaviest -> (kept, new_length).

    The slots that stay move together, in place or into the pages of ``new_table``;
    weight_out (default: weight itself) receives their weights.
    kept: [sequences, Hkv, keep] int32, the slots they had (-1: none).
    """
    torch = _TORCH or _torch()
    _, device, batch, width = _paged_tables(kv, cache, page_table, length)
    _need_weights("weight", weight, kv, batch, device)
    if weight_out is None:
        weight_out = weight
    else:
        _need_like("weight_out", weight_out, weight.shape, torch.float32, device)
    if new_table is None:
        new_table = page_table
    elif not isinstance(new_table, torch.Tensor) or new_table.dim() != 2:
        raise ValueError("new_table must be an int32 tensor of shape (sequences, pages of a sequence)")
    else:
        _need_like("new_table", new_table, (batch, new_table.shape[1]), torch.int32, device)
    keep, hk = int(keep), kv.problem["heads_kv"]
    if kept is not None:
        _need_like("kept", kept, (batch, hk, keep), torch.int32, device)
    if new_length is not None:
        _need_like("new_length", new_length, (batch,), torch.int32, device)
    if kept is None or new_length is None:
        with _alloc_on(stream):
            if kept is None:
                kept = torch.empty((batch, hk, max(keep, 0)), dtype=torch.int32, device=device)
            if new_length is None:
                new_length = torch.empty((batch,), dtype=torch.int32, device=device)
    _check(load_library().ra_paged_evict(kv.handle, _ptr(cache), batch, _ptr(page_table), width, _ptr(length),
                                         _ptr(weight), _ptr(weight_out), weight.shape[2], keep, int(first), int(recent),
                                         _ptr(new_table), new_table.shape[1], _ptr(kept), _ptr(new_length), _stream(stream)))
    return kept, new_length


def ra_paged_sync_status(kv, stream=None):
    """Synchronize the stream and raise RaError if a call met a page index, offset, length or
    slot out of range."""
    _check(load_library().ra_paged_sync_status(kv.handle, _stream(stream)))
