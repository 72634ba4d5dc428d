"""Python binding of libds4moe, the routed MoE FFN of a DeepSeek-V4-Flash layer
on GB300 (sm_103a).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. PyTorch supplies device memory and streams. There is no CPU fallback:
if the compiled library cannot be loaded, importing the binding fails.

Entry points mirror the C ABI in include/ds4moe.h:
``Layer(desc, weights)`` = ds4moe_create, ``Layer.route`` = ds4moe_route,
``Layer.forward`` = ds4moe_forward, ``Layer.forward_rmsnorm`` =
ds4moe_forward_rmsnorm, ``Layer.forward_host`` = ds4moe_forward_host,
``rmsnorm`` = ds4moe_rmsnorm, ``route_noalloc`` =
ds4moe_route_noalloc, ``Dense`` = the ds4moe_dense_* calls, ``Attention`` (with
``AttentionDesc`` and ``KVCache``) = ds4moe_attn_* and ds4moe_kv_append,
``token_probs`` = ds4moe_token_probs, ``verify_drafts`` = ds4moe_verify_drafts.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

from . import build as _build

ABI_VERSION = 1
F32, Q8_0, Q2S, Q4S = 0, 1, 2, 3
FMT = {"f32": F32, "q8_0": Q8_0, "q2s": Q2S, "q4s": Q4S}
ROUTE_LEARNED, ROUTE_HASH = 0, 1
STATUS = {0: "OK", 1: "ERR_INVALID_ARG", 2: "ERR_UNSUPPORTED", 3: "ERR_OOM", 4: "ERR_CUDA", 5: "ERR_DEVICE"}
DEVERR_TOKEN_ID, DEVERR_NONFINITE, DEVERR_TIMEOUT, DEVERR_INTERNAL, DEVERR_PAGE, DEVERR_LENGTH = 1, 2, 4, 8, 16, 32
DT_F32, DT_BF16, DT_F16 = 0, 1, 2
DTYPE = {"fp32": DT_F32, "bf16": DT_BF16, "fp16": DT_F16}
ATTN_MAX_NEW, MAX_DRAFT = 16, 64

LIB_PATH = _build.LIB


class Ds4MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class _Desc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("ffn", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("route", ctypes.c_int32), ("vocab", ctypes.c_int32), ("router_fmt", ctypes.c_int32),
                ("routed_fmt", ctypes.c_int32), ("shared_fmt", ctypes.c_int32), ("route_scale", ctypes.c_float),
                ("max_tokens", ctypes.c_int32)]


class _Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("router_w", "router_bias", "hash_table", "gate", "up", "down", "sh_gate", "sh_up", "sh_down")]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("window", ctypes.c_int32),
                ("n_sink", ctypes.c_int32), ("scale", ctypes.c_float), ("max_seqs", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("k_page_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("v_row_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_lib = None


def lib():
    """Load libds4moe.so (building it in-tree first if it is missing or stale)."""
    global _lib
    if _lib is None:
        if _build.stale():
            _build.build()
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libds4moe.so not found at {LIB_PATH}")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, u32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64
        sigs = {
            "ds4moe_create": (i32, [ctypes.POINTER(_Desc), ctypes.POINTER(_Weights), ctypes.POINTER(vp)]),
            "ds4moe_destroy": (None, [vp]),
            "ds4moe_route": (i32, [vp, vp, vp, i32, vp, vp, vp]),
            "ds4moe_route_noalloc": (i32, [ctypes.POINTER(_Desc), ctypes.POINTER(_Weights), vp, vp, i32, vp, vp,
                                           vp, vp]),
            "ds4moe_forward": (i32, [vp, vp, i32, vp, vp, vp]),
            "ds4moe_forward_host": (i32, [vp, vp, i32, vp, vp, vp]),
            "ds4moe_forward_rmsnorm": (i32, [vp, vp, i32, vp, ctypes.c_float, vp, vp]),
            "ds4moe_rmsnorm": (i32, [vp, vp, i32, i32, ctypes.c_float, vp]),
            "ds4moe_get_device_error": (i32, [vp, vp, ctypes.POINTER(u32)]),
            "ds4moe_debug_scratch": (i32, [vp, i32, ctypes.POINTER(vp), ctypes.POINTER(ctypes.c_uint64)]),
            "ds4moe_device_bytes": (ctypes.c_uint64, [vp]),
            "ds4moe_profile_enable": (i32, [vp, i32]),
            "ds4moe_profile_collect": (i32, [vp]),
            "ds4moe_profile_read": (i32, [vp, ctypes.POINTER(ctypes.c_double), i32,
                                          ctypes.POINTER(ctypes.c_int64)]),
            "ds4moe_launch_count": (ctypes.c_uint64, [vp]),
            "ds4moe_debug_set_wait_limit": (i32, [vp, ctypes.c_int64]),
            "ds4moe_debug_fail_alloc": (i32, [i32]),
            "ds4moe_status_string": (ctypes.c_char_p, [i32]),
            "ds4moe_abi_version": (u32, []),
            "ds4moe_dense_create": (i32, [i32, i32, i32, vp, ctypes.POINTER(vp)]),
            "ds4moe_dense_forward": (i32, [vp, vp, i32, vp, vp]),
            "ds4moe_dense_get_device_error": (i32, [vp, vp, ctypes.POINTER(u32)]),
            "ds4moe_dense_destroy": (None, [vp]),
            "ds4moe_dense_device_bytes": (ctypes.c_uint64, [vp]),
            "ds4moe_dense_launch_count": (ctypes.c_uint64, [vp]),
            "ds4moe_dense_debug_config": (i32, [vp, i32, i32, i32, i32]),
            "ds4moe_attn_create": (i32, [ctypes.POINTER(_AttnDesc), ctypes.POINTER(vp)]),
            "ds4moe_attn_destroy": (None, [vp]),
            "ds4moe_kv_append": (i32, [vp, ctypes.POINTER(_KvCache), vp, i64, vp, i64, i32, vp, vp, i32, i32, vp]),
            "ds4moe_attn_decode": (i32, [vp, ctypes.POINTER(_KvCache), vp, i64, vp, i32, i32, vp, i64, vp]),
            "ds4moe_attn_prefill": (i32, [vp, ctypes.POINTER(_KvCache), vp, i64, vp, vp, i32, i32, vp, i64, vp]),
            "ds4moe_attn_get_device_error": (i32, [vp, vp, ctypes.POINTER(u32)]),
            "ds4moe_attn_device_bytes": (ctypes.c_uint64, [vp]),
            "ds4moe_attn_launch_count": (ctypes.c_uint64, [vp]),
            "ds4moe_token_probs": (i32, [vp, i64, i32, i32, ctypes.c_float, vp, i64, vp]),
            "ds4moe_verify_drafts": (i32, [vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]),
        }
        for name, (res, args) in sigs.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        if L.ds4moe_abi_version() != ABI_VERSION:
            raise ImportError("libds4moe ABI version mismatch")
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise Ds4MoeError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        from torch import _C
        # torch.cuda.current_stream() without building a Stream object (a
        # quarter of a small call's host time)
        return ctypes.c_void_p(_C._cuda_getCurrentRawStream(_C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


@dataclass
class LayerDesc:
    hidden: int
    n_experts: int
    top_k: int
    ffn: int
    n_shared: int
    route: int  # ROUTE_LEARNED | ROUTE_HASH
    vocab: int
    router_fmt: int
    routed_fmt: int
    shared_fmt: int
    route_scale: float = 1.0
    max_tokens: int = 1

    def c(self) -> _Desc:
        return _Desc(ABI_VERSION, self.hidden, self.n_experts, self.top_k, self.ffn, self.n_shared, self.route,
                     self.vocab, self.router_fmt, self.routed_fmt, self.shared_fmt, self.route_scale,
                     self.max_tokens)


class _CudaArray:
    """A device buffer described by __cuda_array_interface__ (for torch.as_tensor)."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr, False),
                                         "version": 3, "strides": None}


class Layer:
    """One MoE layer handle (ds4moe_create). `weights` maps the names of
    ds4moe_weights (router_w, router_bias, hash_table, gate, up, down, sh_gate,
    sh_up, sh_down) to CUDA tensors in the canonical byte layouts."""

    def __init__(self, desc: LayerDesc, weights: dict):
        L = lib()
        self.desc = desc
        w = _Weights(*[_ptr(weights.get(n)) for n, _ in _Weights._fields_])
        h = ctypes.c_void_p()
        _check(L.ds4moe_create(ctypes.byref(desc.c()), ctypes.byref(w), ctypes.byref(h)), "ds4moe_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().ds4moe_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def device_bytes(self) -> int:
        return int(lib().ds4moe_device_bytes(self._h))

    STAGES = ("quantize", "route", "bucket", "gateup", "down", "combine")

    def profile(self, on: bool = True):
        """Record CUDA events around every stage of later forwards (ds4moe_profile_enable)."""
        _check(lib().ds4moe_profile_enable(self._h, 1 if on else 0), "ds4moe_profile_enable")

    def profile_collect(self):
        """Wait for the last forward's events and add its stage times (ds4moe_profile_collect)."""
        _check(lib().ds4moe_profile_collect(self._h), "ds4moe_profile_collect")

    def profile_read(self):
        """(per-stage total ms, number of collected calls) (ds4moe_profile_read)."""
        ms = (ctypes.c_double * len(self.STAGES))()
        calls = ctypes.c_int64()
        _check(lib().ds4moe_profile_read(self._h, ms, len(self.STAGES), ctypes.byref(calls)),
               "ds4moe_profile_read")
        return dict(zip(self.STAGES, list(ms))), int(calls.value)

    def launch_count(self) -> int:
        """Kernels launched by this handle since create (ds4moe_launch_count)."""
        return int(lib().ds4moe_launch_count(self._h))

    def forward(self, x, y, token_ids=None, stream=None, n_tok=None):
        """y += MoE(x) on the device (ds4moe_forward)."""
        n = x.shape[0] if n_tok is None else n_tok
        _check(lib().ds4moe_forward(self._h, _ptr(x), n, _ptr(token_ids), _ptr(y), _stream(stream)),
               "ds4moe_forward")

    def forward_rmsnorm(self, x, y, eps: float = 1e-6, token_ids=None, stream=None, n_tok=None):
        """y += MoE(RMSNorm(x)) on the device (ds4moe_forward_rmsnorm); y may be x."""
        n = x.shape[0] if n_tok is None else n_tok
        _check(lib().ds4moe_forward_rmsnorm(self._h, _ptr(x), n, _ptr(token_ids), eps, _ptr(y), _stream(stream)),
               "ds4moe_forward_rmsnorm")

    def forward_host(self, x, y, token_ids=None, stream=None):
        """y += MoE(x) on host tensors (ds4moe_forward_host; synchronises)."""
        _check(lib().ds4moe_forward_host(self._h, _ptr(x), x.shape[0], _ptr(token_ids), _ptr(y),
                                         _stream(stream)), "ds4moe_forward_host")

    def route(self, x=None, token_ids=None, ids_out=None, w_out=None, stream=None, n_tok=None):
        """Expert ids and weights (ds4moe_route). Returns (ids_out, w_out)."""
        import torch
        n = n_tok if n_tok is not None else (x.shape[0] if x is not None else token_ids.shape[0])
        dev = (x if x is not None else token_ids).device
        if ids_out is None:
            ids_out = torch.empty((n, self.desc.top_k), dtype=torch.int32, device=dev)
        if w_out is None:
            w_out = torch.empty((n, self.desc.top_k), dtype=torch.float32, device=dev)
        _check(lib().ds4moe_route(self._h, _ptr(x), _ptr(token_ids), n, _ptr(ids_out), _ptr(w_out),
                                  _stream(stream)), "ds4moe_route")
        return ids_out, w_out

    def set_wait_limit(self, cycles: int):
        """Bound of the decode expert kernels' hand-off waits, in SM cycles
        (0: the default); a test hook (ds4moe_debug_set_wait_limit)."""
        _check(lib().ds4moe_debug_set_wait_limit(self._h, int(cycles)), "ds4moe_debug_set_wait_limit")

    def device_error(self, stream=None) -> int:
        """Synchronise, read and clear the device error flags (0 = none)."""
        f = ctypes.c_uint32(0)
        st = lib().ds4moe_get_device_error(self._h, _stream(stream), ctypes.byref(f))
        if st not in (0, 5):
            raise Ds4MoeError(st, "ds4moe_get_device_error")
        return int(f.value)

    _SCRATCH = {"xq": (0, "|i1"), "dx": (1, "<f4"), "gs": (2, "<i2"), "ids": (3, "<i4"), "w": (4, "<f4"),
                "hq": (5, "|i1"), "dh": (6, "<f4"), "a": (7, "<f4")}

    def scratch(self, name: str):
        """Torch view (treat as read-only) of an intermediate buffer (ds4moe_debug_scratch), flat."""
        import torch
        which, typestr = self._SCRATCH[name]
        p, n = ctypes.c_void_p(), ctypes.c_uint64()
        _check(lib().ds4moe_debug_scratch(self._h, which, ctypes.byref(p), ctypes.byref(n)), "ds4moe_debug_scratch")
        itemsize = int(typestr[2:])
        return torch.as_tensor(_CudaArray(p.value, (n.value // itemsize,), typestr), device="cuda")


class Dense:
    """A dense Q8_0 matrix beside the MoE (ds4moe_dense_create): `w` is the
    canonical [n_out][n_in] Q8_0 matrix as a CUDA uint8 tensor."""

    def __init__(self, n_out: int, n_in: int, w, max_tokens: int = 1):
        L = lib()
        h = ctypes.c_void_p()
        _check(L.ds4moe_dense_create(n_out, n_in, max_tokens, _ptr(w), ctypes.byref(h)), "ds4moe_dense_create")
        self._h, self.n_out, self.n_in = h, n_out, n_in

    def close(self):
        if getattr(self, "_h", None):
            lib().ds4moe_dense_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, y=None, stream=None, n_tok=None):
        """y = W x (ds4moe_dense_forward); returns y."""
        import torch
        n = x.shape[0] if n_tok is None else n_tok
        if y is None:
            y = torch.empty((n, self.n_out), dtype=torch.float32, device=x.device)
        _check(lib().ds4moe_dense_forward(self._h, _ptr(x), n, _ptr(y), _stream(stream)), "ds4moe_dense_forward")
        return y

    def device_error(self, stream=None) -> int:
        f = ctypes.c_uint32(0)
        st = lib().ds4moe_dense_get_device_error(self._h, _stream(stream), ctypes.byref(f))
        if st not in (0, 5):
            raise Ds4MoeError(st, "ds4moe_dense_get_device_error")
        return int(f.value)

    def launch_count(self) -> int:
        return int(lib().ds4moe_dense_launch_count(self._h))

    def debug_config(self, ks=0, nst=0, ns=0, tc=0):
        """Override the kernel's K steps per stage, stages per warp, units per
        32 rows and block-dot step (tc 1: dp4a, 2: tensor cores; 0:
        automatic); a tuning and test hook (ds4moe_dense_debug_config)."""
        _check(lib().ds4moe_dense_debug_config(self._h, int(ks), int(nst), int(ns), int(tc)),
               "ds4moe_dense_debug_config")


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, name, dtype, shape, inner=None):
    """Elements from one row of `t` to the next: `shape` after the leading
    dimensions, contiguous, the leading dimensions evenly spaced. `inner`: the
    elements of a row, where the caller has them."""
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype):
        raise ValueError(f"{name}: a CUDA tensor of {dtype}")
    size = t.shape
    lead = len(size) - len(shape)
    if lead < 1 or size[lead:] != shape:
        raise ValueError(f"{name}: shape [..., {', '.join(map(str, shape))}]")
    if inner is None:
        inner = 1
        for n in shape:
            inner *= n
    if t.is_contiguous():
        return inner
    step = 1
    for n, s in zip(reversed(shape), reversed(t.stride()[lead:])):
        _need(n == 1 or s == step, f"{name}: a row must be contiguous")
        step *= n
    row, step = None, None  # the stride of a row; the stride the next leading dimension must have
    for n, s in zip(reversed(size[:lead]), reversed(t.stride()[:lead])):
        if n == 1:
            continue
        if row is None:
            row = s
        else:
            _need(s == step, f"{name}: rows must be evenly spaced")
        step = s * n
    return inner if row is None else row


def _vec(t, name, dtype, n):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.numel() == n and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous CUDA tensor of {n} {dtype}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """A tensor that a call writes on `stream`. The allocator hands out memory
    in the order of the stream that is current: a block freed there may still be
    in use by what that stream has queued, for which another one would not wait.
    So it comes from `stream`'s own blocks, and goes back to them only when the
    current stream, where the caller goes on, is done with it too."""
    import torch
    if stream is None or torch.device(device).type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    here = torch.cuda.current_stream(device)
    if stream.cuda_stream == here.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(here)
    return out


def _torch_dtype(dt):
    import torch
    return {DT_F32: torch.float32, DT_BF16: torch.bfloat16, DT_F16: torch.float16}[dt]


@dataclass
class AttentionDesc:
    """Shape of the attention beside the MoE (ds4moe_attn_desc). `scale` None:
    1 / sqrt(head_dim)."""
    n_heads: int
    n_kv_heads: int
    head_dim: int
    dtype: str = "bf16"  # "bf16" | "fp16": q, cache and output
    window: int = 0
    n_sink: int = 0
    scale: float | None = None
    max_seqs: int = 1
    max_tokens: int = 1

    def c(self) -> _AttnDesc:
        scale = self.scale if self.scale is not None else max(self.head_dim, 1) ** -0.5
        return _AttnDesc(ABI_VERSION, self.n_heads, self.n_kv_heads, self.head_dim, DTYPE[self.dtype], self.window,
                         self.n_sink, scale, self.max_seqs, self.max_tokens)


class KVCache:
    """A paged cache (ds4moe_kv_cache): `k`, `v` are CUDA tensors [n_pages,
    page_size, n_kv_heads, head_dim] (any strides over the first three),
    `block_table` int32 [n_seq, max_pages]. Keeps the tensors; their contents
    may change between calls."""

    def __init__(self, k, v, block_table):
        import torch
        for t, name in ((k, "k"), (v, "v")):
            _need(isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 4 and t.stride(3) == 1,
                  f"{name}: a CUDA tensor [n_pages, page_size, n_kv_heads, head_dim], head_dim contiguous")
        _need(k.shape == v.shape and k.dtype == v.dtype, "k and v: the same shape and type")
        _need(isinstance(block_table, torch.Tensor) and block_table.is_cuda and block_table.dim() == 2 and
              block_table.dtype == torch.int32 and (block_table.shape[1] == 1 or block_table.stride(1) == 1),
              "block_table: a CUDA int32 tensor [n_seq, max_pages] with contiguous rows")
        self.k, self.v, self.block_table = k, v, block_table
        stride = block_table.stride(0) if block_table.shape[0] > 1 else block_table.shape[1]
        self.row, self.dtype, self.n_seq = tuple(k.shape[2:]), k.dtype, block_table.shape[0]
        self.c = _KvCache(k.data_ptr(), v.data_ptr(), k.shape[0], k.stride(0), k.stride(1), k.stride(2), v.stride(0),
                          v.stride(1), v.stride(2), block_table.data_ptr(), stride, k.shape[1], block_table.shape[1])
        self.ref = ctypes.byref(self.c)


class Attention:
    """Append to, and attention over, a paged key-value cache (ds4moe_attn_*).
    One serves all layers of its shape that run one after another on a stream.

    A call with `stream` does not wait for the current stream, nor that for the
    call: order them. Its outputs may be used on either; the tensors passed in
    must live until it is done."""

    def __init__(self, desc: AttentionDesc):
        h = ctypes.c_void_p()
        _check(lib().ds4moe_attn_create(ctypes.byref(desc.c()), ctypes.byref(h)), "ds4moe_attn_create")
        self.desc, self._h = desc, h
        self._dt, self._code = _torch_dtype(DTYPE[desc.dtype]), DTYPE[desc.dtype]
        self._q_row, self._q_len = (desc.n_heads, desc.head_dim), desc.n_heads * desc.head_dim
        self._kv_row, self._kv_len = (desc.n_kv_heads, desc.head_dim), desc.n_kv_heads * desc.head_dim

    def close(self):
        if getattr(self, "_h", None):
            lib().ds4moe_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _cache(self, cache, n_seq):
        if not isinstance(cache, KVCache):
            raise ValueError("cache: a KVCache")
        if cache.row != self._kv_row or cache.dtype != self._dt:
            raise ValueError("cache: heads, dimension or type differ from the handle's")
        if cache.n_seq < n_seq:
            raise ValueError("cache: a block-table row for every sequence")
        return cache.ref

    def append(self, cache, k, v, kv_len, cu_q=None, stream=None):
        """Write new keys and values (ds4moe_kv_append): k, v [n_tok, n_kv_heads,
        head_dim] or [n_seq, n_new, ...], fp32 or the cache's type; v may be None
        (the keys only). kv_len int32 [n_seq] counts the new tokens."""
        import torch
        n_seq = kv_len.numel()
        if cu_q is None and k.dim() == 4 and k.shape[0] != n_seq:
            raise ValueError("k: [n_seq, n_new, ...] for the sequences of kv_len")
        dt = torch.float32 if k.dtype == torch.float32 else self._dt
        ks = _rows(k, "k", dt, self._kv_row, self._kv_len)
        vs = 0
        if v is not None:
            vs = _rows(v, "v", dt, self._kv_row, self._kv_len)
            if v.shape != k.shape:
                raise ValueError("v: the shape of k")
        _check(_lib.ds4moe_kv_append(
            self._h, self._cache(cache, n_seq), k.data_ptr(), ks, None if v is None else v.data_ptr(), vs,
            DT_F32 if dt == torch.float32 else self._code,
            None if cu_q is None else _vec(cu_q, "cu_q", torch.int32, n_seq + 1),
            _vec(kv_len, "kv_len", torch.int32, n_seq), n_seq, k.numel() // self._kv_len, _stream(stream)),
            "ds4moe_kv_append")

    def _out(self, q, out, stream):
        """The output and its row stride."""
        if out is None:
            return _empty(q.shape, q.dtype, q.device, stream), self._q_len
        if out.shape != q.shape:
            raise ValueError("out: the shape of q")
        return out, _rows(out, "out", self._dt, self._q_row, self._q_len)

    def decode(self, cache, q, kv_len, out=None, stream=None):
        """Attention of the last n_new tokens of every sequence
        (ds4moe_attn_decode): q [n_seq, n_new, n_heads, head_dim]; returns out."""
        import torch
        if q.dim() != 4:
            raise ValueError("q: [n_seq, n_new, n_heads, head_dim]")
        n_seq, n_new = q.shape[:2]
        qs = _rows(q, "q", self._dt, self._q_row, self._q_len)
        out, os_ = self._out(q, out, stream)
        _check(_lib.ds4moe_attn_decode(self._h, self._cache(cache, n_seq), q.data_ptr(), qs,
                                       _vec(kv_len, "kv_len", torch.int32, n_seq), n_seq, n_new, out.data_ptr(), os_,
                                       _stream(stream)), "ds4moe_attn_decode")
        return out

    def prefill(self, cache, q, cu_q, kv_len, out=None, stream=None):
        """Attention of ragged runs of new tokens (ds4moe_attn_prefill): q
        [n_tok, n_heads, head_dim], cu_q int32 [n_seq + 1]; returns out."""
        import torch
        if q.dim() != 3:
            raise ValueError("q: [n_tok, n_heads, head_dim]")
        n_seq = kv_len.numel()
        qs = _rows(q, "q", self._dt, self._q_row, self._q_len)
        out, os_ = self._out(q, out, stream)
        _check(_lib.ds4moe_attn_prefill(self._h, self._cache(cache, n_seq), q.data_ptr(), qs,
                                        _vec(cu_q, "cu_q", torch.int32, n_seq + 1),
                                        _vec(kv_len, "kv_len", torch.int32, n_seq), n_seq, q.shape[0], out.data_ptr(),
                                        os_, _stream(stream)), "ds4moe_attn_prefill")
        return out

    def device_error(self, stream=None) -> int:
        """Synchronise, read and clear the device error flags (0 = none)."""
        f = ctypes.c_uint32(0)
        st = lib().ds4moe_attn_get_device_error(self._h, _stream(stream), ctypes.byref(f))
        if st not in (0, 5):
            raise Ds4MoeError(st, "ds4moe_attn_get_device_error")
        return int(f.value)

    def device_bytes(self) -> int:
        return int(lib().ds4moe_attn_device_bytes(self._h))

    def launch_count(self) -> int:
        return int(lib().ds4moe_attn_launch_count(self._h))


def token_probs(logits, temperature: float = 1.0, out=None, stream=None):
    """softmax(logits / temperature) over the last dimension of an fp32 CUDA
    tensor (ds4moe_token_probs); temperature 0: one at the lowest index of the
    maximum. `out` may be `logits`; returns out."""
    import torch
    V = logits.shape[-1]
    if out is None:
        out = _empty(logits.shape, torch.float32, logits.device, stream)
    elif out.shape != logits.shape:
        raise ValueError("out: the shape of logits")
    one = logits.dim() == 1
    xs = _rows(logits[None] if one else logits, "logits", torch.float32, (V,), V)
    os_ = _rows(out[None] if one else out, "out", torch.float32, (V,), V)
    _check(lib().ds4moe_token_probs(logits.data_ptr(), xs, logits.numel() // max(V, 1), V, temperature, out.data_ptr(),
                                    os_, _stream(stream)), "ds4moe_token_probs")
    return out


def verify_drafts(target, draft, tokens, u_accept, u_sample, n_draft=None, n_accepted=None, tokens_out=None,
                  err_flags=None, stream=None):
    """Which drafted tokens stay, and the token after them
    (ds4moe_verify_drafts): target fp32 [n_seq, max_draft + 1, vocab], draft
    fp32 [n_seq, max_draft, vocab] or None, tokens int32 [n_seq, max_draft].
    Returns (n_accepted int32 [n_seq], tokens_out int32 [n_seq, max_draft + 1])."""
    import torch
    lib()
    i32, f32 = torch.int32, torch.float32
    if target.dim() != 3:
        raise ValueError("target: [n_seq, max_draft + 1, vocab]")
    B, G, V = target.shape
    G -= 1
    ts, ds = _rows(target, "target", f32, (V,), V), 0
    if draft is not None:
        if tuple(draft.shape) != (B, G, V):
            raise ValueError("draft: [n_seq, max_draft, vocab]")
        ds = _rows(draft, "draft", f32, (V,), V)
    if n_accepted is None:
        n_accepted = _empty((B,), i32, target.device, stream)
    else:
        _vec(n_accepted, "n_accepted", i32, B)
    if tokens_out is None:
        tokens_out = _empty((B, G + 1), i32, target.device, stream)
    else:
        _vec(tokens_out, "tokens_out", i32, B * (G + 1))
    _check(_lib.ds4moe_verify_drafts(
        target.data_ptr(), ts, None if draft is None else draft.data_ptr(), ds, _vec(tokens, "tokens", i32, B * G),
        None if n_draft is None else _vec(n_draft, "n_draft", i32, B), _vec(u_accept, "u_accept", f32, B * G),
        _vec(u_sample, "u_sample", f32, B), B, G, V, n_accepted.data_ptr(), tokens_out.data_ptr(),
        None if err_flags is None else _vec(err_flags, "err_flags", i32, 1), _stream(stream)), "ds4moe_verify_drafts")
    return n_accepted, tokens_out


def rmsnorm(x, out, eps: float = 1e-6, stream=None):
    """out = x / sqrt(mean(x^2) + eps) row-wise (ds4moe_rmsnorm); out may be x."""
    _check(lib().ds4moe_rmsnorm(_ptr(x), _ptr(out), x.shape[0], x.shape[1], eps, _stream(stream)),
           "ds4moe_rmsnorm")


NOALLOC_SCRATCH_BYTES = 512 * 1024


def route_noalloc(desc: LayerDesc, weights: dict, x=None, token_ids=None, ids_out=None, w_out=None,
                  err_flags=None, stream=None, n_tok=None):
    """Routing from the canonical router buffers in `weights` (router_w,
    router_bias or hash_table; CUDA tensors) with no handle and no device
    allocation by the library (ds4moe_route_noalloc). ids_out / w_out are
    allocated here by torch when not given. Returns (ids_out, w_out)."""
    import torch
    n = n_tok if n_tok is not None else (x.shape[0] if x is not None else token_ids.shape[0])
    dev = (x if x is not None else token_ids).device
    if ids_out is None:
        ids_out = torch.empty((n, desc.top_k), dtype=torch.int32, device=dev)
    if w_out is None:
        w_out = torch.empty((n, desc.top_k), dtype=torch.float32, device=dev)
    w = _Weights(*[_ptr(weights.get(name)) for name, _ in _Weights._fields_])
    _check(lib().ds4moe_route_noalloc(ctypes.byref(desc.c()), ctypes.byref(w), _ptr(x), _ptr(token_ids), n,
                                      _ptr(ids_out), _ptr(w_out), _ptr(err_flags), _stream(stream)),
           "ds4moe_route_noalloc")
    return ids_out, w_out


def fail_alloc(n: int):
    """Make the n-th device allocation the library makes from now on fail as
    if out of memory (0: off); a test hook (ds4moe_debug_fail_alloc)."""
    _check(lib().ds4moe_debug_fail_alloc(int(n)), "ds4moe_debug_fail_alloc")


def status_string(status: int) -> str:
    return lib().ds4moe_status_string(status).decode()
