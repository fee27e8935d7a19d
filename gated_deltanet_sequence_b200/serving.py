"""One serving step of a batch of requests: the binding of gdn_plan_batch, gdn_kv_append,
gdn_kv_attn and gdn_decode_slots (include/gdn.h).

A step of a model that mixes gated delta-rule layers with softmax layers:

    plan = BatchPlan.empty(N, max_tokens, "cuda")                     # once
    gdn_plan_batch(ctx_lens, new_lens, block_table, free_list, free_count, 64, plan)   # once a step
    # each softmax layer
    gdn_kv_append(cache, k, v, plan.slot_map)
    o, _ = gdn_kv_attn(cache, q, block_table, plan.cu_seqlens, plan.kv_lens, max_q_len=m, scale=d ** -0.5)
    # each delta-rule layer
    o = gdn_decode_slots(q, k, v, beta, g, state, slots, plan.cu_seqlens)

Token rows are token-major, (T, heads, d); q, k and v may be column ranges of one fused
projection (any row stride that keeps rows 16-byte aligned, heads and columns contiguous).
As in :mod:`._lib`, this marshals arguments only.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib
from ._lib import _check, _new, _out_opts, _raise, lib

_BLOCK_SIZES = (16, 32, 64, 128)


# The calls below run once a layer and decoded token, on batches whose kernels take a few microseconds, so what they do
# on the host is kept short: the raw stream handle where torch offers it, one comparison for a tensor that is right.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_i32, _f32, _bf16 = torch.int32, torch.float32, torch.bfloat16


def _stream_of(dev: torch.device, stream) -> int:
    """The stream a call for tensors on ``dev`` goes to: ``stream``, or that device's current one."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {dev}")
    if stream is None:
        return _raw_stream(dev.index) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _call(f, fn: str, dev: torch.device, args) -> None:
    """One call of the library with ``dev`` current (it launches on the current device)."""
    if dev.index == _device_now():
        st = f(*args)
    else:
        with torch.cuda.device(dev):
            st = f(*args)
    if st:
        _raise(fn, st)


def _want(name: str, t: torch.Tensor, shape, dtype, dev):
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return
    _check(name, t, shape, dtype, dev)


def _rows(name: str, t: torch.Tensor, shape, dtype, dev) -> int:
    """Row stride of a (T, heads, d) tensor whose rows are contiguous."""
    T, h, d = shape
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return h * d
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    s = t.stride()
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        raise ValueError(f"{name}: heads and columns of a row must be contiguous")
    if T <= 1:
        return h * d
    if s[0] < h * d:
        raise ValueError(f"{name}: rows overlap (row stride {s[0]} < {h * d})")
    return s[0]


class KvCache:
    """A paged cache of one softmax layer: k, v (num_blocks, Hkv, block_size, d) e4m3 and their
    scales k_scale, v_scale (num_blocks, Hkv) fp32. Checked once, here."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "num_blocks", "heads", "block_size", "d", "device", "_args")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4:
            raise ValueError(f"k: expected (num_blocks, Hkv, block_size, d), got {tuple(k.shape)}")
        nb, h, bs, d = k.shape
        if bs not in _BLOCK_SIZES or d not in (64, 128):
            raise ValueError(f"block_size must be one of {_BLOCK_SIZES} and d 64 or 128, got {bs} and {d}")
        _check("k", k, (nb, h, bs, d), torch.float8_e4m3fn)
        _check("v", v, (nb, h, bs, d), torch.float8_e4m3fn, k.device)
        _check("k_scale", k_scale, (nb, h), torch.float32, k.device)
        _check("v_scale", v_scale, (nb, h), torch.float32, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_blocks, self.heads, self.block_size, self.d, self.device = nb, h, bs, d, k.device
        self._args = (k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())

    @classmethod
    def empty(cls, num_blocks: int, heads: int, block_size: int, d: int, device="cuda") -> "KvCache":
        shape = (num_blocks, heads, block_size, d)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones(num_blocks, heads, dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


class BatchPlan:
    """What gdn_plan_batch writes, for N requests and T token rows: cu_seqlens (N + 1), kv_lens (N),
    positions, seq_ids, slot_map (T), info (4: new tokens, longest kv length, missing blocks, free blocks
    left), all int32."""

    __slots__ = ("cu_seqlens", "kv_lens", "positions", "seq_ids", "slot_map", "info", "N", "T", "device", "_args")

    def __init__(self, cu_seqlens, kv_lens, positions, seq_ids, slot_map, info):
        N, T, dev = kv_lens.numel(), slot_map.numel(), kv_lens.device
        for name, t, n in (("cu_seqlens", cu_seqlens, N + 1), ("kv_lens", kv_lens, N), ("positions", positions, T),
                           ("seq_ids", seq_ids, T), ("slot_map", slot_map, T), ("info", info, 4)):
            _check(name, t, (n,), torch.int32, dev)
            setattr(self, name, t)
        self.N, self.T, self.device = N, T, dev
        self._args = tuple(t.data_ptr() for t in (cu_seqlens, kv_lens, positions, seq_ids, slot_map, info))

    @classmethod
    def empty(cls, N: int, T: int, device="cuda") -> "BatchPlan":
        return cls(*(torch.zeros(n, dtype=torch.int32, device=device) for n in (N + 1, N, T, T, T, 4)))


def gdn_plan_batch(ctx_lens, new_lens, block_table, free_list, free_count, block_size: int, plan: BatchPlan,
                   stream=None) -> BatchPlan:
    """Block tables, slot maps and packed offsets of a step from the requests' lengths (N,) int32: ctx_lens tokens
    cached (``plan.kv_lens`` of the step before will do), new_lens tokens brought (0: waiting, -1: finished, its blocks are
    freed). Updates block_table
    (N, max_blocks), free_list (num_blocks,) and free_count (1,) in place, fills ``plan`` and returns it."""
    dev, N = plan.device, plan.N
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected (N, max_blocks), got {tuple(block_table.shape)}")
    mb, nb = block_table.shape[1], free_list.numel()
    _want("ctx_lens", ctx_lens, (N,), _i32, dev)
    _want("new_lens", new_lens, (N,), _i32, dev)
    _want("block_table", block_table, (N, mb), _i32, dev)
    _want("free_list", free_list, (nb,), _i32, dev)
    _want("free_count", free_count, (1,), _i32, dev)
    _call(lib.gdn_plan_batch, "gdn_plan_batch", dev,
          (ctx_lens.data_ptr(), new_lens.data_ptr(), N, block_table.data_ptr(), mb, free_list.data_ptr(),
           free_count.data_ptr(), nb, block_size, plan.T, *plan._args, _stream_of(dev, stream)))
    return plan


def gdn_kv_append(cache: KvCache, k, v, slot_map, stream=None) -> KvCache:
    """Write k, v (T, Hkv, d) bf16 / fp32 into the cache rows slot_map (T,) int32 names (-1: skipped). The rows of one
    block must be consecutive, as BatchPlan.slot_map has them."""
    dev, T = cache.device, k.shape[0]
    shape = (T, cache.heads, cache.d)
    ks = _rows("k", k, shape, k.dtype, dev)
    vs = _rows("v", v, shape, k.dtype, dev)
    _want("slot_map", slot_map, (T,), _i32, dev)
    kc, vc, kscale, vscale = cache._args
    _call(lib.gdn_kv_append, "gdn_kv_append", dev,
          (k.data_ptr(), v.data_ptr(), ks, vs, slot_map.data_ptr(), kc, vc, kscale, vscale, T, cache.heads, cache.d,
           cache.num_blocks, cache.block_size, _lib._dtype_code(k), _stream_of(dev, stream)))
    return cache


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(index: Optional[int], N: int, T: int, Hq: int, Hkv: int, d: int, max_q_len: int) -> int:
    """The size on device ``index`` (it grows with the device's SMs); None: no device."""
    if index is None or index == _device_now():
        return int(lib.gdn_kv_attn_workspace_bytes(N, T, Hq, Hkv, d, max_q_len))
    with torch.cuda.device(index):
        return int(lib.gdn_kv_attn_workspace_bytes(N, T, Hq, Hkv, d, max_q_len))


def gdn_kv_attn_workspace_bytes(N: int, T: int, Hq: int, Hkv: int, d: int, max_q_len: int = 1, device=None) -> int:
    """Bytes of device workspace gdn_kv_attn needs on ``device`` (the current one when None; 0 for unsupported sizes)."""
    index = None
    if torch.cuda.is_available():
        index = torch.device("cuda" if device is None else device).index
        index = _device_now() if index is None else index
    return _workspace_bytes(index, N, T, Hq, Hkv, d, max_q_len)


def gdn_kv_attn(cache: KvCache, q, block_table, cu_seqlens, kv_lens, max_q_len: int = 1, window: int = 0,
                scale: float = 1.0, o=None, lse=None, out_dtype: Optional[torch.dtype] = None, workspace=None,
                stream=None):
    """Causal softmax attention of q (T, Hq, d), rows cu_seqlens[n] .. cu_seqlens[n+1]-1 being the last tokens of
    request n, over its kv_lens[n] cached tokens (window > 0: the last ``window`` of each query only). Returns
    (o, lse): o (T, Hq, d) of o.dtype, else out_dtype, else fp32; lse (T, Hq) fp32 when a tensor or True is passed,
    else None. Rows behind the last request are left as they were (unspecified in tensors allocated here).
    ``max_q_len`` bounds the rows of one request. ``workspace``: a device tensor of at least
    gdn_kv_attn_workspace_bytes(...) bytes (allocated with torch when None)."""
    dev = cache.device
    if q.dim() != 3:
        raise ValueError(f"q: expected (T, Hq, d), got shape {tuple(q.shape)}")
    T, Hq, d = q.shape
    if d != cache.d:
        raise ValueError(f"q: head size {d}, the cache has {cache.d}")
    if Hq % cache.heads != 0 or Hq == 0:
        raise ValueError(f"q: {Hq} query heads over {cache.heads} KV heads")
    qs = _rows("q", q, q.shape, q.dtype, dev)
    N = kv_lens.numel()
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected (N, max_blocks), got {tuple(block_table.shape)}")
    mb = block_table.shape[1]
    _want("kv_lens", kv_lens, (N,), _i32, dev)
    _want("cu_seqlens", cu_seqlens, (N + 1,), _i32, dev)
    _want("block_table", block_table, (N, mb), _i32, dev)
    odt = o.dtype if o is not None else (out_dtype or _f32)
    if odt is not _f32 and odt is not _bf16:
        raise TypeError(f"o / out_dtype must be float32 or bfloat16, got {odt}")
    dt = _lib._dtype_code(q)
    raw = _stream_of(dev, stream)
    need = _workspace_bytes(dev.index, N, T, Hq, cache.heads, d, max_q_len)
    if o is None:
        o = _new(q, (T, Hq, d), odt, stream)
    else:
        _want("o", o, (T, Hq, d), odt, dev)
    if lse is False:
        lse = None
    if lse is True:
        lse = _new(q, (T, Hq), _f32, stream)
    elif lse is not None:
        _want("lse", lse, (T, Hq), _f32, dev)
    if workspace is None:
        workspace = _new(q, max(need, 16), torch.uint8, stream, result=False)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    kc, vc, kscale, vscale = cache._args
    _call(lib.gdn_kv_attn, "gdn_kv_attn", dev, (q.data_ptr(), qs, kc, vc, kscale, vscale, block_table.data_ptr(), cu_seqlens.data_ptr(),
          kv_lens.data_ptr(), o.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), N, T, Hq, cache.heads, d, cache.num_blocks, cache.block_size, mb,
          max_q_len, window, scale, dt, _lib.GDN_BF16 if odt is _bf16 else _lib.GDN_F32, raw))
    return o, lse


def gdn_decode_slots(q, k, v, beta, g, state, slots, cu_seqlens=None, o=None, scale: float = 1.0, stream=None,
                     out_dtype=None, d_skip=None, xnorm=None, xnorm_weight=None, xnorm_eps: float = 1e-6):
    """The gated delta rule's recurrence over ``state`` (n_slots, Hv, dk, dv) fp32, updated in place: request n takes
    its rows of q, k (T, Hk, dk) and v (T, Hv, dv) through state slots[n] (-1: skipped), token by token; cu_seqlens
    (N + 1,) int32 gives its rows (None: row n). Value head h reads key head h // (Hv // Hk). beta, g (T, Hv) or None,
    g (T, Hv, dk) for a vector-valued gate; the options as for gdn_decode_step. Returns o (T, Hv, dv); rows of no
    request are left as they were (unspecified when ``o`` is allocated here)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q, v: expected (T, heads, d), got {tuple(q.shape)} and {tuple(v.shape)}")
    T, Hk, dk = q.shape
    _, Hv, dv = v.shape
    dev = q.device
    qs = _rows("q", q, q.shape, q.dtype, dev)
    ks = _rows("k", k, q.shape, q.dtype, dev)
    vs = _rows("v", v, torch.Size((T, Hv, dv)), q.dtype, dev)
    if Hk == 0 or Hv % Hk != 0:
        raise ValueError(f"{Hv} value heads over {Hk} key heads")
    if beta is not None:
        _want("beta", beta, (T, Hv), _f32, dev)
    vec = False
    if g is not None:
        vec = g.dim() == 3
        _want("g", g, (T, Hv, dk) if vec else (T, Hv), _f32, dev)
    if state.dim() != 4:
        raise ValueError(f"state: expected (n_slots, Hv, dk, dv), got {tuple(state.shape)}")
    n_slots = state.shape[0]
    _want("state", state, (n_slots, Hv, dk, dv), _f32, dev)
    N = slots.numel()
    _want("slots", slots, (N,), _i32, dev)
    if cu_seqlens is None:
        if T != N:
            raise ValueError(f"{T} rows for {N} slots: give cu_seqlens")
    else:
        _want("cu_seqlens", cu_seqlens, (N + 1,), _i32, dev)
    if o is None and not vec and d_skip is None and xnorm is None and xnorm_weight is None and out_dtype in (None, _f32):
        odt, opts = _f32, None
    else:
        odt, opts = _out_opts(o, out_dtype, d_skip, Hv, dv, dev, vec, xnorm, xnorm_weight, xnorm_eps)
    dt = _lib._dtype_code(q)
    raw = _stream_of(dev, stream)
    if o is None:
        o = _new(q, (T, Hv, dv), odt, stream)
    else:
        _want("o", o, (T, Hv, dv), odt, dev)
    _call(lib.gdn_decode_slots, "gdn_decode_slots", dev, (q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
          None if beta is None else beta.data_ptr(), None if g is None else g.data_ptr(), state.data_ptr(),
          slots.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), o.data_ptr(), N, T, Hk, Hv,
          n_slots, dk, dv, scale, dt, None if opts is None else ctypes.byref(opts), raw))
    return o
