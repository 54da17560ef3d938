"""Frame-aware class attention: a learned bias by frame distance (with its gradient and the masks
a bucket map expresses), and an 8-bit frame cache with the attention that reads it, for
frame-by-frame generation.

As the rest of the package, these functions check and marshal arguments; the work runs in the
library's sm_100a kernels. Every function exists for Skiparse-2D and Skiparse-1D. A call works on
the tensors' own device and, unless `stream` is given, on that device's current stream; what it
allocates (outputs, workspaces) belongs to the stream it works on.
"""

from __future__ import annotations

import functools
import math
from typing import NamedTuple

import torch

from ._lib import check, lib

BLOCK = 64  # tokens of one class, frame and head that share a scale in the cache


def frame_buckets(max_distance: int, num_buckets: int, causal: bool = False, window: int | None = None,
                  device="cuda") -> torch.Tensor:
    """The usual bucket map of relative distances, as a (2*max_distance+1) int32 tensor for the
    distances -max_distance .. max_distance (frame of the query minus frame of the key): of the
    buckets of a direction, half hold one distance each, from 0, and half are spaced by the
    distance's logarithm up to max_distance. Without `causal` the earlier frames take the first
    half of the buckets and the later ones the second. `causal` masks later frames (-1); `window`
    masks distances of `window` frames and more."""
    if not 0 <= max_distance <= 255:
        raise ValueError("max_distance must be between 0 and 255")
    if num_buckets < 1:
        raise ValueError("num_buckets must be positive")
    per = num_buckets if causal else max(1, num_buckets // 2)
    half = max(1, per // 2)

    def bucket(a: int) -> int:
        if a < half:
            return min(a, per - 1)
        span = math.log(max(2.0, (max_distance + 1) / half))
        return min(per - 1, half + int(math.log(a / half) / span * (per - half)))

    out = []
    for u in range(-max_distance, max_distance + 1):
        g = bucket(abs(u))
        if u < 0:
            g = -1 if causal else min(num_buckets - 1, g + per)
        out.append(-1 if window is not None and abs(u) >= window else g)
    return torch.tensor(out, dtype=torch.int32, device=device)


class FrameCache(NamedTuple):
    """The e4m3 frame cache of one layer, a ring of `capacity` frames (see frame_cache)."""

    k: torch.Tensor        # (B*P*P, heads, capacity, F, d) float8_e4m3fn
    v: torch.Tensor
    k_scale: torch.Tensor  # (B*P*P, heads, capacity, ceil(F/64)) float8_e8m0fnu
    v_scale: torch.Tensor

    @property
    def capacity(self) -> int:
        return self.k.shape[2]


def frame_cache(B: int, capacity: int, H: int, W: int, heads: int, d: int, P: int, dims: int = 2,
                device="cuda") -> FrameCache:
    """An empty cache for `capacity` frames of an (H, W) latent (Skiparse-2D or, dims=1, -1D)."""
    F = _entry("skiparse@_cache_frame_tokens", dims)(H, W, P)
    if F < 0 or min(B, capacity, heads, d) < 1:
        raise ValueError("invalid cache shape")
    rows = (B * P * P, heads, capacity, F)
    codes = [torch.zeros(rows + (d,), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full(rows[:3] + (-(-F // BLOCK),), 127, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)
              for _ in range(2)]
    return FrameCache(*codes, *scales)


def _entry(name: str, dims: int):
    if dims not in (1, 2):
        raise ValueError("dims must be 1 (Skiparse-1D) or 2 (Skiparse-2D)")
    return getattr(lib(), name.replace("@", "1d" if dims == 1 else "2d"))


@functools.lru_cache(maxsize=256)
def _size_of(name: str, *args) -> int:
    """A size the library computes from sizes alone; name is the entry point's."""
    return getattr(lib(), name)(*args)


def _need(name: str, t, dtype, shape=None, device: int | None = None) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape)
            and (t.get_device() == device if device is not None else t.is_cuda)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")


def _tokens(name: str, t):
    """Checks a (B,T,H,W,heads,d) tensor; returns its shape and device index."""
    _need(name, t, torch.bfloat16)
    if t.dim() != 6:
        raise ValueError(f"{name} must be (B,T,H,W,heads,d)")
    return t.shape, t.get_device()


def _bias(table, buckets, heads: int, device: int):
    """Pointers and sizes of the bias arguments."""
    _need("table", table, torch.bfloat16, None, device)
    _need("buckets", buckets, torch.int32, None, device)
    if table.dim() != 2 or table.shape[0] < 1 or table.shape[1] != heads:
        raise ValueError(f"table must be (num_buckets, {heads})")
    n = buckets.numel()
    if buckets.dim() != 1 or n % 2 == 0 or n > 511:
        raise ValueError("buckets must hold 2*max_distance+1 entries, max_distance <= 255")
    return table.data_ptr(), buckets.data_ptr(), table.shape[0], n // 2


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same pointer without a Stream object, several microseconds of a small call, where torch has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _on(device: int, stream, call):
    """Runs call(stream pointer) with the tensors' device and the stream to work on current, so that
    what it allocates belongs to that stream."""
    if stream is None and device == torch.cuda.current_device():
        return call(_current_stream(device))
    if stream is not None and stream.device_index != device:
        raise ValueError(f"stream must be on cuda:{device}, got cuda:{stream.device_index}")
    with torch.cuda.device(device):
        if stream is None:
            return call(_current_stream(device))
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _relbias_fwd(dims, q, k, v, table, buckets, P, mode, out, lse, out_lo, stream):
    shape, dev = _tokens("q", q)
    bf16 = torch.bfloat16
    _need("k", k, bf16, shape, dev)
    _need("v", v, bf16, shape, dev)
    bias = _bias(table, buckets, shape[4], dev)
    if out is not None:
        _need("out", out, bf16, shape, dev)
    if out_lo is not None:
        _need("out_lo", out_lo, bf16, shape, dev)
    if lse is not None:
        _need("lse", lse, torch.float32, shape[:5], dev)
    name = "skiparse@_attn_relbias_fwd"

    def call(st):
        o = torch.empty_like(q) if out is None else out
        l = q.new_empty(shape[:5], dtype=torch.float32) if lse is None else lse
        check(_entry(name, dims)(q.data_ptr(), k.data_ptr(), v.data_ptr(), *bias, o.data_ptr(),
                                 None if out_lo is None else out_lo.data_ptr(), l.data_ptr(), *shape, P, mode, st), name)
        return o, l

    return _on(dev, stream, call)


def _relbias_bwd(dims, q, k, v, out, dout, lse, table, buckets, P, mode, dq, dk, dv, dtable, out_lo, workspace,
                 stream):
    shape, dev = _tokens("q", q)
    bf16 = torch.bfloat16
    for what, t in (("k", k), ("v", v), ("out", out), ("dout", dout)):
        _need(what, t, bf16, shape, dev)
    _need("lse", lse, torch.float32, shape[:5], dev)
    bias = _bias(table, buckets, shape[4], dev)
    for what, t in (("out_lo", out_lo), ("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None:
            _need(what, t, bf16, shape, dev)
    if dtable is not None:
        _need("dtable", dtable, bf16, table.shape, dev)
    if workspace is not None:
        _need("workspace", workspace, torch.uint8, None, dev)
    name = "skiparse@_attn_relbias_bwd"
    need = _size_of(f"skiparse{dims}d_attn_relbias_bwd_workspace_bytes", *shape, P, bias[3])
    if need < 0:
        raise ValueError("invalid shape or P")

    def call(st):
        grads = [torch.empty_like(q) if g is None else g for g in (dq, dk, dv)]
        grads.append(torch.empty_like(table) if dtable is None else dtable)
        ws = q.new_empty(need, dtype=torch.uint8) if workspace is None else workspace
        check(_entry(name, dims)(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 None if out_lo is None else out_lo.data_ptr(), dout.data_ptr(), lse.data_ptr(), *bias,
                                 *(g.data_ptr() for g in grads), ws.data_ptr(), ws.numel(), *shape, P, mode, st), name)
        return tuple(grads)

    return _on(dev, stream, call)


def skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P: int, mode: int, out=None, lse=None, out_lo=None,
                                stream=None):
    """Class attention with a learned bias by frame distance; returns (out, lse).

    q, k, v, out: (B,T,H,W,heads,d) bf16; table: (num_buckets, heads) bf16; buckets:
    (2*max_distance+1) int32, the bucket of each frame distance t_q - t_k (frame_buckets makes the
    usual map), a value outside [0, num_buckets) masking it, as an entry of the table at or below
    -65504 does (keys and values have to be finite there too); lse: (B,T,H,W,heads) fp32, natural
    log; out_lo: an optional bf16 tensor like q that receives what rounding took from out, for a more
    exact backward pass. A row without a visible key gives 0 and lse -inf."""
    return _relbias_fwd(2, q, k, v, table, buckets, P, mode, out, lse, out_lo, stream)


def skiparse1d_attn_relbias_fwd(q, k, v, table, buckets, P: int, mode: int, out=None, lse=None, out_lo=None,
                                stream=None):
    """Skiparse-1D forward with the bias, as skiparse2d_attn_relbias_fwd."""
    return _relbias_fwd(1, q, k, v, table, buckets, P, mode, out, lse, out_lo, stream)


def skiparse2d_attn_relbias_bwd(q, k, v, out, dout, lse, table, buckets, P: int, mode: int, dq=None, dk=None, dv=None,
                                dtable=None, out_lo=None, workspace=None, stream=None):
    """Backward pass of skiparse2d_attn_relbias_fwd: returns (dq, dk, dv, dtable). `out_lo`: the
    forward's, if it stored one (for a more exact dq). `workspace`: an optional CUDA
    uint8 tensor of skiparse2d_attn_relbias_bwd_workspace_bytes() bytes."""
    return _relbias_bwd(2, q, k, v, out, dout, lse, table, buckets, P, mode, dq, dk, dv, dtable, out_lo, workspace,
                        stream)


def skiparse1d_attn_relbias_bwd(q, k, v, out, dout, lse, table, buckets, P: int, mode: int, dq=None, dk=None, dv=None,
                                dtable=None, out_lo=None, workspace=None, stream=None):
    """Skiparse-1D backward pass with the bias, as skiparse2d_attn_relbias_bwd."""
    return _relbias_bwd(1, q, k, v, out, dout, lse, table, buckets, P, mode, dq, dk, dv, dtable, out_lo, workspace,
                        stream)


class SkiparseRelBiasAttention(torch.autograd.Function):
    """Differentiable class attention with the learned frame bias: gradients of q, k, v and table."""

    @staticmethod
    def forward(ctx, q, k, v, table, buckets, P: int, mode: int, dims: int = 2):
        q, k, v, table = q.contiguous(), k.contiguous(), v.contiguous(), table.contiguous()
        out_lo = torch.empty_like(q) if any(ctx.needs_input_grad) else None
        out, lse = _relbias_fwd(dims, q, k, v, table, buckets, P, mode, None, None, out_lo, None)
        ctx.save_for_backward(q, k, v, table, buckets, out, lse, out_lo)
        ctx.P, ctx.mode, ctx.dims = P, mode, dims
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, table, buckets, out, lse, out_lo = ctx.saved_tensors
        grads = _relbias_bwd(ctx.dims, q, k, v, out, dout.contiguous(), lse, table, buckets, ctx.P, ctx.mode,
                             None, None, None, None, out_lo, None, None)
        return (*grads, None, None, None, None)


def _cache_shapes(dims, cache, shape, P, device):
    """Checks a cache against a call's sizes; returns its capacity."""
    B, _, H, W, heads, d = shape
    if dims not in (1, 2):
        raise ValueError("dims must be 1 (Skiparse-1D) or 2 (Skiparse-2D)")
    F = _size_of(f"skiparse{dims}d_cache_frame_tokens", H, W, P)
    if F < 0:
        raise ValueError("invalid shape or P")
    k, v, k_scale, v_scale = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 5:
        raise ValueError("cache.k must be (B*P*P, heads, capacity, F, d)")
    capacity = k.shape[2]
    rows = (B * P * P, heads, capacity, F)
    _need("cache.k", k, torch.float8_e4m3fn, rows + (d,), device)
    _need("cache.v", v, torch.float8_e4m3fn, rows + (d,), device)
    blocks = rows[:3] + (-(-F // BLOCK),)
    _need("cache.k_scale", k_scale, torch.float8_e8m0fnu, blocks, device)
    _need("cache.v_scale", v_scale, torch.float8_e8m0fnu, blocks, device)
    return capacity


def _cache_append(dims, k, v, start, cache, P, mode, stream):
    shape, dev = _tokens("k", k)
    _need("v", v, torch.bfloat16, shape, dev)
    _need("start", start, torch.int32, shape[:1], dev)
    if cache is None:
        raise ValueError("cache must be a FrameCache")
    capacity = _cache_shapes(dims, cache, shape, P, dev)
    name = "skiparse@_cache_append"

    def call(st):
        check(_entry(name, dims)(k.data_ptr(), v.data_ptr(), start.data_ptr(), *(t.data_ptr() for t in cache),
                                 *shape, P, mode, capacity, st), name)
        return cache

    return _on(dev, stream, call)


def _attn_cached(dims, q, cache, start, P, mode, table, buckets, out, lse, workspace, stream):
    shape, dev = _tokens("q", q)
    _need("start", start, torch.int32, shape[:1], dev)
    if cache is None:
        raise ValueError("cache must be a FrameCache")
    capacity = _cache_shapes(dims, cache, shape, P, dev)
    if (table is None) != (buckets is None):
        raise ValueError("table and buckets belong together")
    bias = (None, None, 0, 0) if table is None else _bias(table, buckets, shape[4], dev)
    if out is not None:
        _need("out", out, torch.bfloat16, shape, dev)
    if lse is not None:
        _need("lse", lse, torch.float32, shape[:5], dev)
    if workspace is not None:
        _need("workspace", workspace, torch.uint8, None, dev)
    name = "skiparse@_attn_cached"
    need = _size_of(f"skiparse{dims}d_attn_cached_workspace_bytes", *shape, P, capacity)
    if need < 0:
        raise ValueError("invalid shape, P or capacity")

    def call(st):
        o = torch.empty_like(q) if out is None else out
        ws = workspace
        if ws is None and need:
            ws = q.new_empty(need, dtype=torch.uint8)
        check(_entry(name, dims)(q.data_ptr(), *(t.data_ptr() for t in cache), start.data_ptr(), *bias, o.data_ptr(),
                                 None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
                                 0 if ws is None else ws.numel(), *shape, P, mode, capacity, st), name)
        return o

    return _on(dev, stream, call)


def skiparse2d_cache_append(k, v, start, cache: FrameCache, P: int, mode: int, stream=None) -> FrameCache:
    """Quantises the keys and values of new frames, (B,T,H,W,heads,d) bf16, into the cache, in place.
    start: (B) int32 on the device, the frames each sequence has had before (the new ones go to
    slots start[b] .. start[b]+T-1 modulo the capacity); negative: the sequence is left alone."""
    return _cache_append(2, k, v, start, cache, P, mode, stream)


def skiparse1d_cache_append(k, v, start, cache: FrameCache, P: int, mode: int, stream=None) -> FrameCache:
    """Skiparse-1D form of skiparse2d_cache_append."""
    return _cache_append(1, k, v, start, cache, P, mode, stream)


def skiparse2d_attn_cached(q, cache: FrameCache, start, P: int, mode: int, table=None, buckets=None, out=None, lse=None,
                           workspace=None, stream=None) -> torch.Tensor:
    """Attention of the newest T frames' queries over the cache, to which these frames have been
    appended with the same `start`; table and buckets as in skiparse2d_attn_relbias_fwd, or none.
    A sequence with a negative start leaves its rows of `out` as they were (so pass one: those of a
    new tensor are not set). `lse`: an optional (B,T,H,W,heads) fp32 tensor that receives the
    log-sum-exp. `workspace`: an optional CUDA uint8 tensor of
    skiparse2d_attn_cached_workspace_bytes() bytes."""
    return _attn_cached(2, q, cache, start, P, mode, table, buckets, out, lse, workspace, stream)


def skiparse1d_attn_cached(q, cache: FrameCache, start, P: int, mode: int, table=None, buckets=None, out=None, lse=None,
                           workspace=None, stream=None) -> torch.Tensor:
    """Skiparse-1D form of skiparse2d_attn_cached."""
    return _attn_cached(1, q, cache, start, P, mode, table, buckets, out, lse, workspace, stream)
