"""CPU checks of the frame-aware operators: refusals before any CUDA call, geometry, bucket maps."""

from __future__ import annotations

import pytest
import torch

import fixed_pattern_sparse_b200 as fps
from fixed_pattern_sparse_b200 import _lib
from fixed_pattern_sparse_b200 import build as libbuild

from frames_reference import members

FAKE = 0x10000  # never dereferenced: every call below fails before any CUDA call
MB = 1 << 20
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return _lib.lib()


def at(i):
    return FAKE + i * MB


DIMS = dict(B=1, T=2, H=8, W=8, heads=2, d=32, P=2, mode=0)


def fwd(L, n="2d", ptr=None, num_buckets=4, max_distance=3, **dims):
    a = dict(q=at(0), k=at(1), v=at(2), table=at(3), buckets=at(4), out=at(5), out_lo=at(6), lse=at(7))
    a.update(ptr or {})
    s = {**DIMS, **dims}
    return getattr(L, f"skiparse{n}_attn_relbias_fwd")(a["q"], a["k"], a["v"], a["table"], a["buckets"], num_buckets,
                                                       max_distance, a["out"], a["out_lo"], a["lse"], *s.values(), None)


def bwd(L, n="2d", ptr=None, num_buckets=4, max_distance=3, ws_bytes=MB, **dims):
    names = ("q", "k", "v", "out", "out_lo", "dout", "lse", "table", "buckets", "dq", "dk", "dv", "dtable", "ws")
    a = {m: at(i) for i, m in enumerate(names)}
    a.update(ptr or {})
    s = {**DIMS, **dims}
    return getattr(L, f"skiparse{n}_attn_relbias_bwd")(*(a[m] for m in names[:9]), num_buckets, max_distance,
                                                       *(a[m] for m in names[9:]), ws_bytes, *s.values(), None)


def append(L, n="2d", ptr=None, capacity=4, **dims):
    names = ("k", "v", "start", "kc", "vc", "ks", "vs")
    a = {m: at(i) for i, m in enumerate(names)}
    a.update(ptr or {})
    return getattr(L, f"skiparse{n}_cache_append")(*(a[m] for m in names), *{**DIMS, **dims}.values(), capacity, None)


def cached(L, n="2d", ptr=None, num_buckets=4, max_distance=3, ws_bytes=MB, capacity=4, **dims):
    names = ("q", "kc", "vc", "ks", "vs", "start", "table", "buckets", "out", "lse", "ws")
    a = {m: at(i) for i, m in enumerate(names)}
    a.update(ptr or {})
    return getattr(L, f"skiparse{n}_attn_cached")(*(a[m] for m in names[:8]), num_buckets, max_distance,
                                                  *(a[m] for m in names[8:]), ws_bytes, *{**DIMS, **dims}.values(), capacity, None)


SHARED = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(mode=2), INVALID), (dict(P=0), INVALID), (dict(P=9), UNSUPPORTED),
          (dict(d=48), UNSUPPORTED), (dict(heads=1 << 20), UNSUPPORTED), (dict(H=1 << 25), UNSUPPORTED)]


@pytest.mark.parametrize("n", ["1d", "2d"])
@pytest.mark.parametrize("dims,code", SHARED, ids=[str(s[0]) for s in SHARED])
def test_every_entry_checks_its_sizes(L, n, dims, code):
    for call in (fwd, bwd, append, cached):
        assert call(L, n, **dims) == code, call.__name__


@pytest.mark.parametrize("call,args,code", [
    (fwd, dict(ptr=dict(table=0)), INVALID), (fwd, dict(ptr=dict(buckets=0)), INVALID), (fwd, dict(ptr=dict(out=0)), INVALID),
    (fwd, dict(num_buckets=0), INVALID), (fwd, dict(max_distance=-1), INVALID), (fwd, dict(max_distance=256), UNSUPPORTED),
    (fwd, dict(ptr=dict(q=at(0) + 8)), MISALIGNED), (fwd, dict(ptr=dict(buckets=at(4) + 2)), MISALIGNED),
    (fwd, dict(ptr=dict(out_lo=at(6) + 4)), MISALIGNED), (fwd, dict(ptr=dict(lse=at(7) + 2)), MISALIGNED),
    (fwd, dict(ptr=dict(out=at(0))), INVALID), (fwd, dict(ptr=dict(out_lo=at(5))), INVALID), (fwd, dict(ptr=dict(lse=at(3))), INVALID),
    (bwd, dict(ptr=dict(dtable=at(7))), INVALID), (bwd, dict(ptr=dict(ws=at(9))), INVALID), (bwd, dict(ptr=dict(ws=0)), INVALID),
    (bwd, dict(ws_bytes=100), INVALID), (bwd, dict(ptr=dict(ws=at(13) + 16)), MISALIGNED), (bwd, dict(ptr=dict(dtable=at(12) + 1)), MISALIGNED),
    (bwd, dict(ptr=dict(lse=0)), INVALID), (bwd, dict(max_distance=300), UNSUPPORTED),
    (append, dict(capacity=1), INVALID), (append, dict(capacity=0), INVALID), (append, dict(ptr=dict(start=0)), INVALID),
    (append, dict(ptr=dict(ks=0)), INVALID), (append, dict(ptr=dict(kc=at(3) + 8)), MISALIGNED), (append, dict(ptr=dict(start=at(2) + 2)), MISALIGNED),
    (append, dict(ptr=dict(vc=at(3))), INVALID), (append, dict(ptr=dict(kc=at(0))), INVALID),
    (append, dict(capacity=(1 << 24) + 1), UNSUPPORTED), (append, dict(capacity=1 << 24, H=64, W=64), UNSUPPORTED),
    (cached, dict(ptr=dict(table=0)), INVALID), (cached, dict(ptr=dict(buckets=0)), INVALID), (cached, dict(ptr=dict(vs=0)), INVALID),
    (cached, dict(ptr=dict(out=at(0))), INVALID), (cached, dict(ptr=dict(out=at(1))), INVALID), (cached, dict(ptr=dict(out=at(8) + 4)), MISALIGNED),
    (cached, dict(ptr=dict(ws=at(10) + 128)), MISALIGNED), (cached, dict(capacity=1), INVALID), (cached, dict(max_distance=256), UNSUPPORTED),
    (cached, dict(capacity=4000, ptr=dict(ws=0)), INVALID), (cached, dict(capacity=4000, ws_bytes=64), INVALID),
])
def test_refusals(L, call, args, code):
    assert call(L, **args) == code


def test_workspaces_and_geometry(L):
    assert L.skiparse2d_attn_relbias_bwd_workspace_bytes(1, 2, 8, 8, 2, 32, 9, 4) == -1
    assert L.skiparse2d_attn_relbias_bwd_workspace_bytes(1, 2, 8, 8, 2, 32, 2, 256) == -1
    assert L.skiparse2d_attn_relbias_bwd_workspace_bytes(1, 2, 8, 8, 2, 32, 2, 0) > 0
    assert L.skiparse2d_attn_cached_workspace_bytes(1, 2, 8, 8, 2, 32, 2, 1) == -1
    assert L.skiparse2d_attn_cached_workspace_bytes(1, 1, 8, 8, 2, 32, 2, 1) >= 0
    for dims, n in ((1, "1d"), (2, "2d")):
        assert getattr(L, f"skiparse{n}_cache_frame_tokens")(0, 8, 2) == -1
        for (H, W, P) in [(8, 8, 2), (5, 7, 3), (1, 1, 1), (45, 80, 2), (1, 1, 8)]:
            F = getattr(L, f"skiparse{n}_cache_frame_tokens")(H, W, P)
            for mode in (0, 1):
                sizes = [m.numel() for m in members(H, W, P, mode, dims)]
                assert max(sizes) <= F and sum(sizes) == H * W
            assert F == fps.rearranged_shape((1, 1, H, W, 1, 32), P, dims)[1]


def test_binding_refuses_what_it_cannot_marshal():
    x = torch.zeros((1, 1, 4, 4, 1, 32), dtype=torch.bfloat16)
    table, buckets = torch.zeros((4, 1), dtype=torch.bfloat16), fps.frame_buckets(3, 4, device="cpu")
    with pytest.raises(ValueError):
        fps.skiparse2d_attn_relbias_fwd(x, x, x, table, buckets, 2, 0)
    with pytest.raises(ValueError):
        fps.skiparse_attention(x, x, x, 2, 0, table=table)
    with pytest.raises(ValueError):
        fps.skiparse2d_cache_append(x, x, torch.zeros(1, dtype=torch.int32), None, 2, 0)
    with pytest.raises(ValueError):
        fps.frame_cache(1, 4, 8, 8, 1, 32, 9, device="cpu")
    with pytest.raises(ValueError):
        fps.frame_buckets(256, 8)


@pytest.mark.parametrize("D,NB,causal,window", [(0, 1, False, None), (7, 8, False, None), (31, 32, True, None), (255, 32, False, 5),
                                                (3, 40, True, 2), (16, 3, False, None)])
def test_frame_buckets(D, NB, causal, window):
    """Ranges, masks, and monotone growth with distance in each direction."""
    m = fps.frame_buckets(D, NB, causal=causal, window=window, device="cpu")
    assert m.dtype == torch.int32 and m.numel() == 2 * D + 1 and int(m.max()) < NB
    past, future = m[D:].tolist(), m[:D + 1].flip(0).tolist()
    for u, g in enumerate(past):
        assert (g == -1) == (window is not None and u >= window)
    seen = [g for g in past if g >= 0]
    assert seen == sorted(seen) and seen[0] == 0
    for u, g in enumerate(future):
        if u:
            assert (g == -1) == (causal or (window is not None and u >= window))
    later = [g for g in future[1:] if g >= 0]
    assert later == sorted(later)


def test_empty_cache_layout():
    c = fps.frame_cache(2, 5, 10, 14, 3, 64, 2, device="cpu")
    F = 6 * 8  # padded 12 x 16, classes of 6 x 8
    assert c.k.shape == (8, 3, 5, F, 64) and c.v_scale.shape == (8, 3, 5, 1) and c.capacity == 5
    assert float(c.k.float().abs().max()) == 0 and float(c.k_scale.float().min()) == 1
