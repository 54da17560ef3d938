"""GPU tests of the attention over the e4m3 frame cache where the blocks' scales differ widely, between
frames and between the 64-token blocks of one frame, in both kernels (up to 32 queries a class, and
more): a block must count by its own values, whatever the scale of its neighbours and of what the bias masks.

Tolerances, element by element, against fp64 over the cache's own values: the weights enter their
product as f16, half a step 2^-11 relative; 2^-13 covers the fp32 arithmetic (scores, exponentials, sums, as
in frames_reference.py); the output is rounded to bf16 once, 2^-8. A weight times its block's scale that
lies far below the row's largest is an f16 subnormal, off by up to 2^-32 of that largest: times a code of
at most 448, for every key."""

from __future__ import annotations

import math

import pytest
import torch

from frames_reference import attend, cache_values, check, frames_of, pair_bias

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fixed_pattern_sparse_b200 as m
    return m


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)).cuda()


def expected(q, cache, start, table, buckets):
    """out with its tolerance, and lse, of one sequence with a single class."""
    _, T, H, W, h, d = q.shape
    n, cap = H * W, cache.capacity
    times = list(range(max(0, start + T - cap), start + T))
    tq, tk = frames_of(T, n, "cuda", start), torch.tensor(times, device="cuda").repeat_interleave(n)
    k, v = (torch.stack([torch.cat([cache_values(cache, m, 0, i, t % cap, n) for t in times]) for i in range(h)], 1) for m in "kv")
    e = torch.stack([torch.cat([cache.v_scale[0, i, t % cap].double().repeat_interleave(64)[:n] for t in times]) for i in range(h)])
    bias, _ = pair_bias(tq, tk, table, buckets)
    o, lse, p = attend(q[0].reshape(T * n, h, d).double(), k, v, bias, torch.ones(T * n, tk.numel(), dtype=torch.bool, device="cuda"))
    top = torch.minimum(p.amax(-1) * e.amax(-1)[:, None], 2.0 ** 8 * (p * e[:, None]).amax(-1))
    tol = (2.0 ** -11 + 2.0 ** -13) * torch.einsum("hqk,khd->qhd", p, v.abs()) + 2.0 ** -8 * o.abs()
    tol += (tk.numel() * 448 * 2.0 ** -32 * top).t()[..., None]
    return o.reshape(q.shape), tol.reshape(q.shape), lse.reshape(q.shape[:5])


# T, H, W, heads, d, capacity, frames before: 12 queries, keys in one part and in several; 128-query CTAs over a
# ring that has turned, over many frames cut into parts, and of small frames; 256-query CTAs
CALLS = [(1, 3, 4, 2, 64, 8, 6), (1, 3, 4, 2, 128, 400, 900), (2, 3, 5, 2, 32, 9, 3), (2, 10, 10, 2, 128, 7, 12),
         (2, 10, 10, 2, 32, 7, 5), (1, 10, 15, 2, 64, 60, 70), (1, 5, 7, 2, 64, 9, 31), (1, 10, 16, 148, 64, 4, 10)]


def parity_map(D, masked):
    """A bucket for even distances and one for odd ones, the even ones masked or not."""
    u = torch.arange(-D, D + 1).abs()
    return torch.where(u % 2 == 0, 0, -1 if masked else 1).to(torch.int32).cuda()


@pytest.mark.parametrize("spread", [4, 8, 9, 14, 16, 24, 30, 60])
@pytest.mark.parametrize("kind", ["v", "v_masked", "k", "k_and_v"])
@pytest.mark.parametrize("call", CALLS, ids=lambda c: "x".join(map(str, c)))
def test_frames_of_unequal_scale(fps, call, kind, spread):
    """Every other frame is 2^spread times larger. Its values get weights 2^-spread by the bias, so that both
    kinds count ("v"), or are masked, so that rows see one kind only ("v_masked"); or its keys are the
    larger ones, in columns where q is 0, so that the others alone decide the scores ("k"); or both."""
    T, H, W, h, d, cap, start = call
    shape = (1, cap, H, W, h, d)
    big = 2.0 ** (spread * (torch.arange(cap) % 2)).cuda().view(1, cap, 1, 1, 1, 1)
    k, v, q = normal(shape, 1), normal(shape, 2), normal((1, T) + shape[2:], 3)
    if kind != "k":
        v = v * big
    if kind in ("k", "k_and_v"):
        odd = (big > 1).expand(shape[:-1] + (d // 2,))
        k[..., d // 2:] = torch.where(odd, k[..., d // 2:] * big, 0.0)
        k[..., :d // 2] = torch.where(odd, 0.0, k[..., :d // 2])
        k[..., :4] = 0  # and q is large where no key is
        q[..., d // 2:] = 0
        q[..., :4] *= 2.0 ** 16
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    cache = fps.frame_cache(1, cap, H, W, h, d, 1)
    fps.skiparse2d_cache_append(k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), cache, 1, 0)
    # the newest frame's distance parity is that of its keys' slot where the capacity is even
    newest_is_big = ((start + T - 1) % cap) % 2 == 1
    low = -spread * math.log(2.0) if kind in ("v", "k_and_v") else 0.0
    table = torch.tensor([[low], [0.0]] if newest_is_big else [[0.0], [low]]).repeat(1, h).to(torch.bfloat16).cuda()
    if kind == "v_masked":
        buckets = parity_map(255, True)
    else:
        buckets = parity_map(255, False)
    first = torch.tensor([start], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:5], float("nan"), device="cuda")
    fps.skiparse2d_attn_cached(q, cache, first, 1, 0, table=table, buckets=buckets, out=out, lse=lse)
    assert fps.get_device_status() == 0
    want, tol, want_lse = expected(q, cache, start, table, buckets)
    check("lse", lse, want_lse, torch.full_like(want_lse, 1e-4))
    check("out", out, want, tol)


@pytest.mark.parametrize("spread", [6, 12, 25, 40])
@pytest.mark.parametrize("call", [c for c in CALLS if c[1] * c[2] > 64], ids=lambda c: "x".join(map(str, c)))
def test_blocks_of_unequal_scale(fps, call, spread):
    """Every other 64-token block of each frame is 2^spread times larger in V, its keys such that its weights
    are about 2^-spread; K's blocks alternate the other way, in columns where q is 0."""
    T, H, W, h, d, cap, start = call
    shape = (1, cap, H, W, h, d)
    place = torch.arange(H * W, device="cuda").view(1, 1, H, W, 1, 1)
    odd = (place // 64) % 2 == 1
    k, v, q = normal(shape, 4) * 0.5, normal(shape, 5), normal((1, T) + shape[2:], 6) * 0.5
    v = v * torch.where(odd, 2.0 ** spread, 1.0)
    k[..., -8:] = torch.where(odd, 0.0, k[..., -8:] * 2.0 ** spread)
    q[..., -8:] = 0
    q[..., 0] = 4.0  # q.k / sqrt(d) = -spread ln 2 in the first column
    k[..., :1] = torch.where(odd, -spread * math.log(2.0) * math.sqrt(d) / 4.0, 0.0)
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    cache = fps.frame_cache(1, cap, H, W, h, d, 1)
    fps.skiparse2d_cache_append(k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), cache, 1, 0)
    table, buckets = torch.zeros((1, h), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    first = torch.tensor([start], dtype=torch.int32, device="cuda")
    want, tol, want_lse = expected(q, cache, start, table, buckets)
    for bias in (dict(), dict(table=table, buckets=buckets)):
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:5], float("nan"), device="cuda")
        fps.skiparse2d_attn_cached(q, cache, first, 1, 0, out=out, lse=lse, **bias)
        assert fps.get_device_status() == 0
        check("lse", lse, want_lse, torch.full_like(want_lse, 1e-4))
        check("out", out, want, tol)


@pytest.mark.parametrize("call", CALLS, ids=lambda c: "x".join(map(str, c)))
def test_frames_of_zeros(fps, call):
    """A frame of zeros, whose scale is the smallest there is, beside ordinary ones."""
    T, H, W, h, d, cap, start = call
    shape = (1, cap, H, W, h, d)
    q, k, v = (normal(s, 7 + i).to(torch.bfloat16) for i, s in enumerate([(1, T) + shape[2:], shape, shape]))
    k[:, 1], v[:, 1] = 0, 0
    cache = fps.frame_cache(1, cap, H, W, h, d, 1)
    fps.skiparse2d_cache_append(k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), cache, 1, 0)
    table, buckets = normal((4, h), 11).to(torch.bfloat16), fps.frame_buckets(5, 4, causal=True)
    first = torch.tensor([start], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:5], float("nan"), device="cuda")
    fps.skiparse2d_attn_cached(q, cache, first, 1, 0, table=table, buckets=buckets, out=out, lse=lse)
    assert fps.get_device_status() == 0
    want, tol, want_lse = expected(q, cache, start, table, buckets)
    check("lse", lse, want_lse, torch.full_like(want_lse, 1e-4))
    check("out", out, want, tol)


@pytest.mark.parametrize("call", [CALLS[0], CALLS[3], CALLS[7]], ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("wide", [False, True])
def test_a_block_that_is_not_finite(fps, call, wide):
    """A frame with a NaN makes every row that attends to it NaN, whether or not the other scales differ."""
    T, H, W, h, d, cap, start = call
    shape = (1, cap, H, W, h, d)
    q, k, v = (normal(s, 7 + i).to(torch.bfloat16) for i, s in enumerate([(1, T) + shape[2:], shape, shape]))
    if wide:
        v[:, 0] *= 2.0 ** 30
    v[0, 1, 0, 0, 0, 3], k[0, 2, H - 1, W - 1, -1, 0] = float("nan"), float("inf")
    cache = fps.frame_cache(1, cap, H, W, h, d, 1)
    fps.skiparse2d_cache_append(k, v, torch.zeros(1, dtype=torch.int32, device="cuda"), cache, 1, 0)
    out = torch.zeros_like(q)
    fps.skiparse2d_attn_cached(q, cache, torch.tensor([start], dtype=torch.int32, device="cuda"), 1, 0, out=out)
    assert fps.get_device_status() == 0
    assert torch.isnan(out[..., 0, :].float()).all() and torch.isnan(out[..., -1, :].float()).all()
