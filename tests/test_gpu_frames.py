"""GPU tests of the frame-aware operators: the learned bias by frame distance (forward, backward),
the e4m3 frame cache, and attention over it, against plain fp64 statements of each
(frames_reference.py). Tolerances count roundings, element by element."""

from __future__ import annotations

import pytest
import torch

from frames_reference import (BLOCK, attend, cache_values, cached_reference, check, frames_of, members, pair_bias, quantise,
                              reference, token_classes)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fixed_pattern_sparse_b200 as m
    return m


def normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def inputs(shape, NB, D, causal=False, window=None, seed=1):
    import fixed_pattern_sparse_b200 as m
    q, k, v, g = (normal(shape, seed * 10 + i) for i in range(4))
    return q, k, v, g, normal((NB, shape[4]), seed * 10 + 5, 0.7), m.frame_buckets(D, NB, causal=causal, window=window)


def api(fps, name, dims):
    return getattr(fps, f"skiparse{dims}d_{name}")


# (B, T, H, W, heads, d), P, mode, dims, (NB, D, causal, window)
SHAPES = [
    ((1, 1, 1, 1, 1, 64), 2, 0, 2, (1, 0, False, None)),       # one token; three classes without any
    ((1, 7, 1, 1, 2, 32), 1, 0, 2, (4, 3, True, None)),        # a token a frame, distances past D
    ((2, 5, 3, 5, 2, 64), 1, 1, 2, (8, 4, False, 2)),          # frames of 15 inside a tile
    ((1, 300, 1, 1, 1, 32), 1, 0, 2, (32, 255, True, 40)),     # long: tiles the window hides
    ((1, 3, 8, 16, 2, 128), 1, 0, 2, (6, 2, True, None)),      # frame == key tile
    ((1, 5, 8, 8, 2, 128), 1, 0, 2, (6, 7, False, None)),      # two frames a tile, D > T
    ((1, 4, 16, 12, 1, 128), 1, 1, 2, (5, 3, True, None)),     # frames of 1.5 tiles
    ((1, 5, 4, 24, 1, 128), 1, 0, 2, (5, 1, False, None)),     # frames of 96, D = 1 < T
    ((2, 3, 10, 14, 3, 64), 2, 0, 2, (8, 5, False, None)),     # padded, unequal classes
    ((1, 3, 11, 17, 2, 32), 3, 1, 2, (7, 4, True, None)),
    ((1, 2, 9, 40, 1, 64), 2, 1, 1, (4, 3, False, None)),      # Skiparse-1D
    ((2, 4, 5, 7, 2, 128), 2, 0, 1, (9, 6, True, 3)),
    ((1, 2, 33, 34, 1, 32), 8, 1, 2, (3, 2, False, None)),     # 64 classes, some empty
    ((1, 2, 20, 31, 1, 128), 1, 0, 2, (4, 1, True, None)),     # frames of 620: whole tiles hidden
    ((1, 1, 12, 17, 2, 64), 1, 0, 2, (3, 2, False, None)),     # one frame, one bucket: dtable is 0 but for fp32
    ((1, 3, 9, 15, 2, 64), 1, 0, 2, (4, 2, True, None)),       # 405 queries: a last CTA of 149
]
IDS = ["x".join(map(str, s[0])) + f"_p{s[1]}m{s[2]}d{s[3]}" for s in SHAPES]


@pytest.mark.parametrize("shape,P,mode,dims,bias", SHAPES, ids=IDS)
def test_forward(fps, shape, P, mode, dims, bias):
    q, k, v, _, table, buckets = inputs(shape, *bias)
    out, lse, lo = torch.full_like(q, float("nan")), torch.full(shape[:5], float("nan"), device="cuda"), torch.empty_like(q)
    api(fps, "attn_relbias_fwd", dims)(q, k, v, table, buckets, P, mode, out=out, lse=lse, out_lo=lo)
    assert fps.get_device_status() == 0
    want = reference(q, k, v, table, buckets, P, mode, dims)
    check("out", out, *want["out"])
    check("lse", lse, *want["lse"])
    # out + out_lo lacks the output's own rounding: P's is left, and half a step squared
    value, tol = want["out"]
    check("out + out_lo", out.double() + lo.double(), value, tol - 2.0 ** -8 * value.abs() * (1 - 2.0 ** -7))


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("shape,P,mode,dims,bias", SHAPES, ids=IDS)
def test_backward(fps, shape, P, mode, dims, bias, residual):
    q, k, v, g, table, buckets = inputs(shape, *bias)
    lo = torch.empty_like(q) if residual else None
    out, lse = api(fps, "attn_relbias_fwd", dims)(q, k, v, table, buckets, P, mode, out_lo=lo)
    grads = [torch.full_like(x, float("nan")) for x in (q, k, v, table)]
    api(fps, "attn_relbias_bwd", dims)(q, k, v, out, g, lse, table, buckets, P, mode, *grads, out_lo=lo)
    assert fps.get_device_status() == 0
    want = reference(q, k, v, table, buckets, P, mode, dims, dout=g, exact_d=residual)
    for name, got in zip(("dq", "dk", "dv", "dtable"), grads):
        check(name, got, *want[name])


def test_masks_that_leave_rows_empty(fps):
    """Only later frames visible: the last frame's rows see nothing and give 0, lse -inf, zero
    gradients; a map or a table that masks everything gives that for every row."""
    shape, P = (1, 3, 6, 10, 2, 64), 2
    q, k, v, g, table, _ = inputs(shape, 4, 3)
    later = torch.tensor([0, 1, 2, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, later, P, 0)
    grads = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, later, P, 0)
    assert fps.get_device_status() == 0
    want = reference(q, k, v, table, later, P, 0, dout=g, exact_d=False)
    for name, got in zip(("out", "lse", "dq", "dk", "dv", "dtable"), (out, lse) + grads):
        check(name, got, *want[name])
    assert (out[:, 2] == 0).all() and (lse[:, 2] == -float("inf")).all() and (grads[0][:, 2] == 0).all()
    assert (grads[3][3] == 0).all()  # the bucket of no pair
    zero = torch.zeros(7, dtype=torch.int32, device="cuda")
    for t, m in ((table, torch.full_like(zero, -1)), (table, torch.full_like(zero, 4)), (torch.full_like(table, -float("inf")), zero)):
        out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, t, m, P, 1)
        grads = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, t, m, P, 1)
        assert fps.get_device_status() == 0
        assert (out == 0).all() and (lse == -float("inf")).all() and all((x == 0).all() for x in grads)


def test_table_entries_that_mask(fps):
    """-inf and the type's lowest value in the table mask their bucket, for that head only."""
    shape, P, mode = (1, 4, 8, 8, 2, 32), 2, 1
    q, k, v, g, table, buckets = inputs(shape, 6, 3)
    table[1, 0], table[3, 1] = -float("inf"), torch.finfo(torch.bfloat16).min
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode)
    grads = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, mode)
    want = reference(q, k, v, table, buckets, P, mode, dout=g, exact_d=False)
    for name, got in zip(("out", "lse", "dq", "dk", "dv", "dtable"), (out, lse) + grads):
        check(name, got, *want[name])
    assert grads[3][1, 0] == 0 and grads[3][3, 1] == 0


# calls of enough query tiles for 256-query CTAs, where the tensor core adds the bias of frames of 64 .. 8d tokens
WIDE = [
    ((1, 4, 9, 10, 64, 32), 1, 0, 2, (8, 3, True, None)),       # 90 tokens a frame, five frames a CTA
    ((2, 6, 10, 13, 32, 64), 2, 1, 1, (9, 255, False, 4)),      # Skiparse-1D, frames of up to 36: ten a CTA
    ((1, 3, 13, 17, 60, 64), 1, 0, 2, (5, 1, False, None)),     # 221 tokens, a last CTA of 151
    ((1, 2, 19, 22, 70, 128), 1, 1, 2, (3, 4, True, None)),     # 418 tokens
    ((3, 5, 16, 18, 16, 128), 2, 0, 2, (7, 6, False, 3)),       # 72 tokens, window
    ((1, 5, 8, 16, 60, 32), 1, 0, 2, (1, 0, False, None)),      # D = 0: one bias for all
]


@pytest.mark.parametrize("scale", [1.0, 12.0])  # entries up to 40: their sum with q.k in fp32 keeps within 2^-13
@pytest.mark.parametrize("shape,P,mode,dims,bias", WIDE, ids=["x".join(map(str, s[0])) for s in WIDE])
def test_forward_of_many_queries(fps, shape, P, mode, dims, bias, scale):
    q, k, v, _, table, buckets = inputs(shape, *bias)
    table = (table * scale).contiguous()
    out, lse = api(fps, "attn_relbias_fwd", dims)(q, k, v, table, buckets, P, mode)
    assert fps.get_device_status() == 0
    want = reference(q, k, v, table, buckets, P, mode, dims)
    check("out", out, *want["out"])
    check("lse", lse, *want["lse"])


@pytest.mark.parametrize("shape", [(1, 4, 9, 10, 64, 32), (1, 4, 6, 10, 2, 64)])
@pytest.mark.parametrize("wild", [float("inf"), float("nan")])
def test_entries_that_are_not_finite(fps, shape, wild):
    """A bucket of +inf or NaN makes the rows that see it NaN, and no others."""
    q, k, v, _, table, _ = inputs(shape, 4, 3)
    causal = torch.tensor([-1, -1, -1, 0, 1, 2, 3], dtype=torch.int32, device="cuda")
    table[2, ::2] = wild
    out, _ = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, causal, 1, 0)
    assert fps.get_device_status() == 0
    assert torch.isnan(out[:, 2:, :, :, ::2].float()).all()
    table[2, ::2] = 0
    want, tol = reference(q, k, v, table, causal, 1, 0)["out"]
    check("out", out[:, :2], want[:, :2], tol[:, :2])
    check("out", out[:, :, :, :, 1::2], want[:, :, :, :, 1::2], tol[:, :, :, :, 1::2])


def test_wide_masks_that_leave_rows_empty(fps):
    """As above, in a call of many queries: only later frames visible, or nothing."""
    shape = (1, 4, 9, 10, 64, 32)
    q, k, v, _, table, _ = inputs(shape, 4, 3)
    later = torch.tensor([0, 1, 2, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, later, 1, 0)
    want = reference(q, k, v, table, later, 1, 0)
    check("out", out, *want["out"])
    check("lse", lse, *want["lse"])
    assert (out[:, 3] == 0).all() and (lse[:, 3] == -float("inf")).all()
    low = torch.full_like(table, torch.finfo(torch.bfloat16).min)
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, low, later, 1, 0)
    assert fps.get_device_status() == 0
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_no_mask_and_zero_table_is_the_plain_forward(fps):
    """A zero table without masks says what the plain forward says."""
    for shape, P in (((1, 2, 16, 16, 2, 128), 1), ((2, 3, 10, 14, 2, 64), 2)):
        q, k, v, _, table, buckets = inputs(shape, 3, 2)
        zero = torch.zeros_like(table)
        out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, zero, buckets, P, 0)
        plain, plain_lse = fps.skiparse2d_attn_fwd_lse(q, k, v, P, 0)
        want = reference(q, k, v, zero, buckets, P, 0)
        for x, l in ((out, lse), (plain, plain_lse)):
            check("out", x, *want["out"])
            check("lse", l, *want["lse"])


def test_backward_repeats_bit_for_bit(fps):
    q, k, v, g, table, buckets = inputs((2, 5, 9, 13, 3, 64), 8, 4, causal=True)
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, 2, 0)
    first = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, 2, 0)
    for _ in range(3):
        again = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, 2, 0)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gradients_against_differences(fps):
    """The kernels' gradients against central differences of the fp64 formula along random
    directions of every input (step 1e-4: the difference's own error is about 1e-8)."""
    shape, P, mode = (1, 3, 6, 7, 2, 32), 2, 0
    q, k, v, g, table, buckets = inputs(shape, 5, 3)
    B, T, H, W, h, d = shape
    cls = token_classes(H, W, P, mode, 2).cuda().repeat(T)
    t = frames_of(T, H * W, "cuda")

    def loss(q, k, v, table):
        bias, _ = pair_bias(t, t, table, buckets)
        flat = [x.double().reshape(-1, h, d) for x in (q, k, v)]
        return float((attend(*flat, bias, cls[:, None] == cls[None, :])[0] * g.double().reshape(-1, h, d)).sum())

    lo = torch.empty_like(q)
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode, out_lo=lo)
    grads = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, mode, out_lo=lo)
    tols = reference(q, k, v, table, buckets, P, mode, dout=g)
    args = [x.double() for x in (q, k, v, table)]
    for i, name in enumerate(("dq", "dk", "dv", "dtable")):
        way = torch.randn(args[i].shape, generator=torch.Generator("cpu").manual_seed(i), dtype=torch.float64).cuda()
        ends = [loss(*(a + s * 1e-4 * way if j == i else a for j, a in enumerate(args))) for s in (1, -1)]
        want = (ends[0] - ends[1]) / 2e-4
        assert abs(float((grads[i].double() * way).sum()) - want) <= float((tols[name][1] * way.abs()).sum()) + 1e-5, name


def test_autograd(fps):
    shape, P, mode = (1, 3, 10, 14, 2, 64), 2, 1
    q, k, v, g, table, buckets = inputs(shape, 6, 3, causal=True)
    leaves = [x.clone().requires_grad_() for x in (q, k, v, table)]
    for dims in (2, 1):
        for x in leaves:
            x.grad = None
        out = fps.skiparse_attention(*leaves[:3], P, mode, dims=dims, table=leaves[3], buckets=buckets)
        out.backward(g.transpose(2, 3).contiguous().transpose(2, 3))  # not contiguous
        want = reference(q, k, v, table, buckets, P, mode, dims, dout=g)
        check("out", out.detach(), *want["out"])
        for name, x in zip(("dq", "dk", "dv", "dtable"), leaves):
            check(name, x.grad, *want[name])


def test_second_derivatives_are_refused(fps):
    q, k, v, _, table, buckets = inputs((1, 2, 4, 4, 1, 32), 2, 1)
    leaf = q.requires_grad_()
    (grad,) = torch.autograd.grad(fps.skiparse_attention(leaf, k, v, 1, 0, table=table, buckets=buckets).float().square().sum(), leaf,
                                  create_graph=True)
    with pytest.raises(RuntimeError):
        grad.float().sum().backward()


def test_captured_forward_and_backward(fps):
    """The entry points captured into a graph, while an eager graph of the same leaves lives; the
    replay on new inputs gives what the eager calls give."""
    shape, P, mode = (1, 4, 8, 12, 2, 64), 2, 0
    q, k, v, g, table, buckets = inputs(shape, 6, 3, causal=True)
    leaves = [x.clone().requires_grad_() for x in (q, k, v, table)]
    eager = fps.skiparse_attention(*leaves[:3], P, mode, table=leaves[3], buckets=buckets)

    def step():
        out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode)
        return (out, *fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, mode))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (7, 8):
        for x, y in zip((q, k, v, g), inputs(shape, 6, 3, seed=seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))
    eager.backward(g)
    assert fps.get_device_status() == 0


def test_own_stream_and_workspace(fps):
    shape, P, mode = (1, 5, 12, 14, 2, 64), 2, 0
    q, k, v, g, table, buckets = inputs(shape, 6, 3)
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode)
    want = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, mode)
    need = fps._lib.lib().skiparse2d_attn_relbias_bwd_workspace_bytes(*shape, P, 3)
    ws = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")  # NaNs: nothing may rely on it
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, l2 = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode, stream=side)
    got = fps.skiparse2d_attn_relbias_bwd(q, k, v, o2, g, l2, table, buckets, P, mode, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, lse) + want, (o2, l2) + got))
    assert (ws[need:] == 0xff).all()


# ------------------------------------------------------------------------------------ the cache

CACHES = [
    ((1, 1, 1, 1, 1, 64), 2, 0, 2, 3, [5]),
    ((2, 2, 10, 14, 3, 64), 2, 0, 2, 5, [0, 4]),
    ((1, 3, 19, 37, 2, 32), 2, 1, 2, 3, [8]),
    ((2, 1, 9, 21, 2, 128), 3, 1, 2, 4, [2, 3]),
    ((1, 2, 12, 25, 2, 128), 1, 0, 2, 2, [1]),
    ((2, 2, 9, 10, 1, 64), 2, 1, 1, 4, [3, 0]),
    ((1, 1, 33, 34, 1, 32), 8, 0, 2, 2, [7]),
]


@pytest.mark.parametrize("shape,P,mode,dims,cap,start", CACHES, ids=lambda x: str(x) if isinstance(x, (int, list)) else "x".join(map(str, x)))
def test_append(fps, shape, P, mode, dims, cap, start):
    """Codes and scales equal the definition's, value for value; other slots and unused places stay."""
    B, T, H, W, h, d = shape
    k, v = normal(shape, 3, 2.0), normal(shape, 4)
    v[..., : d // 2] *= 2.0 ** -20  # wide ranges inside a block
    cache = fps.frame_cache(B, cap, H, W, h, d, P, dims)
    for x in cache:
        x.view(torch.uint8).fill_(0x5a)
    api(fps, "cache_append", dims)(k, v, torch.tensor(start, dtype=torch.int32, device="cuda"), cache, P, mode)
    assert fps.get_device_status() == 0
    want = {n: getattr(cache, n).view(torch.uint8).clone().fill_(0x5a) for n in cache._fields}
    for b in range(B):
        for c, at in enumerate(members(H, W, P, mode, dims)):
            for t in range(T):
                slot, seq = (start[b] + t) % cap, b * P * P + c
                for name, x in (("k", k), ("v", v)):
                    y = x[b, t].reshape(H * W, h, d)[at.cuda()].double().transpose(0, 1)  # h, n, d
                    for first in range(0, at.numel(), BLOCK):
                        codes, e = quantise(y[:, first:first + BLOCK])
                        want[name][seq, :, slot, first:first + BLOCK][:, : codes.shape[1]] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
                        want[name + "_scale"][seq, :, slot, first // BLOCK] = (e + 127).to(torch.uint8)
    for n in cache._fields:
        got, ref = getattr(cache, n).view(torch.uint8), want[n]
        if n in ("k", "v"):  # -0 and +0 are one value
            got, ref = (torch.where(x == 0x80, 0, x) for x in (got, ref))
        assert torch.equal(got, ref), n


def test_append_extremes(fps):
    """Zero blocks, bf16's largest and smallest values, ties, infinities and NaN."""
    shape = (1, 1, 2, 4, 1, 32)
    for fill in (0.0, 3.3895e38, 1e-40, 448.0, 450.0, 2.0 ** -118):
        x = torch.full(shape, fill).to(torch.bfloat16).cuda()
        cache = fps.frame_cache(1, 1, 2, 4, 1, 32, 1)
        fps.skiparse2d_cache_append(x, -x, torch.zeros(1, dtype=torch.int32, device="cuda"), cache, 1, 0)
        codes, want_e = quantise(x[0, 0].double().reshape(1, 8, 32))
        assert int(cache.k_scale.view(torch.uint8)[0, 0, 0, 0]) == int(want_e) + 127
        assert torch.equal(cache.k[0, 0, 0].double(), codes[0]) and torch.equal(cache.v[0, 0, 0].double(), -codes[0])
    for bad in (float("inf"), float("nan")):
        x = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
        x[0, 0, 1, 2, 0, 5] = bad
        cache = fps.frame_cache(1, 1, 2, 4, 1, 32, 1)
        start = torch.zeros(1, dtype=torch.int32, device="cuda")
        fps.skiparse2d_cache_append(x, x, start, cache, 1, 0)
        assert torch.isnan(cache.k_scale.float()).all() and torch.isnan(cache.k.float()).all()
        out = fps.skiparse2d_attn_cached(torch.ones_like(x), cache, start, 1, 0)
        assert torch.isnan(out.float()).all()


def test_every_code_reads_as_its_value(fps):
    """One key with weight 1: the output is the value that code and scale stand for, exactly."""
    codes = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f], dtype=torch.uint8)
    codes = torch.cat([codes, torch.zeros(2, dtype=torch.uint8)]).reshape(2, 4, 32).cuda()  # 8 rows of 32
    for byte in (17, 100, 119, 127, 134, 135, 180, 240):
        cache = fps.frame_cache(1, 8, 1, 1, 1, 32, 1)
        cache.v.view(torch.uint8)[0, 0, :, 0] = codes.reshape(8, 32)
        cache.v_scale.view(torch.uint8).fill_(byte)
        q = torch.zeros((1, 1, 1, 1, 1, 32), dtype=torch.bfloat16, device="cuda")
        for f in range(8):  # the newest frame alone is visible
            only = torch.tensor([-1, 0, -1], dtype=torch.int32, device="cuda")
            table = torch.zeros((1, 1), dtype=torch.bfloat16, device="cuda")
            start = torch.tensor([f], dtype=torch.int32, device="cuda")
            out = fps.skiparse2d_attn_cached(q, cache, start, 1, 0, table=table, buckets=only)
            want = codes.reshape(8, 32)[f].view(torch.float8_e4m3fn).double() * 2.0 ** (byte - 127)
            assert torch.equal(out.double().flatten(), want.to(torch.bfloat16).double()), (byte, f)


# shape, P, mode, dims, capacity, start, (NB, D, causal, window) or None
READS = [
    ((1, 1, 1, 1, 1, 64), 2, 0, 2, 3, [2], None),
    ((2, 1, 2, 2, 2, 128), 2, 0, 2, 700, [650, 3], (8, 100, True, None)),     # single tokens, long history
    ((1, 1, 2, 2, 3, 32), 1, 1, 2, 900, [2000], (8, 255, True, None)),        # wrapped, past the largest distance
    ((2, 1, 7, 9, 2, 64), 2, 1, 2, 40, [33, 100], (6, 20, True, 10)),         # a dozen tokens a frame
    ((3, 2, 10, 14, 2, 64), 2, 0, 2, 6, [0, 3, 9], None),
    ((2, 3, 11, 17, 2, 32), 3, 1, 2, 7, [4, 50], (5, 4, False, None)),
    ((1, 2, 20, 31, 1, 128), 1, 0, 2, 5, [7], (5, 9, True, None)),            # 620 tokens a frame, ring of odd length
    ((2, 4, 9, 10, 2, 128), 2, 1, 1, 9, [5, 20], (5, 9, True, 5)),            # Skiparse-1D
    ((1, 1, 40, 50, 1, 64), 2, 0, 2, 12, [11], (9, 12, True, None)),
    ((1, 1, 4, 4, 2, 64), 1, 0, 2, 300, [299], None),                         # 16 tokens a frame
    ((1, 1, 17, 1, 1, 128), 1, 0, 2, 200, [120], (9, 12, True, None)),        # 17 tokens a frame
    ((1, 2, 13, 12, 1, 64), 1, 0, 2, 8, [6], (9, 12, True, None)),            # 312 queries: a last CTA of 56
    ((1, 1, 20, 20, 1, 128), 1, 1, 2, 9, [20], None),                         # 400 queries: of 144
]


@pytest.mark.parametrize("shape,P,mode,dims,cap,start,bias", READS, ids=lambda x: "x".join(map(str, x)) if isinstance(x, tuple) else str(x))
def test_attention_over_the_cache(fps, shape, P, mode, dims, cap, start, bias):
    B, T, H, W, h, d = shape
    cache = fps.frame_cache(B, cap, H, W, h, d, P, dims)
    clip = (B, cap) + shape[2:]
    fill = torch.zeros(B, dtype=torch.int32, device="cuda")
    api(fps, "cache_append", dims)(normal(clip, 21), normal(clip, 22), fill, cache, P, mode)
    first = torch.tensor(start, dtype=torch.int32, device="cuda")
    api(fps, "cache_append", dims)(normal(shape, 23), normal(shape, 24), first, cache, P, mode)
    q = normal(shape, 25)
    table = buckets = None
    if bias:
        table, buckets = normal((bias[0], h), 26, 0.7), fps.frame_buckets(bias[1], bias[0], causal=bias[2], window=bias[3])
    out, lse = torch.full_like(q, float("nan")), torch.full(shape[:5], float("nan"), device="cuda")
    api(fps, "attn_cached", dims)(q, cache, first, P, mode, table=table, buckets=buckets, out=out, lse=lse)
    assert fps.get_device_status() == 0
    want, tol, want_lse = cached_reference(q, cache, start, P, mode, table, buckets, dims)
    check("out", out, want, tol)
    check("lse", lse, want_lse, torch.full_like(want_lse, 1e-4))


@pytest.mark.parametrize("cap,T,shape", [(6, 2, (10, 14, 2, 64)), (400, 1, (2, 2, 2, 128)), (500, 1, (7, 9, 1, 64))])
def test_skipped_sequences_are_left_alone(fps, cap, T, shape):
    B, P, mode = 3, 2, 0
    H, W, h, d = shape
    cache = fps.frame_cache(B, cap, H, W, h, d, P)
    fps.skiparse2d_cache_append(normal((B, cap) + shape, 1), normal((B, cap) + shape, 2), torch.zeros(B, dtype=torch.int32, device="cuda"), cache, P, mode)
    start = [cap - T, -1, (1 << 30) + 1]
    first = torch.tensor(start, dtype=torch.int32, device="cuda")
    before = [x.view(torch.uint8).clone() for x in cache]
    full = (B, T) + shape
    fps.skiparse2d_cache_append(normal(full, 3), normal(full, 4), first, cache, P, mode)
    for x, y in zip(cache, before):
        assert torch.equal(x.view(torch.uint8)[P * P:], y[P * P:])
    q, out = normal(full, 5), torch.full(full, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(full[:5], 7.0, device="cuda")
    fps.skiparse2d_attn_cached(q, cache, first, P, mode, out=out, lse=lse)
    assert fps.get_device_status() == 0
    assert (out[1:] == 7).all() and (lse[1:] == 7).all()
    want, tol, _ = cached_reference(q, cache, [start[0], -1, -1], P, mode)
    check("out", out[:1], want[:1], tol[:1])


@pytest.mark.parametrize("d,cap,start", [(32, 9, [8, 30, 4]), (64, 9, [8, 30, -1]), (128, 9, [3, -1, 20])])
def test_last_wave_is_cut(fps, d, cap, start):
    """More query tiles than one wave: the keys of the tiles behind the last full wave, those of the last
    sequence, are cut into parts and joined."""
    shape, P, mode = (3, 1, 29, 41, 13, d), 2, 0
    B, T, H, W, h, _ = shape
    need = fps._lib.lib().skiparse2d_attn_cached_workspace_bytes(*shape, P, cap)
    assert 0 < need < B * T * H * W * h * d * 4  # parts of some rows only
    cache = fps.frame_cache(B, cap, H, W, h, d, P)
    fill = torch.zeros(B, dtype=torch.int32, device="cuda")
    fps.skiparse2d_cache_append(normal((B, cap, H, W, h, d), 41), normal((B, cap, H, W, h, d), 42), fill, cache, P, mode)
    first = torch.tensor(start, dtype=torch.int32, device="cuda")
    fps.skiparse2d_cache_append(normal(shape, 43), normal(shape, 44), first, cache, P, mode)
    q, table, buckets = normal(shape, 45), normal((9, h), 46, 0.7), fps.frame_buckets(12, 9, causal=True)
    out, lse = torch.full_like(q, 7.0), torch.full(shape[:5], 7.0, device="cuda")
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    fps.skiparse2d_attn_cached(q, cache, first, P, mode, table=table, buckets=buckets, out=out, lse=lse, workspace=ws)
    assert fps.get_device_status() == 0
    want, tol, want_lse = cached_reference(q, cache, start, P, mode, table, buckets)
    for b in range(B):
        if start[b] < 0:
            assert (out[b] == 7).all() and (lse[b] == 7).all()
        else:
            check("out", out[b], want[b], tol[b])
            check("lse", lse[b], want_lse[b], torch.full_like(want_lse[b], 1e-4))


def test_a_row_without_visible_keys(fps):
    """A map that shows only frames further back than the cache holds."""
    for cap, shape in ((3, (1, 1, 8, 8, 2, 64)), (600, (1, 1, 2, 2, 2, 64))):
        cache = fps.frame_cache(1, cap, *shape[2:], 2)
        start = torch.tensor([1], dtype=torch.int32, device="cuda")
        x = normal(shape, 1)
        fps.skiparse2d_cache_append(x, x, start, cache, 2, 0)
        far = torch.tensor([-1] * 9 + [0] * 2, dtype=torch.int32, device="cuda")  # distances 4 and 5 of D = 5
        out, lse = torch.full_like(x, 9.0), torch.full(shape[:5], 9.0, device="cuda")
        fps.skiparse2d_attn_cached(x, cache, start, 2, 0, table=torch.zeros((1, 2), dtype=torch.bfloat16, device="cuda"),
                                   buckets=far, out=out, lse=lse)
        assert fps.get_device_status() == 0
        assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("shape,cap", [((2, 1, 10, 14, 2, 64), 5), ((2, 1, 2, 2, 2, 64), 600)])
def test_streaming_captured_once(fps, shape, cap):
    """Frame by frame through one captured graph (append, attend, advance), past the ring's end, with
    a bias: each step equals the reference on the cache as it stands; the trained form of the same
    bias over all frames agrees with the last step within the cache's own rounding."""
    B, T, H, W, h, d = shape
    P, mode, steps = 2, 1, 9
    table, buckets = normal((6, h), 2, 0.7), fps.frame_buckets(7, 6, causal=True)
    clip = [normal((B, steps) + shape[2:], 30 + i) for i in range(3)]
    cache = fps.frame_cache(B, cap, H, W, h, d, P)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = (x[:, :1].clone() for x in clip)
    out = torch.empty_like(q)

    def step():
        fps.skiparse2d_cache_append(k, v, start, cache, P, mode)
        fps.skiparse2d_attn_cached(q, cache, start, P, mode, table=table, buckets=buckets, out=out)
        start.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    start.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in range(steps):
        for x, y in zip((q, k, v), clip):
            x.copy_(y[:, s:s + 1])
        graph.replay()
        torch.cuda.synchronize()
        assert fps.get_device_status() == 0 and int(start[0]) == s + 1
        want, tol, _ = cached_reference(q, cache, [s] * B, P, mode, table, buckets)
        check(f"step {s}", out, want, tol)
        if s + 1 == min(cap, steps):  # no frame has left the ring yet
            whole, _ = fps.skiparse2d_attn_relbias_fwd(*(x[:, : s + 1].contiguous() for x in clip), table, buckets, P, mode)
            a, b = out[:, 0].double(), whole[:, s].double()
            assert float((a - b).norm() / b.norm()) < 0.1  # codes of 3 mantissa bits: 2^-4 each


def test_cached_uses_its_own_stream_and_workspace(fps):
    shape, cap = (1, 1, 2, 2, 2, 128), 3000
    cache = fps.frame_cache(1, cap, 2, 2, 2, 128, 2)
    for x in (cache.k, cache.v):
        x.copy_(normal(x.shape, 5, 1.0, torch.float32).to(torch.float8_e4m3fn))
    q, start = normal(shape, 6), torch.tensor([2900], dtype=torch.int32, device="cuda")
    want = fps.skiparse2d_attn_cached(q, cache, start, 2, 0)
    need = fps._lib.lib().skiparse2d_attn_cached_workspace_bytes(*shape, 2, cap)
    assert need > 0
    ws = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fps.skiparse2d_attn_cached(q, cache, start, 2, 0, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and (ws[need:] == 0xff).all()


def test_offsets_beyond_32_bits(fps):
    """A cache whose codes pass 2^32 bytes: the last sequence's and head's rows are read and written."""
    shape, cap, P = (2, 1, 30, 32, 12, 128), 1600, 1
    F = 960
    cache = fps.frame_cache(2, cap, 30, 32, 12, 128, P)
    assert cache.k.numel() > 2 ** 32
    start = torch.tensor([-1, 1598], dtype=torch.int32, device="cuda")
    k, v = normal(shape, 1), normal(shape, 2)
    fps.skiparse2d_cache_append(k, v, start, cache, P, 0)
    y = k[1, 0].reshape(F, 12, 128)[:, 11].double()
    codes, e = quantise(y.reshape(15, 64, 128))
    assert torch.equal(cache.k[1, 11, 1598].double(), codes.reshape(F, 128))
    only = torch.tensor([-1, 0, -1], dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 12), dtype=torch.bfloat16, device="cuda")
    q = normal(shape, 3)
    out = fps.skiparse2d_attn_cached(q, cache, start, P, 0, table=table, buckets=only)
    assert fps.get_device_status() == 0
    vals = [cache_values(cache, n, 1, 11, 1598, F) for n in ("k", "v")]
    o, _, p = attend(q[1, 0].reshape(F, 12, 128)[:, 11:].double(), vals[0][:, None], vals[1][:, None],
                     torch.zeros(1, F, F, dtype=torch.float64, device="cuda"), torch.ones(F, F, dtype=torch.bool, device="cuda"))
    tol = (2.0 ** -8 + 2.0 ** -13) * torch.einsum("hqk,khd->qhd", p, vals[1][:, None].abs()) + 2.0 ** -8 * o.abs() + 1e-6
    check("out", out[1, 0].reshape(F, 12, 128)[:, 11:], o, tol)


# ---------------------------------------------------------------------------- failure detection

def test_lost_arrivals_time_out_and_recover(fps):
    """A producer that never signals: the call reports the timeout, and the next one is right."""
    L = fps._lib.lib()
    shape, P, mode = (1, 3, 10, 14, 2, 64), 2, 0
    q, k, v, g, table, buckets = inputs(shape, 6, 3)
    cache = fps.frame_cache(1, 3, *shape[2:], P)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    fps.skiparse2d_cache_append(k, v, start, cache, P, mode)
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode)
    calls = [(1, lambda: fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode)[0]),
             (2, lambda: fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, mode)[1]),
             (1, lambda: fps.skiparse2d_attn_cached(q, cache, start, P, mode))]
    for kind, call in calls:
        want = call()
        assert fps.get_device_status() == 0
        prev = L.skiparse_set_wait_limit_ns(100_000_000)
        try:
            assert L.skiparse_debug_inject_fault(kind) == 0
            call()
            assert fps.get_device_status() == 5
        finally:
            L.skiparse_debug_inject_fault(0)
            L.skiparse_set_wait_limit_ns(prev)
        assert torch.equal(call(), want) and fps.get_device_status() == 0


def test_debug_build_reports_nothing_and_matches(fps, monkeypatch):
    """The bounds-checking build on the same calls: no row outside, the same bits."""
    import os
    from fixed_pattern_sparse_b200 import build as libbuild
    if not os.path.exists(fps._lib.DEBUG_LIB_PATH):
        libbuild.build(debug=True)

    def calls(shape, P, mode, cap):
        q, k, v, g, table, buckets = inputs(shape, 6, 3, causal=True)
        cache = fps.frame_cache(shape[0], cap, *shape[2:], P)
        start = torch.full((shape[0],), cap - 1, dtype=torch.int32, device="cuda")
        fps.skiparse2d_cache_append(k, v, start, cache, P, mode)
        out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, mode)
        grads = fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, mode)
        c = fps.skiparse2d_attn_cached(q, cache, start, P, mode, table=table, buckets=buckets)
        return (out, lse, *grads, c, *(x.view(torch.uint8) for x in cache)), fps.get_device_status()

    for args in (((2, 2, 11, 17, 2, 64), 3, 1, 5), ((1, 1, 3, 5, 2, 128), 2, 0, 300), ((1, 3, 20, 30, 1, 32), 2, 0, 4)):
        release, st = calls(*args)
        assert st == 0
        with monkeypatch.context() as m:
            debug = fps._lib.debug_lib()
            m.setattr(fps.frames, "lib", lambda: debug)
            m.setattr(fps, "lib", lambda: debug)
            checked, st = calls(*args)
        assert st == 0
        assert all(torch.equal(a, b) for a, b in zip(release, checked))
