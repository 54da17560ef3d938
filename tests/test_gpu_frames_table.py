"""GPU tests of large entries in the table of the bias by frame distance: those at or below -65504 (fp16's lowest
value, in bf16 -65536) mask like a bucket outside the table, whatever their size, rows that see nothing else
included; those within +-65504 count, and a constant one leaves the softmax as it is.

A score near c is rounded to fp32, by up to 2^-24 |c| in each of its additions and conversions (the tensor
core's additions truncate: twice that), and so is the log-sum-exp that the backward pass reads: fewer than
sixteen of these together, so that weights and gradients are off by 2^-20 (|c| + 16) relative (16: more than any
q.k / sqrt(d) here), beside the tolerance without a table. The bounds of frames_reference.py hold 2^-8 of the sums of
magnitudes that this factor applies to, those of dtable 2^-13."""

from __future__ import annotations

import math

import pytest
import torch

from frames_reference import check, reference

pytestmark = pytest.mark.gpu

NAMES = ("out", "lse", "dq", "dk", "dv", "dtable")
# few queries, frames of 140 and of 12 tokens a class; many, with the bias added by the tensor core
SHAPES = [((1, 4, 10, 14, 2, 64), 1), ((2, 5, 7, 7, 2, 32), 2), ((1, 4, 9, 10, 64, 32), 1), ((1, 3, 16, 24, 1, 128), 2)]


@pytest.fixture(scope="module")
def fps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fixed_pattern_sparse_b200 as m
    return m


def normal(shape, seed, std=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def run(fps, q, k, v, g, table, buckets, P):
    lo = torch.empty_like(q)
    out, lse = fps.skiparse2d_attn_relbias_fwd(q, k, v, table, buckets, P, 0, out_lo=lo)
    got = (out, lse, *fps.skiparse2d_attn_relbias_bwd(q, k, v, out, g, lse, table, buckets, P, 0, out_lo=lo))
    assert fps.get_device_status() == 0
    return got


@pytest.mark.parametrize("value", [-65504.0, -1e9, -9e29, -1e30, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("shape,P", SHAPES, ids=lambda x: "x".join(map(str, x)) if isinstance(x, tuple) else f"p{x}")
def test_low_entries_mask(fps, shape, P, value):
    """In the buckets of some distances, and in every bucket that the last frame sees."""
    q, k, v, g = (normal(shape, i) for i in range(4))
    for causal_low in (False, True):
        buckets = torch.tensor([0, 1, 2, 3, 2, 1, 0], dtype=torch.int32, device="cuda")
        table = normal((4, shape[4]), 5, 0.7)
        table[1] = value
        if causal_low:  # later frames alone count
            buckets = torch.tensor([0, 2, 3, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
        masks = torch.where(table == table[1:2], -math.inf, table)
        masks[1] = -math.inf
        got = run(fps, q, k, v, g, table, buckets, P)
        want = reference(q, k, v, masks, buckets, P, 0, dout=g)
        for name, x in zip(NAMES, got):
            check(name, x, *want[name])
        if causal_low:
            assert (got[0][:, -1] == 0).all() and (got[1][:, -1] == -math.inf).all() and (got[2][:, -1] == 0).all()


@pytest.mark.parametrize("value", [4096.0, -4096.0, 32768.0, -65280.0, 65280.0])
@pytest.mark.parametrize("shape,P", SHAPES, ids=lambda x: "x".join(map(str, x)) if isinstance(x, tuple) else f"p{x}")
def test_constant_tables_leave_the_softmax(fps, shape, P, value):
    q, k, v, g = (normal(shape, i) for i in range(4))
    buckets = torch.tensor([0, 1, 1, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
    table = torch.full((2, shape[4]), value, dtype=torch.bfloat16, device="cuda")
    got = run(fps, q, k, v, g, table, buckets, P)
    want = reference(q, k, v, torch.zeros_like(table), buckets, P, 0, dout=g)
    off = 2.0 ** -20 * (abs(value) + 16)
    for name, x in zip(NAMES, got):
        val, tol = want[name]
        if name == "lse":
            val, tol = val + value, tol + 2.0 ** -22 * abs(value)
        else:
            tol = tol * (1 + off * (2.0 ** 13 if name == "dtable" else 2.0 ** 8))
        check(name, x, val, tol)


@pytest.mark.parametrize("value", [-65504.0, -1e9, -9e29, -65280.0, 65280.0])
@pytest.mark.parametrize("H,W", [(3, 4), (10, 14)])  # both kernels
def test_over_the_cache(fps, H, W, value):
    """Low entries mask there too; rows that see nothing else give 0. A constant table leaves the softmax."""
    shape, cap = (1, 2, H, W, 2, 64), 6
    cache = fps.frame_cache(1, cap, H, W, 2, 64, 1)
    fps.skiparse2d_cache_append(normal((1, cap) + shape[2:], 1, 3.0), normal((1, cap) + shape[2:], 2),
                                torch.zeros(1, dtype=torch.int32, device="cuda"), cache, 1, 0)
    q, start = normal(shape, 3, 3.0), torch.tensor([4], dtype=torch.int32, device="cuda")
    table = torch.full((2, 2), value, dtype=torch.bfloat16, device="cuda")
    table[0] = 0 if value <= -65504 else value
    even = torch.tensor([1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")  # bucket 1 at even distances, 0 at odd

    def call(t, m):
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:5], 9.0, device="cuda")
        fps.skiparse2d_attn_cached(q, cache, start, 1, 0, table=t, buckets=m, out=out, lse=lse)
        assert fps.get_device_status() == 0
        return out, lse

    out, lse = call(table, even)
    if value <= -65504:
        want = call(table, torch.where(even == 1, -1, even))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        out, lse = call(table, torch.ones_like(even))
        assert (out == 0).all() and (lse == -math.inf).all()
    else:
        plain, plain_lse = call(torch.zeros_like(table), even)
        off = 2.0 ** -20 * (abs(value) + 16)
        assert float((lse.double() - value - plain_lse).abs().max()) <= 1e-4 + 2.0 ** -22 * abs(value)
        # weights off by `off` relative, in f16 and out in bf16, each rounded in both calls
        most = cache.v.double().mul(cache.v_scale.double().repeat_interleave(64, 3)[:, :, :, :H * W, None]).abs().amax()
        assert float((out.double() - plain.double()).abs().max()) <= float(most) * (off + 2.0 ** -10 + 2.0 ** -7)
