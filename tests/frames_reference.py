"""Plain fp64 statements of the frame-aware operators (test infrastructure), over all tokens at
once with explicit masks: the class of a token from its coordinates, no rearranged layout."""

from __future__ import annotations

import math

import torch

HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative
BLOCK = 64


def token_classes(H, W, P, mode, dims):
    """Class of every token of a frame, (H*W)."""
    if dims == 1:
        x = torch.arange(H * W)
        return x % (P * P) if mode == 0 else (x // (P * P)) % (P * P)
    h, w = torch.arange(H)[:, None], torch.arange(W)[None, :]
    ci, cj = (h % P, w % P) if mode == 0 else ((h // P) % P, (w // P) % P)
    return (ci * P + cj).reshape(-1)


def members(H, W, P, mode, dims):
    """In-frame token indices of each class, in raster order (the order of its places)."""
    cls = token_classes(H, W, P, mode, dims)
    return [torch.nonzero(cls == c)[:, 0] for c in range(P * P)]


def pair_bias(tq, tk, table, buckets):
    """(heads, Nq, Nk) fp64 bias by frame distance, -inf where masked; and the buckets."""
    D = (buckets.numel() - 1) // 2
    g = buckets.long()[(tq[:, None] - tk[None, :]).clamp(-D, D) + D]
    t = table.double()
    t = torch.where(t < -1e30, torch.full_like(t, -math.inf), t)
    bad = (g < 0) | (g >= table.shape[0])
    b = t[g.clamp(0, table.shape[0] - 1)].permute(2, 0, 1)
    return b.masked_fill(bad, -math.inf), torch.where(bad, -1, g)


def attend(q, k, v, bias, same):
    """q (Nq,h,d), k, v (Nk,h,d) fp64, bias (h,Nq,Nk), same (Nq,Nk): out, lse, P."""
    s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(q.shape[-1]) + bias
    s = s.masked_fill(~same, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[..., None])
    return torch.einsum("hqk,khd->qhd", p, v), lse.t(), p


def frames_of(T, n, device, first=0):
    return torch.arange(first, first + T, device=device).repeat_interleave(n)


def reference(q, k, v, table, buckets, P, mode, dims=2, dout=None, exact_d=True):
    """out, lse, (dq, dk, dv, dtable) in fp64 with the bound on each one's error, as a dict
    name -> (value, tolerance). The bounds count roundings: P and dS enter their products as bf16
    (half a step each), results are rounded to bf16 once; 2^-13 covers the fp32 arithmetic between
    (scores, exponentials, differences). For dq, D = dout . out is taken from the forward's out, whose
    error is that of P in P V, (e + 2^-13) P|V|, and its own rounding, e |out|, or e^2 of it where
    the residual is passed (rounded once itself, hence 2 e^2): |dout| times that is D's error. For
    dk and dtable D is corrected by the fp32 sum of its row of dS."""
    B, T, H, W, h, d = q.shape
    dev, n = q.device, H * W
    cls = token_classes(H, W, P, mode, dims).to(dev).repeat(T)
    same = cls[:, None] == cls[None, :]
    t = frames_of(T, n, dev)
    bias, g = pair_bias(t, t, table, buckets)
    names = ("out", "lse") + (("dq", "dk", "dv") if dout is not None else ())
    got = {m: [] for m in names}
    tol = {m: [] for m in names}
    dtable = torch.zeros(table.shape, dtype=torch.float64, device=dev)
    dtol = torch.zeros_like(dtable)
    e, fine, sc = HALF_BF16, 2.0 ** -13, 1 / math.sqrt(d)
    for b in range(B):
        qb, kb, vb = (x[b].reshape(T * n, h, d).double() for x in (q, k, v))
        o, l, p = attend(qb, kb, vb, bias, same)
        got["out"].append(o)
        tol["out"].append((e + fine) * torch.einsum("hqk,khd->qhd", p, vb.abs()) + e * o.abs())
        got["lse"].append(l)
        tol["lse"].append(torch.full_like(l, 1e-4))
        if dout is None:
            continue
        do = dout[b].reshape(T * n, h, d).double()
        dp = torch.einsum("qhd,khd->hqk", do, vb)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        o_err = (e + fine) * torch.einsum("hqk,khd->qhd", p, vb.abs()) + (e * e * 2 if exact_d else e) * o.abs()
        e_d = torch.einsum("qhd,qhd->hq", do.abs(), o_err)[..., None]
        mean = (p * dp.abs()).sum(-1, keepdim=True)
        e_ds = fine * p * (dp.abs() + mean)
        rows = e_ds + e * ds.abs()
        rows_q = rows + p * e_d
        for m, val, bound in (("dq", torch.einsum("hqk,khd->qhd", ds, kb) * sc, torch.einsum("hqk,khd->qhd", rows_q, kb.abs()) * sc),
                              ("dk", torch.einsum("hqk,qhd->khd", ds, qb) * sc, torch.einsum("hqk,qhd->khd", rows, qb.abs()) * sc),
                              ("dv", torch.einsum("hqk,qhd->khd", p, do), torch.einsum("hqk,qhd->khd", (e + fine) * p, do.abs()))):
            got[m].append(val)
            tol[m].append(bound + e * val.abs())
        for i in range(table.shape[0]):
            at = (g == i) & same
            dtable[i] += (ds * at).sum((1, 2))
            dtol[i] += (e_ds * at).sum((1, 2))
    full = (B, T, H, W, h, d)
    res = {m: (torch.stack(got[m]).reshape(full if m != "lse" else full[:5]),
               torch.stack(tol[m]).reshape(full if m != "lse" else full[:5]) + 1e-6) for m in names}
    if dout is not None:
        res["dtable"] = (dtable, dtol + e * dtable.abs() + 1e-6)
    return res


def check(name, got, want, tol):
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{name}: finite in other places"
    assert torch.equal(got[~fin], want[~fin]), f"{name}: other infinities"
    over = ((got - want).abs() - tol)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{name}: {float(over.max()):.3e} beyond its tolerance"


def quantise(x):
    """(blocks.., tokens, d) fp64 values -> codes' values, scale exponent, by definition."""
    # by frexp: a logarithm of an exact power of two may be off by its last bit
    m, ex = torch.frexp(x.abs().amax((-1, -2)) / 448.0)
    e = torch.where(m > 0.5, ex, ex - 1).masked_fill(m == 0, -110).clamp(min=-110).double()
    y = x / torch.exp2(e)[..., None, None]
    _, ex = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(y), ex - 4)
    return torch.round(y / step) * step, e


def cache_values(cache, name, seq, head, slot, n):
    """fp64 values of the first n places of one slot."""
    codes = getattr(cache, name)[seq, head, slot, :n].double()
    scale = getattr(cache, name + "_scale")[seq, head, slot].double().repeat_interleave(BLOCK)[:n]
    return codes * scale[:, None]


def cached_reference(q, cache, start, P, mode, table=None, buckets=None, dims=2):
    """out and lse over the cache's own (dequantised) values, with tolerances as in reference();
    rows of skipped sequences are NaN in both."""
    B, T, H, W, h, d = q.shape
    dev = q.device
    out = torch.full((B, T, H * W, h, d), math.nan, dtype=torch.float64, device=dev)
    tol, lse = torch.zeros_like(out), out[..., 0].clone()
    mem = members(H, W, P, mode, dims)
    for b in range(B):
        s0 = int(start[b])
        if s0 < 0:
            continue
        times = list(range(max(0, s0 + T - cache.capacity), s0 + T))
        for c, at in enumerate(mem):
            n = at.numel()
            if n == 0:
                continue
            tq, tk = frames_of(T, n, dev, s0), torch.tensor(times, device=dev).repeat_interleave(n)
            ki, vi = (torch.stack([torch.cat([cache_values(cache, m, b * P * P + c, i, t % cache.capacity, n) for t in times])
                                   for i in range(h)], 1) for m in ("k", "v"))
            bias = torch.zeros(h, tq.numel(), tk.numel(), dtype=torch.float64, device=dev)
            if table is not None:
                bias, _ = pair_bias(tq, tk, table, buckets)
            qi = q[b].reshape(T, H * W, h, d)[:, at.to(dev)].reshape(-1, h, d).double()
            o, l, p = attend(qi, ki, vi, bias, torch.ones(tq.numel(), tk.numel(), dtype=torch.bool, device=dev))
            w = (HALF_BF16 + 2.0 ** -13) * torch.einsum("hqk,khd->qhd", p, vi.abs()) + HALF_BF16 * o.abs() + 1e-6
            out[b, :, at] = o.reshape(T, n, h, d)
            tol[b, :, at] = w.reshape(T, n, h, d)
            lse[b, :, at] = l.reshape(T, n, h)
    return out.reshape(q.shape), tol.reshape(q.shape), lse.reshape(q.shape[:5])
