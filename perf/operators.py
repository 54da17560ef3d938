"""Calls of the frame-aware class attention operators, to be timed and compared.

Four operators on video tokens (B, T, H, W, heads, d) in bf16, in both class rules:

  forward   class attention with a learned bias by frame distance (buckets; a bucket outside the
            table masks the pair), with the log-sum-exp that a backward pass needs
  train     the same and its backward pass: gradients of q, k, v and of the bias table
  append    new frames' keys and values, rearranged by class, into a cache held in e4m3 with a
            power-of-two scale for every 64 tokens of a frame's class and head
  cached    attention of the newest frames over that cache

Every case is a dict of plain values; `run` computes the plain form in 32 bits, or, where `own`
is true, calls the package."""

import math

import torch

own = False

BLOCK = 64        # tokens of one class and frame that share a scale
LOW_EXP = -110    # the smallest scale exponent


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest forward: four frames of a thumbnail, where the launch is what counts
        dict(name="forward_thumbnail", op="forward", B=1, T=4, H=8, W=8, heads=4, d=64, P=2, mode=0, mask="both", D=8, NB=8),
        # a batch of long clips of small odd frames, every class dense (P = 1), within a window
        dict(name="forward_window_odd", op="forward", B=2, T=33, H=7, W=13, heads=8, d=32, P=1, mode=0, mask="window", D=16, NB=12),
        # one layer of a 480p clip, frame-causal
        dict(name="forward_480p_causal", op="forward", B=1, T=21, H=30, W=52, heads=12, d=128, P=2, mode=1, mask="causal", D=32, NB=32),
        # training steps: an odd latent that pads on both axes; a middle one; a 480p clip
        dict(name="train_anyres", op="train", B=2, T=3, H=10, W=14, heads=4, d=64, P=2, mode=1, mask="both", D=8, NB=8),
        dict(name="train_p3_causal", op="train", B=1, T=9, H=27, W=40, heads=6, d=64, P=3, mode=1, mask="causal", D=16, NB=16),
        dict(name="train_480p", op="train", B=1, T=21, H=30, W=52, heads=12, d=128, P=2, mode=0, mask="both", D=32, NB=32),
        # one frame of a 720p stream; a whole 480p clip at once
        dict(name="append_720p_frame", op="append", B=1, T=1, H=45, W=80, heads=40, d=128, P=2, mode=1, cap=21, start=30),
        dict(name="append_480p_clip", op="append", B=2, T=21, H=30, W=52, heads=12, d=128, P=2, mode=0, cap=24, start=0),
        # one token per class and step over a long history
        dict(name="cached_token", op="cached", B=4, T=1, H=2, W=2, heads=12, d=128, P=2, mode=0, cap=8192, start=8000, mask="causal", D=128, NB=32),
        # small frames: a dozen tokens per class and step
        dict(name="cached_small_frames", op="cached", B=2, T=1, H=7, W=9, heads=8, d=64, P=2, mode=1, cap=400, start=333, mask="causal", D=64, NB=32),
        # a chunk of three 480p frames over a full ring of 24
        dict(name="cached_480p_chunk", op="cached", B=2, T=3, H=30, W=52, heads=12, d=128, P=2, mode=0, cap=24, start=40, mask="causal", D=32, NB=32),
        # one 720p frame over the 20 before it
        dict(name="cached_720p_frame", op="cached", B=1, T=1, H=45, W=80, heads=40, d=128, P=2, mode=1, cap=21, start=20, mask="both", D=32, NB=32),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    most = {c["op"]: 0.0 for c in listed()}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    op = rng.choice(sorted(most))
    while True:
        c = dict(op=op, B=_spread(rng, 1, 4), T=_spread(rng, 1, 3 if op == "cached" else 40), H=_spread(rng, 1, 45),
                 W=_spread(rng, 1, 80), heads=_spread(rng, 1, 40), d=rng.choice([32, 64, 128, 128]),
                 P=rng.choice([1, 2, 2, 3]), mode=rng.choice([0, 1]))
        if op in ("append", "cached"):
            c["cap"] = c["T"] + _spread(rng, 1, 2000 if op == "cached" else 20)
            c["start"] = rng.randrange(0, 2 * c["cap"])
        if op != "append":
            c["D"] = _spread(rng, 1, 128)
            c["mask"] = rng.choice(["both", "causal", "window"])
            c["NB"] = _spread(rng, 4, 40)
        # a row of dS sums to zero: where every row sees one bucket alone, the table's gradient is 0 and has no
        # size that an error could be compared with
        one_bucket = op == "train" and (c["T"] < 2 or c["mask"] == "window" and c["D"] < 4)
        if 0.0005 * most[op] <= _cost(c) <= most[op] and not one_bucket:
            return c


def _cost(c):
    """The plain form's size: padded scores (or padded tokens), whatever the mask."""
    P2 = c["P"] ** 2
    F = math.prod(-(-x // P2) * c["P"] for x in (c["H"], c["W"]))
    tokens = c["B"] * P2 * c["heads"] * c["T"] * F
    if c["op"] == "append":
        return float(tokens * c["d"])
    # scores, and the cache's own size where there is one (32-bit copies of it are made)
    keys = F * (c["T"] if c["op"] != "cached" else c["cap"])
    return float(tokens) * keys + (c["B"] * P2 * c["heads"] * keys * c["d"] * 4.0 if c["op"] == "cached" else 0.0)


# ----------------------------------------------------------------------------------- inputs

def _bucket_map(c):
    """int32 (2D+1): the bucket of each frame distance from -D to D, half of the buckets for single distances
    and half spaced by their logarithm, for each direction; -1 masks."""
    D, NB = c["D"], c["NB"]
    u = torch.arange(-D, D + 1)
    a = u.abs().double()
    per = NB if c["mask"] == "causal" else max(1, NB // 2)
    half = max(1, per // 2)
    far = half + torch.floor(torch.log2((a / half).clamp(min=1)) / math.log2(max(2.0, (D + 1) / half)) * (per - half)).long()
    g = torch.where(a < half, a.long(), far.clamp(max=per - 1)).clamp(max=per - 1)
    if c["mask"] == "causal":
        g = torch.where(u < 0, -1, g)
    else:
        g = torch.where(u < 0, g + per, g).clamp(max=NB - 1)
    if c["mask"] == "window":
        g = torch.where(u.abs() >= max(1, D // 2), -1, g)
    return g.to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shape = (c["B"], c["T"], c["H"], c["W"], c["heads"], c["d"])

    def normal(s, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(s, generator=gen, device="cuda") * std).to(dtype)

    s = {"case": c}
    if c["op"] != "append":
        s["q"] = normal(shape)
        s["table"] = normal((c["NB"], c["heads"]), 0.7)
        s["buckets"] = _bucket_map(c).cuda()
    if c["op"] != "cached":
        s["k"], s["v"] = normal(shape), normal(shape)
    if c["op"] == "train":
        s["dout"] = normal(shape)
    if c["op"] in ("append", "cached"):
        # sequences of a batch are not equally long
        s["start"] = torch.tensor([max(0, c["start"] - 3 * b) for b in range(c["B"])], dtype=torch.int32, device="cuda")
        F = math.prod(-(-x // c["P"] ** 2) * c["P"] for x in (c["H"], c["W"]))
        rows = (c["B"] * c["P"] ** 2, c["heads"], c["cap"], F, c["d"])
        blocks = rows[:3] + (-(-F // BLOCK),)
        for name in ("k", "v"):
            if c["op"] == "append":
                s[name + "_cache"] = torch.zeros(rows, dtype=torch.float8_e4m3fn, device="cuda")
                s[name + "_scale"] = torch.full(blocks, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
            else:  # codes near the top of their range, as a writer leaves them, with scales around 2^-7
                s[name + "_cache"] = normal(rows, 110.0, torch.float32).clamp(-448, 448).to(torch.float8_e4m3fn)
                s[name + "_scale"] = torch.randint(119, 122, blocks, generator=gen, device="cuda").to(torch.uint8).view(torch.float8_e8m0fnu)
    return s


# -------------------------------------------------------------------------------- plain form

def _positions(c, device):
    """For every class and place in it: the token's index in its frame, and whether it is a real one. A class's
    real tokens come first, in raster order."""
    P, P2 = c["P"], c["P"] ** 2
    R, S = (-(-x // P2) * P for x in (c["H"], c["W"]))
    cls = torch.arange(P, device=device)

    def axis(n):
        i = torch.arange(n, device=device)
        return cls[:, None] + P * i if c["mode"] == 0 else (i // P) * P2 + cls[:, None] * P + i % P

    h, w = axis(R), axis(S)
    real = (h < c["H"])[:, None, :, None] & (w < c["W"])[None, :, None, :]
    at = h[:, None, :, None] * c["W"] + w[None, :, None, :]
    at, real = at.reshape(P2, R * S), real.reshape(P2, R * S)
    order = torch.argsort(~real, dim=1, stable=True)
    at, real = at.gather(1, order), real.gather(1, order)
    return torch.where(real, at, 0), real


def _by_class(x, at):
    """(B,T,H,W,heads,d) -> (B, classes, heads, T, places, d)."""
    B, T, H, W, heads, d = x.shape
    return x.reshape(B, T, H * W, heads, d)[:, :, at].permute(0, 2, 4, 1, 3, 5)


def _to_tokens(y, c, real, at):
    """The inverse of _by_class, for real places."""
    B, P2, heads, T, F, d = y.shape
    out = torch.empty(B, T, c["H"] * c["W"], heads, d, dtype=y.dtype, device=y.device)
    out[:, :, at[real]] = y.permute(0, 3, 1, 4, 2, 5)[:, :, real]
    return out.reshape(B, T, c["H"], c["W"], heads, d)


def _frame_bias(s, tq, tk):
    """(.., heads, Tq, Tk) bias of each pair of frames, -inf where it is masked, and the buckets."""
    D = (s["buckets"].numel() - 1) // 2
    u = (tq[..., :, None] - tk[..., None, :]).clamp(-D, D)
    g = s["buckets"].long()[u + D]
    b = s["table"].float()[g.clamp(min=0)].movedim(-1, -3)
    return b.masked_fill((g < 0).unsqueeze(-3), -math.inf), g


def _softmax_rows(scores):
    """exp(scores - max) in place, its row sums and maxima; a row of -inf gives zeros."""
    top = scores.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    e = scores.sub_(top).exp_()
    return e, e.sum(-1, keepdim=True), top


def _plain_scores(q, k, bias, key_real):
    """Scores (B, classes, heads, Tq*F, Tk*F) of (.., T, F, d) queries and keys."""
    B, C, h, Tq, F, d = q.shape
    Tk = k.shape[3]
    scores = q.reshape(B, C, h, Tq * F, d) @ k.reshape(B, C, h, Tk * F, d).transpose(-1, -2)
    scores.mul_(1.0 / math.sqrt(d))
    view = scores.view(B, C, h, Tq, F, Tk, F)
    view.add_(bias[..., :, None, :, None])
    view.masked_fill_(~key_real[None, :, None, None, None, None, :], -math.inf)
    return scores


def _plain_attention(s):
    c = s["case"]
    at, real = _positions(c, s["q"].device)
    q, k, v = (_by_class(s[n], at).float() for n in "qkv")
    frames = torch.arange(c["T"], device=q.device)
    bias, g = _frame_bias(s, frames, frames)
    e, total, top = _softmax_rows(_plain_scores(q, k, bias, real))
    p = e.div_(total.clamp(min=1e-38))
    lse = (top + total.log()).view(q.shape[:5] + (1,))
    out = p @ v.flatten(3, 4)
    return c, at, real, q, k, v, g, p, out, lse


def _plain_forward(s):
    c, at, real, q, k, v, g, p, out, lse = _plain_attention(s)
    return {"out": _to_tokens(out.view_as(q), c, real, at).to(torch.bfloat16),
            "lse": _to_tokens(lse, c, real, at)[..., 0].contiguous()}


def _plain_train(s):
    c, at, real, q, k, v, g, p, out, lse = _plain_attention(s)
    dout = _by_class(s["dout"], at).float().masked_fill(~real[None, :, None, None, :, None], 0.0).flatten(3, 4)
    dv = p.transpose(-1, -2) @ dout
    ds = dout @ v.flatten(3, 4).transpose(-1, -2)
    ds.sub_((dout * out).sum(-1, keepdim=True)).mul_(p)
    scale = 1.0 / math.sqrt(c["d"])
    dq, dk = (ds @ k.flatten(3, 4)) * scale, (ds.transpose(-1, -2) @ q.flatten(3, 4)) * scale
    by_frames = ds.view(q.shape[:5] + (c["T"], q.shape[4])).sum((4, 6)).double().sum((0, 1))
    seen = g >= 0
    dtable = torch.zeros(c["NB"], c["heads"], dtype=torch.float64, device=q.device)
    dtable.index_add_(0, g[seen], by_frames[:, seen].t())
    grads = {n: _to_tokens(x.view_as(q), c, real, at).to(torch.bfloat16) for n, x in (("dq", dq), ("dk", dk), ("dv", dv))}
    return {"out": _to_tokens(out.view_as(q), c, real, at).to(torch.bfloat16), **grads, "dtable": dtable.to(torch.bfloat16)}


def _plain_append_one(s, name, at, real):
    c = s["case"]
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    x = _by_class(s[name], at).float().masked_fill(~real[None, :, None, None, :, None], 0.0)  # (B, C, heads, T, F, d)
    F, NB = x.shape[4], scale.shape[3]
    blocks = torch.nn.functional.pad(x, (0, 0, 0, NB * BLOCK - F)).unflatten(4, (NB, BLOCK))
    m, e = torch.frexp(blocks.abs().amax((5, 6)))
    e = torch.where(m <= 0.875, e - 9, e - 8).masked_fill(m == 0, LOW_EXP).clamp(min=LOW_EXP)  # (B, C, heads, T, NB)
    code = torch.ldexp(blocks, -e[..., None, None]).to(torch.float8_e4m3fn).flatten(4, 5)[:, :, :, :, :F]
    frames = s["start"].long()[:, None] + torch.arange(c["T"], device=x.device)  # (B, T)
    slot = frames % c["cap"]
    b = torch.arange(c["B"], device=x.device)[:, None]
    to = cache.view(torch.uint8).view(c["B"], -1, c["heads"], c["cap"], F, c["d"]).permute(0, 3, 1, 4, 2, 5)  # B, slot, C, F, heads, d
    new = code.view(torch.uint8).permute(0, 3, 1, 4, 2, 5)
    to[b, slot] = torch.where(real[None, None, :, :, None, None], new, to[b, slot])
    to = scale.view(torch.uint8).view(c["B"], -1, c["heads"], c["cap"], NB).permute(0, 3, 1, 4, 2)  # B, slot, C, NB, heads
    used = torch.nn.functional.pad(real, (0, NB * BLOCK - F)).unflatten(1, (NB, BLOCK)).any(-1)
    new = (e + 127).to(torch.uint8).permute(0, 3, 1, 4, 2)
    to[b, slot] = torch.where(used[None, None, :, :, None], new, to[b, slot])


def _plain_append(s):
    at, real = _positions(s["case"], s["k"].device)
    _plain_append_one(s, "k", at, real)
    _plain_append_one(s, "v", at, real)
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _read_cache(s, name):
    """(B, classes, heads, slots, places, d) in 32 bits."""
    c = s["case"]
    cache = s[name + "_cache"].float()
    e = s[name + "_scale"].view(torch.uint8).float() - 127.0
    scale = torch.exp2(e).repeat_interleave(BLOCK, dim=3)[:, :, :, : cache.shape[3]]
    return (cache * scale[..., None]).view(c["B"], -1, *cache.shape[1:])


def _plain_cached(s):
    c = s["case"]
    at, real = _positions(c, s["q"].device)
    q = _by_class(s["q"], at).float()
    k, v = _read_cache(s, "k"), _read_cache(s, "v")
    end = s["start"].long()[:, None] + c["T"]
    slot = torch.arange(c["cap"], device=q.device)[None]
    tk = slot + torch.div(end - 1 - slot, c["cap"], rounding_mode="floor") * c["cap"]  # the newest frame of each slot
    tq = s["start"].long()[:, None] + torch.arange(c["T"], device=q.device)
    bias, _ = _frame_bias(s, tq, tk)  # (B, heads, Tq, slots)
    bias = bias.masked_fill((tk < 0)[:, None, None, :], -math.inf)
    e, total, _ = _softmax_rows(_plain_scores(q, k, bias[:, None], real))
    out = (e @ v.flatten(3, 4)) / total.clamp(min=1e-38)
    return {"out": _to_tokens(out.view_as(q), c, real, at).to(torch.bfloat16)}


# --------------------------------------------------------------------------------- run, work

def run(state):
    c, s = state["case"], state
    if own:
        import fixed_pattern_sparse_b200 as fps
        if c["op"] == "forward":
            out, lse = fps.skiparse2d_attn_relbias_fwd(s["q"], s["k"], s["v"], s["table"], s["buckets"], c["P"], c["mode"])
            return {"out": out, "lse": lse}
        if c["op"] == "train":
            out_lo = torch.empty_like(s["q"])  # what rounding took from out
            out, lse = fps.skiparse2d_attn_relbias_fwd(s["q"], s["k"], s["v"], s["table"], s["buckets"], c["P"], c["mode"],
                                                       out_lo=out_lo)
            dq, dk, dv, dtable = fps.skiparse2d_attn_relbias_bwd(s["q"], s["k"], s["v"], out, s["dout"], lse, s["table"],
                                                                 s["buckets"], c["P"], c["mode"], out_lo=out_lo)
            return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dtable": dtable}
        cache = fps.FrameCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] == "append":
            fps.skiparse2d_cache_append(s["k"], s["v"], s["start"], cache, c["P"], c["mode"])
            return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        return {"out": fps.skiparse2d_attn_cached(s["q"], cache, s["start"], c["P"], c["mode"], table=s["table"],
                                                  buckets=s["buckets"])}
    return {"forward": _plain_forward, "train": _plain_train, "append": _plain_append, "cached": _plain_cached}[c["op"]](s)


def _class_sizes(c):
    """Real tokens of a frame in each class."""
    def axis(X):
        P = c["P"]
        return [sum(1 for x in range(X) if (x % P if c["mode"] == 0 else x // P % P) == i) for i in range(P)]
    return [a * b for a in axis(c["H"]) for b in axis(c["W"])]


def work(case):
    """Bytes and operations without which a pass cannot be done: the visible pairs of tokens, each input and
    output once, and of a cache the codes and scales of the frames that some query sees."""
    c = dict(case)
    sizes, tokens = _class_sizes(c), c["B"] * c["T"] * c["H"] * c["W"]
    row = c["heads"] * c["d"]
    blocks = sum(-(-n // BLOCK) for n in sizes) * c["heads"]
    if c["op"] == "append":
        return {"bytes": 2 * (tokens * row * 3 + c["B"] * c["T"] * blocks) + 4 * c["B"], "flops": 0}
    g = _bucket_map(c).tolist()
    D = c["D"]

    def seen(u):
        return g[max(-D, min(D, u)) + D] >= 0

    pairs = frames_read = 0
    for b in range(c["B"]):
        start = max(0, c["start"] - 3 * b) if c["op"] == "cached" else 0
        end = start + c["T"]
        first = max(0, end - c["cap"]) if c["op"] == "cached" else 0
        for tk in range(first, end):
            n = sum(seen(tq - tk) for tq in range(start, end))
            pairs += n
            frames_read += n > 0
    flops = 4 * c["d"] * c["heads"] * pairs * sum(n * n for n in sizes)
    small = c["NB"] * c["heads"] * 2 + (2 * D + 1) * 4
    if c["op"] == "forward":
        return {"bytes": 4 * tokens * row * 2 + tokens * c["heads"] * 4 + small, "flops": flops}
    if c["op"] == "train":
        return {"bytes": 8 * tokens * row * 2 + small + c["NB"] * c["heads"] * 2, "flops": 3.5 * flops}
    cache = 2 * frames_read * (sum(sizes) * row + blocks)
    return {"bytes": 2 * tokens * row * 2 + cache + small + 4 * c["B"], "flops": flops}


# ------------------------------------------------------------------------------------- exact

def _members(c, ci, cj, device):
    """In-frame indices of a class's tokens in raster order, from the rule for a token's class."""
    h, w = torch.arange(c["H"], device=device), torch.arange(c["W"], device=device)
    P = c["P"]
    h, w = ((h % P, w % P) if c["mode"] == 0 else (h // P % P, w // P % P))
    return torch.nonzero(((h == ci)[:, None] & (w == cj)[None, :]).flatten())[:, 0]


def _exact_attention(c, s):
    """out, lse and, with dout, the gradients, one class and head at a time, in 64 bits."""
    B, T, h, d = c["B"], c["T"], c["heads"], c["d"]
    dev, D = s["q"].device, c["D"]
    f64 = dict(dtype=torch.float64, device=dev)
    N = c["H"] * c["W"]
    q = s["q"].reshape(B, T, N, h, d)
    res = {"out": torch.zeros(B, T, N, h, d, **f64), "lse": torch.zeros(B, T, N, h, **f64)}
    train = c["op"] == "train"
    if train:
        res.update({n: torch.zeros(B, T, N, h, d, **f64) for n in ("dq", "dk", "dv")}, dtable=torch.zeros(c["NB"], h, **f64))
    for ci in range(c["P"]):
        for cj in range(c["P"]):
            at = _members(c, ci, cj, dev)
            n = at.numel()
            if n == 0:
                continue
            for b in range(B):
                if c["op"] == "cached":
                    start = int(s["start"][b])
                    times = list(range(max(0, start + T - c["cap"]), start + T))
                    slots = torch.tensor([t % c["cap"] for t in times], device=dev)
                    seq = (b * c["P"] + ci) * c["P"] + cj
                else:
                    start, times = 0, list(range(T))
                tk = torch.tensor(times, device=dev).repeat_interleave(n)
                tq = torch.arange(start, start + T, device=dev).repeat_interleave(n)
                g = s["buckets"].long()[(tq[:, None] - tk[None, :]).clamp(-D, D) + D]
                hidden = g < 0
                for i in range(h):
                    qi = q[b][:, at, i].reshape(-1, d).double()
                    if c["op"] == "cached":
                        ki, vi = ((s[m + "_cache"][seq, i][slots][:, :n].double()
                                   * s[m + "_scale"][seq, i][slots].double().repeat_interleave(BLOCK, 1)[:, :n, None]).reshape(-1, d)
                                  for m in "kv")
                    else:
                        ki, vi = (s[m].reshape(B, T, N, h, d)[b][:, at, i].reshape(-1, d).double() for m in "kv")
                    z = qi @ ki.t() / math.sqrt(d) + s["table"][:, i].double()[g.clamp(min=0)]
                    z[hidden] = -math.inf
                    l = torch.logsumexp(z, 1)
                    p = torch.exp(z - l.masked_fill(l == -math.inf, 0.0)[:, None])
                    o = p @ vi
                    res["out"][b, :, at, i] = o.view(T, n, d)
                    res["lse"][b, :, at, i] = l.view(T, n)
                    if train:
                        do = s["dout"].reshape(B, T, N, h, d)[b][:, at, i].reshape(-1, d).double()
                        dp = do @ vi.t()
                        dz = p * (dp - (p * dp).sum(1, keepdim=True))
                        res["dq"][b, :, at, i] = (dz @ ki / math.sqrt(d)).view(T, n, d)
                        res["dk"][b, :, at, i] = (dz.t() @ qi / math.sqrt(d)).view(T, n, d)
                        res["dv"][b, :, at, i] = (p.t() @ do).view(T, n, d)
                        res["dtable"][:, i] += torch.bincount(g.clamp(min=0).flatten(), weights=dz.flatten(), minlength=c["NB"])
    full = (B, T, c["H"], c["W"], h, d)
    res = {n: x if n == "dtable" else x.reshape(full[: x.dim() + 1]) for n, x in res.items()}
    keep = {"forward": ("out", "lse"), "train": ("out", "dq", "dk", "dv", "dtable"), "cached": ("out",)}[c["op"]]
    return {n: res[n] for n in keep}


def _exact_append(c, s):
    out = {}
    for m in "kv":
        cache, scale = s[m + "_cache"].double(), s[m + "_scale"].double()
        x = s[m].reshape(c["B"], c["T"], c["H"] * c["W"], c["heads"], c["d"])
        for b in range(c["B"]):
            for ci in range(c["P"]):
                for cj in range(c["P"]):
                    at = _members(c, ci, cj, x.device)
                    seq = (b * c["P"] + ci) * c["P"] + cj
                    for first in range(0, at.numel(), BLOCK):
                        y = x[b][:, at[first:first + BLOCK]].double()  # T, tokens, heads, d
                        top = y.abs().amax((1, 3))
                        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(min=LOW_EXP)
                        y = y / torch.exp2(e)[:, None, :, None]
                        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
                        code = torch.round(y / step) * step
                        for t in range(c["T"]):
                            slot = (int(s["start"][b]) + t) % c["cap"]
                            cache[seq, :, slot, first:first + y.shape[1]] = code[t].transpose(0, 1)
                            scale[seq, :, slot, first // BLOCK] = torch.exp2(e[t])
        out[m + "_cache"], out[m + "_scale"] = cache, scale
    return out


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return _exact_append(c, s) if c["op"] == "append" else _exact_attention(c, s)
