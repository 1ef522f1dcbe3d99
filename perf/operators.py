"""The measured operators of rotary positions and of training and serving
block-sparse attention, with their plain forms.

Kinds of case:

  rope          rotary positions with three axes (time, height, width) of the
                queries or keys of a video layer: forward, or (inverse) the
                gradient's rotation; positions from the F x H x W grid, or
                given token by token
  rope_reorder  the same rotation on the way into a head's token order, with
                the mean of every block: what block selection and the
                attention kernels read
  train         block-sparse attention over given kept blocks, forward with
                the log-sum-exp of every row, and backward: out, lse, dq, dk, dv
  query         single tokens against a cached clip: each query row keeps its
                k best blocks by the score q . block mean and attends to their
                tokens; query heads may share a key head

``own`` False: plain torch in 32 bits (selection scores and angles in 64).
``own`` True: the calls a user makes of the package.
"""

import math

import torch

own = False

#: Token orders of a head that the cases take: axes outermost -> innermost.
ORDERS = ((0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0))
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 10000.0


def listed():
    return [
        # one new token of a 480p-shaped layer (12 heads), before it meets the cache: the smallest call
        dict(name="rope_token", kind="rope", type="bf16", B=1, heads=12, F=1, H=1, W=1, d=128,
             inverse=False, interleaved=True, given=True, token_major=True),
        # queries of a 480p-shaped layer as the projection leaves them, [B, N, heads, d]
        dict(name="rope_480p", kind="rope", type="bf16", B=1, heads=12, F=21, H=30, W=52, d=128,
             inverse=False, interleaved=True, given=False, token_major=True),
        # the gradient's rotation in fp32 training, halves paired, tokens of clips of two lengths
        dict(name="rope_grad_f32", kind="rope", type="f32", B=2, heads=4, F=13, H=19, W=27, d=64,
             inverse=True, interleaved=False, given=True, token_major=False),
        # the tiny fp32 workload's queries on the way to selection
        dict(name="rope_reorder_tiny", kind="rope_reorder", type="f32", B=1, heads=2, F=4, H=8,
             W=8, d=64, block=64, interleaved=True, token_major=False),
        # keys of a 720p-shaped layer of 40 heads, straight from the projection
        dict(name="rope_reorder_720p", kind="rope_reorder", type="bf16", B=1, heads=40, F=21,
             H=45, W=80, d=128, block=128, interleaved=True, token_major=True),
        # one training step's attention of the small workload (d 64, block 64)
        dict(name="train_small", kind="train", B=1, heads=4, F=8, H=16, W=16, d=64, block=64,
             k=10, ragged=False),
        # the 480p-shaped layer's training step: the largest
        dict(name="train_480p", kind="train", B=1, heads=12, F=21, H=30, W=52, d=128, block=128,
             k=64, ragged=False),
        # two clips whose rows keep different numbers of blocks, some none, odd sizes
        dict(name="train_ragged", kind="train", B=2, heads=5, F=11, H=23, W=37, d=128, block=128,
             k=24, ragged=True),
        # a low-resolution fine-tuning step with narrow heads on wide blocks
        dict(name="train_narrow", kind="train", B=1, heads=8, F=9, H=21, W=33, d=64, block=128,
             k=13, ragged=True),
        # one token against a 480p clip's keys and values: single-token serving
        dict(name="query_token_480p", kind="query", type="bf16", B=1, heads=12, group=1, M=1, F=21,
             H=30, W=52, d=128, block=128, k=64, ragged=False),
        # sixteen tokens against a 720p clip, 40 heads
        dict(name="query_16_720p", kind="query", type="bf16", B=1, heads=40, group=1, M=16, F=21,
             H=45, W=80, d=128, block=128, k=89, ragged=False),
        # five clips of different lengths (one still empty), 3 query heads to a key head, fp32
        dict(name="query_grouped_f32", kind="query", type="f32", B=5, heads=4, group=3, M=2, F=11,
             H=15, W=17, d=64, block=64, k=9, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("rope", "rope_reorder", "train", "query"))
    d = rng.choice((64, 128))
    block = rng.choice((64, 128))
    c = dict(kind=kind, B=rng.choice((1, 1, 2, 3)), heads=_log_int(rng, 1, 12), F=_log_int(rng, 1, 21),
             H=_log_int(rng, 1, 33), W=_log_int(rng, 3, 52), d=d)
    n = c["F"] * c["H"] * c["W"]
    nb = -(-n // block)
    if kind == "rope":
        c.update(type=rng.choice(("bf16", "f32")), inverse=rng.random() < 0.5,
                 interleaved=rng.random() < 0.5, given=rng.random() < 0.5,
                 token_major=rng.random() < 0.5)
    elif kind == "rope_reorder":
        c.update(type=rng.choice(("bf16", "f32")), block=block, interleaved=rng.random() < 0.5,
                 token_major=rng.random() < 0.5)
    elif kind == "train":
        most = 190000 // (c["B"] * c["heads"] * nb)  # kept tiles: no more than the largest listed case
        c.update(block=block, k=_log_int(rng, 1, max(1, min(nb, most))), ragged=rng.random() < 0.5)
    else:
        c.update(type=rng.choice(("bf16", "f32")), block=block, group=rng.choice((1, 1, 2, 4)),
                 M=_log_int(rng, 1, 24))
        most = 25000 // (c["B"] * c["heads"] * c["group"] * c["M"])  # kept blocks of all rows
        c.update(k=_log_int(rng, 1, max(1, min(nb, most))), ragged=rng.random() < 0.5)
    return c


# ------------------------------------------------------------- inputs -----

def _token_order(case, dev):
    """[heads, N]: the token at each position of a head's order; head h takes order h % 6."""
    F, H, W = case["F"], case["H"], case["W"]
    n = torch.arange(F * H * W, device=dev).view(F, H, W)
    six = torch.stack([n.permute(o).reshape(-1) for o in ORDERS])
    return six[torch.arange(case["heads"], device=dev) % 6]


def _features(case, g, dev):
    """[N, d]: smooth features of the tokens' coordinates, so that near tokens are alike."""
    F, H, W, d = case["F"], case["H"], case["W"], case["d"]
    n = torch.arange(F * H * W, device=dev)
    at = torch.stack((n // (H * W), n // W % H, n % W), -1).float()
    freq = torch.randn(3, d // 2, generator=g, device=dev) * 0.15
    x = at @ freq
    return torch.cat((torch.sin(x), torch.cos(x)), -1) * 0.5


def _normal(shape, g, dev, dtype):
    return torch.randn(shape, generator=g, device=dev).to(dtype)


def rope_pairs(d):
    """Rotated pairs of each axis: d/2 in three parts, the rest to time."""
    third = d // 6
    return (d // 2 - 2 * third, third, third)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, heads, d = case["B"], case["heads"], case["d"]
    N = case["F"] * case["H"] * case["W"]
    s = {"case": case}
    if case["kind"] in ("rope", "rope_reorder"):
        dtype = TYPES[case["type"]]
        if case["token_major"]:
            s["x"] = _normal((B, N, heads, d), g, dev, dtype).transpose(1, 2)
        else:
            s["x"] = _normal((B, heads, N, d), g, dev, dtype)
        s["extent"] = (case["F"], case["H"], case["W"])
        s["positions"] = None
        if case.get("given"):
            s["extent"] = (64, 48, 80)
            s["positions"] = torch.stack([torch.randint(0, e, (B, N), generator=g, device=dev)
                                          for e in s["extent"]], -1).to(torch.int32)
    elif case["kind"] == "train":
        f = _features(case, g, dev)
        s["q"], s["k"] = ((0.7 * torch.randn(B, heads, N, d, generator=g, device=dev) + f).to(torch.bfloat16)
                          for _ in range(2))
        s["v"], s["dout"] = (_normal((B, heads, N, d), g, dev, torch.bfloat16) for _ in range(2))
        nb = -(-N // case["block"])
        rank = torch.rand(B, heads, nb, nb, generator=g, device=dev).argsort(-1)[..., :case["k"]]
        s["idx"] = rank.sort(-1).values.to(torch.int32)
        s["counts"] = None
        if case["ragged"]:
            s["counts"] = torch.randint(0, case["k"] + 1, (B, heads, nb), generator=g, device=dev).to(torch.int32)
            s["counts"][..., 0] = case["k"]
    else:
        dtype = TYPES[case["type"]]
        block = case["block"]
        nb = -(-N // block)
        f = _features(case, g, dev)
        order = _token_order(case, dev)
        pad = nb * block - N

        def cached(x):
            x = x[:, torch.arange(heads, device=dev)[:, None], order]
            return torch.nn.functional.pad(x, (0, 0, 0, pad)).contiguous()

        k = cached((0.7 * torch.randn(B, heads, N, d, generator=g, device=dev) + f).to(dtype))
        s["k"], s["v"] = k, cached(_normal((B, heads, N, d), g, dev, dtype))
        full = torch.full((nb,), block, device=dev)
        full[-1] = block - pad
        s["k_pool"] = k.float().view(B, heads, nb, block, d).sum(3) / full[:, None]
        s["q"] = _normal((B, heads * case["group"], case["M"], d), g, dev, dtype)
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.randint(1, N + 1, (B,), generator=g, device=dev).to(torch.int32)
            if B > 1:
                s["lengths"][B // 2] = 0
    if case["kind"] in ("rope_reorder", "train"):
        s["order"] = _token_order(case, dev)
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a user's program builds once: the problem's sizes and orders, and the rotation table."""
    from block_sparse_attention_34_b200 import paro

    c = s["case"]
    if c["kind"] in ("rope", "rope_reorder"):
        s["rope"] = paro.RopeTable(s["extent"], c["d"], pairs=rope_pairs(c["d"]), theta=THETA,
                                   interleaved=c["interleaved"])
    if c["kind"] != "rope":
        s["problem"] = paro.Problem(c["B"], c["heads"], (c["F"], c["H"], c["W"]), c["d"], c["block"],
                                    [h % 6 for h in range(c["heads"])])


# ---------------------------------------------------------- plain forms -----

def _angles(s, dtype=torch.float64):
    """[B or 1, 1, N, d/2]: the angle of each pair of each token."""
    c = s["case"]
    dev = s["x"].device
    at = s["positions"]
    if at is None:
        n = torch.arange(c["F"] * c["H"] * c["W"], device=dev)
        at = torch.stack((n // (c["H"] * c["W"]), n // c["W"] % c["H"], n % c["W"]), -1)[None]
    at = at.to(dtype)
    parts = []
    for a, m in enumerate(rope_pairs(c["d"])):
        freq = THETA ** (-torch.arange(m, device=dev, dtype=dtype) / m)
        parts.append(at[..., a, None] * freq)
    return torch.cat(parts, -1)[:, None]


def _rotate(s):
    c = s["case"]
    x = s["x"].float()
    angle = _angles(s)
    cos, sin = angle.cos().float(), angle.sin().float()
    if c.get("inverse"):
        sin = -sin
    half = c["d"] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if c["interleaved"] else (x[..., :half], x[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)


def _to_order(x, order, block):
    """[B, heads, N, d] -> [B, heads, NB, block, d] in each head's order, the tail zero."""
    heads, n = order.shape
    x = x[:, torch.arange(heads, device=x.device)[:, None], order]
    nb = -(-n // block)
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * block - n))
    return x.view(x.shape[0], heads, nb, block, -1)


def _from_order(x, order):
    heads, n = order.shape
    x = x.flatten(2, 3)[:, :, :n]
    out = torch.empty_like(x)
    out[:, torch.arange(heads, device=x.device)[:, None], order] = x
    return out


def _plain_rope_reorder(s):
    c = s["case"]
    n, block = s["x"].shape[2], c["block"]
    y = _to_order(_rotate(s), s["order"], block)
    rows = torch.full((y.shape[2],), block, device=y.device)
    rows[-1] = n - (len(rows) - 1) * block
    return y.flatten(2, 3).to(s["x"].dtype), y.sum(3) / rows[:, None]


def _plain_rows(q, k, v, do, idx, kept):
    """Attention and its gradients for whole heads: q, do, k, v [n, NB, block, d]
    (32 bits), idx [n, NB, k] block numbers, kept [n, NB, k, block] truth values."""
    n, nb, block, d = q.shape
    scale = 1.0 / math.sqrt(d)
    head = torch.arange(n, device=q.device)[:, None, None]
    kg, vg = k[head, idx].flatten(2, 3), v[head, idx].flatten(2, 3)
    x = (q @ kg.transpose(-1, -2)) * scale
    x = x.masked_fill(~kept.flatten(2, 3)[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    p = p / torch.where(total == 0, 1.0, total)
    out = p @ vg
    dp = do @ vg.transpose(-1, -2)
    ds = p * (dp - (do * out).sum(-1, keepdim=True)) * scale
    dq = ds @ kg
    to = (head * nb + idx).flatten()
    dk, dv = (torch.zeros(n * nb, block, d, device=q.device).index_add_(
        0, to, (m.transpose(-1, -2) @ y).view(-1, block, d)).view(n, nb, block, d)
        for m, y in ((ds, q), (p, do)))
    return out, lse, dq, dk, dv


def _kept(s, n_tokens, block):
    """[B, heads, NB, k, block]: whether a key at a place of a kept block counts."""
    idx, counts = s["idx"].long(), s["counts"]
    k = idx.shape[-1]
    dev = idx.device
    kept = (idx[..., None] * block + torch.arange(block, device=dev)) < n_tokens
    if counts is not None:
        kept &= (torch.arange(k, device=dev) < counts[..., None])[..., None]
    return kept


def _plain_train(s):
    c = s["case"]
    B, heads, block, d = c["B"], c["heads"], c["block"], c["d"]
    n = s["q"].shape[2]
    q, k, v, do = (_to_order(s[x], s["order"], block).flatten(0, 1) for x in ("q", "k", "v", "dout"))
    idx, kept = s["idx"].long().flatten(0, 1), _kept(s, n, block).flatten(0, 1)
    per_head = 32 * idx.shape[1] * idx.shape[2] * block * max(block, d)
    step = max(1, (40 << 30) // per_head)  # heads whose gathered tiles fit in memory at once
    parts = [_plain_rows(q[i:i + step].float(), k[i:i + step].float(), v[i:i + step].float(),
                         do[i:i + step].float(), idx[i:i + step], kept[i:i + step])
             for i in range(0, B * heads, step)]
    out, lse, dq, dk, dv = (torch.cat(x).unflatten(0, (B, heads)) for x in zip(*parts))
    lse = _from_order(lse[..., None], s["order"])[..., 0]
    return {"out": _from_order(out, s["order"]).bfloat16(), "lse": lse,
            "dq": _from_order(dq, s["order"]).bfloat16(), "dk": _from_order(dk, s["order"]).bfloat16(),
            "dv": _from_order(dv, s["order"]).bfloat16()}


def _plain_query(s):
    c = s["case"]
    B, heads, group, M, block, d, k = (c[x] for x in ("B", "heads", "group", "M", "block", "d", "k"))
    dev = s["q"].device
    n = c["F"] * c["H"] * c["W"]
    nb = s["k_pool"].shape[2]
    length = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), n, device=dev)
    blocks = (length + block - 1) // block
    q = s["q"].view(B, heads, group * M, d)
    score = q.double() @ s["k_pool"].double().transpose(-1, -2)
    open_ = torch.arange(nb, device=dev) < blocks[:, None, None, None]
    score = score.masked_fill(~open_, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    used = torch.arange(k, device=dev) < blocks[:, None, None, None]
    best = torch.where(used, best, nb).sort(-1).values
    idx = torch.where(best < nb, best, -1).to(torch.int32)
    at = best.clamp(max=nb - 1)
    b = torch.arange(B, device=dev)[:, None, None, None]
    h = torch.arange(heads, device=dev)[:, None, None]
    kg = s["k"].view(B, heads, nb, block, d)[b, h, at].flatten(3, 4).float()
    x = (kg @ q.float()[..., None])[..., 0] / math.sqrt(d)
    place = (best[..., None] * block + torch.arange(block, device=dev)).flatten(3)
    x = x.masked_fill((place >= length[:, None, None, None]) | (best.repeat_interleave(block, -1) >= nb), -math.inf)
    del kg
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    p = p / torch.where(total == 0, 1.0, total)
    vg = s["v"].view(B, heads, nb, block, d)[b, h, at].flatten(3, 4).float()
    out = (p[..., None, :] @ vg)[..., 0, :]
    shape = (B, heads * group, M)
    return out.view(*shape, d).to(s["q"].dtype), idx.view(*shape, k), lse.view(shape)


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["kind"] == "rope":
        return _rotate(s).to(s["x"].dtype)
    if c["kind"] == "rope_reorder":
        return _plain_rope_reorder(s)
    return _plain_train(s) if c["kind"] == "train" else _plain_query(s)


def _own(s):
    from block_sparse_attention_34_b200 import paro

    c = s["case"]
    if c["kind"] == "rope":
        return paro.rope3d(s["x"], s["rope"], positions=s["positions"], inverse=c["inverse"])
    pr = s["problem"]
    if c["kind"] == "rope_reorder":
        return paro.rope_reorder(s["x"], s["rope"], pr, with_pool=True)
    if c["kind"] == "query":
        return paro.block_sparse_query_attn(s["q"], s["k"], s["v"], s["k_pool"], pr, c["k"],
                                            lengths=s["lengths"])
    q, k, v = (paro.reorder(s[x], pr) for x in ("q", "k", "v"))
    out, lse = paro.block_sparse_attn_lse(q, k, v, pr, s["idx"], s["counts"])
    dq, dk, dv = paro.block_sparse_attn_backward(s["dout"], q, k, v, out, lse, pr, s["idx"], s["counts"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def work(case):
    n = case["F"] * case["H"] * case["W"]
    heads, d = case["B"] * case["heads"], case["d"]
    size = 4 if case.get("type") == "f32" else 2
    row = heads * n * d
    if case["kind"] == "rope":
        return {"bytes": 2 * row * size, "flops": 3 * row}
    block = case["block"]
    nb = -(-n // block)
    if case["kind"] == "rope_reorder":
        return {"bytes": row * size + heads * nb * d * (block * size + 4), "flops": 4 * row}
    if case["kind"] == "train":
        # mean kept blocks of a row: k, or half of it where rows keep 0 .. k;
        # two products of a tile forward, five backward
        tiles = heads * nb * case["k"] * (0.5 if case["ragged"] else 1.0)
        return {"bytes": 8 * row * 2 + heads * n * 4 + heads * nb * case["k"] * 4,
                "flops": 14 * tiles * block * block * d}
    rows = heads * case["group"] * case["M"]
    share = 0.5 if case["ragged"] else 1.0
    k = min(case["k"], max(1, round(nb * share)))
    blocks = min(rows * k, heads * nb * share)  # a block that several rows keep is read once
    return {"bytes": 2 * blocks * block * d * size + heads * nb * share * d * 4 + rows * (2 * d * size + 4 * k + 4),
            "flops": rows * (2 * nb * share * d + 4 * k * block * d)}


# ------------------------------------------------- the definition, 64 bits --

def _exact_rope(s):
    c = s["case"]
    x = s["x"].double()
    half = c["d"] // 2
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if c["interleaved"] else torch.complex(x[..., :half], x[..., half:])
    turn = _angles(s) * (-1.0 if c.get("inverse") else 1.0)
    z = z * torch.polar(torch.ones_like(turn), turn)
    if c["interleaved"]:
        return torch.view_as_real(z).flatten(-2)
    return torch.cat((z.real, z.imag), -1)


def _exact_train(s):
    """Dense attention of each head under its mask of token pairs, differentiated by torch."""
    c = s["case"]
    B, heads, block, d = c["B"], c["heads"], c["block"], c["d"]
    n = s["q"].shape[2]
    nb = -(-n // block)
    res = {x: torch.zeros(B, heads, n, d, dtype=torch.float64, device=s["q"].device)
           for x in ("out", "dq", "dk", "dv")}
    res["lse"] = torch.zeros(B, heads, n, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        for h in range(heads):
            of = torch.empty(n, dtype=torch.long, device=s["q"].device)  # a token's block
            of[s["order"][h]] = torch.arange(n, device=of.device) // block
            pick = torch.zeros(nb, nb + 1, dtype=torch.bool, device=of.device)
            rows = s["idx"][b, h].long()
            if s["counts"] is not None:
                rows = torch.where(torch.arange(rows.shape[1], device=of.device) < s["counts"][b, h][:, None], rows, nb)
            pick.scatter_(1, rows, True)
            allowed = pick[of][:, of]
            q, k, v = (s[x][b, h].double().requires_grad_() for x in ("q", "k", "v"))
            x = (q @ k.T / math.sqrt(d)).masked_fill(~allowed, -math.inf)
            some = allowed.any(1)
            lse = torch.logsumexp(x, 1)
            out = torch.exp(x - torch.where(some, lse, torch.zeros_like(lse))[:, None]) @ v
            dq, dk, dv = torch.autograd.grad(out, (q, k, v), s["dout"][b, h].double())
            res["out"][b, h], res["lse"][b, h] = out.detach(), lse.detach()
            res["dq"][b, h], res["dk"][b, h], res["dv"][b, h] = torch.where(some[:, None], dq, 0.0), dk, dv
    return res


def _exact_query(s):
    """Each row's softmax over every token of the cache, with those outside its kept blocks left out."""
    c = s["case"]
    B, heads, group, M, block, d, k = (c[x] for x in ("B", "heads", "group", "M", "block", "d", "k"))
    dev = s["q"].device
    outs, ids, lses = [], [], []
    for b in range(B):
        n = int(s["lengths"][b]) if s["lengths"] is not None else c["F"] * c["H"] * c["W"]
        nb = -(-n // block)
        for h in range(heads * group):
            q, kh = s["q"][b, h].double(), h // group
            mean = s["k_pool"][b, kh, :nb].double()
            score = (q[:, None] * mean[None]).sum(-1)
            # a block's rank: the blocks before it, by higher score or equal score and lower number
            number = torch.arange(nb, device=dev)
            ahead = (score[:, None, :] > score[:, :, None]) | (
                (score[:, None, :] == score[:, :, None]) & (number[None, :] < number[:, None])[None])
            keep = ahead.sum(-1) < k
            x = q @ s["k"][b, kh, :n].double().T / math.sqrt(d)
            x = x.masked_fill(~keep.repeat_interleave(block, 1)[:, :n], -math.inf)
            lse = torch.logsumexp(x, 1) if n else torch.full((M,), -math.inf, dtype=torch.float64, device=dev)
            outs.append(torch.exp(x - lse[:, None]) @ s["v"][b, kh, :n].double() if n
                        else torch.zeros(M, d, dtype=torch.float64, device=dev))
            lses.append(lse)
            row = torch.full((M, k), -1, dtype=torch.int32, device=dev)
            kept = min(k, nb)
            if kept:
                row[:, :kept] = keep.nonzero()[:, 1].view(M, kept).int()
            ids.append(row)
    shape = (B, heads * group, M)
    return (torch.stack(outs).view(*shape, d), torch.stack(ids).view(*shape, k), torch.stack(lses).view(shape))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(s)
    if case["kind"] == "rope_reorder":
        y = _exact_rope(s)
        block, n = case["block"], y.shape[2]
        nb = -(-n // block)
        perm = torch.zeros(case["B"], case["heads"], nb * block, case["d"], dtype=torch.float64, device=y.device)
        for h in range(case["heads"]):
            perm[:, h, :n] = y[:, h].index_select(1, s["order"][h])
        mean = torch.stack([perm[:, :, i * block:min(n, (i + 1) * block)].mean(2) for i in range(nb)], 2)
        return perm, mean
    return _exact_train(s) if case["kind"] == "train" else _exact_query(s)
