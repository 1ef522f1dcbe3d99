"""Float64 CPU oracle of rotary positions with three axes, of block-sparse
attention's forward pass with its log-sum-exp and its gradients, and of
single query tokens against a stored clip.

TEST INFRASTRUCTURE ONLY.  Only the tests may import this module.  It shares
no code with the CUDA library; it reuses this oracle's own reorder
(paro_ref.py).  Pins: tests/test_oracle_train.py.

The ``*_bounds`` functions give, element by element, how far a result with
the library's roundings may be from the exact one: U is the relative size of
a rounding to bf16 (half a step), T covers the fp32 arithmetic around it
(sums of at most some hundred terms and the exponential: 2^-24 times the
number of roundings in a chain, below 2^-15)."""

from __future__ import annotations

import math

import numpy as np

from . import paro_ref as ref

U = 2.0 ** -8
T = 2.0 ** -15


# ------------------------------------------------------- rotary positions --

def grid_positions(grid) -> np.ndarray:
    F, H, W = grid
    n = np.arange(F * H * W)
    return np.stack((n // (H * W), n // W % H, n % W), -1)


def rope_angles(pos, d, pairs, theta, first=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0)) -> np.ndarray:
    """[..., 3] coordinates -> [..., d/2] angles; pairs of no axis turn by 0."""
    pos = np.asarray(pos, dtype=np.float64)
    out = np.zeros(pos.shape[:-1] + (d // 2,))
    at = 0
    for a, m in enumerate(pairs):
        for i in range(m):
            out[..., at + i] = (first[a] + step[a] * pos[..., a]) * theta ** (-i / m)
        at += m
    return out


def rope(x, angles, interleaved=True, inverse=False) -> np.ndarray:
    """x [..., N, d] turned by angles [..., N, d/2]."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    c, s = np.cos(angles), np.sin(angles) * (-1.0 if inverse else 1.0)
    y = np.empty_like(x)
    first, second = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0::2], y[..., 1::2] = first, second
    else:
        y[..., :half], y[..., half:] = first, second
    return y


def rope_bounds(x, y, interleaved, bf16) -> np.ndarray:
    """Cosine, sine, two products and a sum, each rounded to fp32, then the
    result to bf16."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    size = np.empty_like(x)
    if interleaved:
        size[..., 0::2] = size[..., 1::2] = a + b
    else:
        size[..., :half] = size[..., half:] = a + b
    return 4 * 2.0 ** -24 * size + (U * np.abs(y) if bf16 else 0.0)


# ---------------------------------------------------------------- training --

def _tiles(q, grid, perms, block, idx, counts):
    """(b, h, key tokens of each token's row as a boolean matrix)."""
    B, nh, N, _ = q.shape
    nb = -(-N // block)
    for h in range(nh):
        order = ref.reorder_head(np.arange(N, dtype=np.float64)[:, None], grid, perms[h],
                                 block)[:N, 0].astype(int)
        of = np.empty(N, dtype=int)
        of[order] = np.arange(N) // block
        for b in range(B):
            keep = np.zeros((nb, nb), dtype=bool)
            for i in range(nb):
                n = idx.shape[-1] if counts is None else counts[b, h, i]
                keep[i, idx[b, h, i, :n]] = True
            yield b, h, keep[of][:, of]


def _softmax(q, k, allowed):
    s = q @ k.T / math.sqrt(q.shape[-1])
    s = np.where(allowed, s, -np.inf)
    m = s.max(1, keepdims=True)
    m0 = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - m0)
    z = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m0 + np.log(z))[:, 0]
    return e / np.where(z == 0, 1.0, z), lse


def attention_lse(q, k, v, grid, perms, block, idx, counts=None):
    """(out [B,h,N,d], lse [B,h,N]), natural token order."""
    out, lse = np.zeros_like(q), np.zeros(q.shape[:3])
    for b, h, allowed in _tiles(q, grid, perms, block, idx, counts):
        p, lse[b, h] = _softmax(q[b, h], k[b, h], allowed)
        out[b, h] = p @ v[b, h]
    return out, lse


def attention_backward(q, k, v, dout, grid, perms, block, idx, counts=None, dlse=None):
    """(dq, dk, dv) of the sum of out * dout + lse * dlse."""
    dq, dk, dv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    for b, h, allowed in _tiles(q, grid, perms, block, idx, counts):
        p, _ = _softmax(q[b, h], k[b, h], allowed)
        dp = dout[b, h] @ v[b, h].T
        dd = (p * dp).sum(1, keepdims=True)
        if dlse is not None:
            dd = dd - dlse[b, h][:, None]
        ds = p * (dp - dd) / math.sqrt(q.shape[-1])
        dq[b, h], dk[b, h], dv[b, h] = ds @ k[b, h], ds.T @ q[b, h], p.T @ dout[b, h]
    return dq, dk, dv


def training_bounds(q, k, v, dout, grid, perms, block, idx, counts=None, dlse=None):
    """Bounds of (out, lse, dq, dk, dv) with P and dS rounded to bf16 for
    their products, D taken from the rounded out, and every result rounded
    once (lse to fp32)."""
    names = ("out", "lse", "dq", "dk", "dv")
    res = {n: np.zeros_like(q) for n in names}
    res["lse"] = np.zeros(q.shape[:3])
    scale = 1.0 / math.sqrt(q.shape[-1])
    for b, h, allowed in _tiles(q, grid, perms, block, idx, counts):
        qh, kh, vh, do = q[b, h], k[b, h], v[b, h], dout[b, h]
        p, lse = _softmax(qh, kh, allowed)
        # a score's error: fp32 sums of exact products, relative to their
        # sizes; the weights follow it
        score = np.where(allowed, np.abs(qh) @ np.abs(kh).T * scale, 0.0)
        worst = score.max(1, keepdims=True) * 2.0 ** -17 + T
        rel = 2 * worst  # of a weight: its score's error and the sum's
        out = p @ vh
        bound_out = (U + rel) * (p @ np.abs(vh)) + U * np.abs(out)
        dp = do @ vh.T
        dd = (p * dp).sum(1, keepdims=True) - (0.0 if dlse is None else dlse[b, h][:, None])
        size = np.abs(do) @ np.abs(vh).T
        err_d = (np.abs(do) * (bound_out + T * np.abs(out))).sum(1, keepdims=True) + T * np.abs(dd)
        ds = p * (dp - dd)
        err = (U + rel + T) * np.abs(ds) + (1 + rel) * p * (err_d + T * size)
        res["out"][b, h] = bound_out
        res["lse"][b, h] = worst[:, 0] + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
        dq, dk, dv = ds @ kh * scale, ds.T @ qh * scale, p.T @ do
        res["dq"][b, h] = scale * (err @ np.abs(kh)) + (U + T) * np.abs(dq)
        res["dk"][b, h] = scale * (err.T @ np.abs(qh)) + (U + T) * np.abs(dk)
        res["dv"][b, h] = ((U + rel + T) * p).T @ np.abs(do) + (U + T) * np.abs(dv)
    return res


# ----------------------------------------------------------------- serving --

def query_attention(q, k_perm, v_perm, k_pool, N, block, k_keep, lengths=None):
    """q [B, hq, M, d]; k_perm, v_perm [B, hk, Np, d], k_pool [B, hk, NB, d] ->
    (out, idx, lse, bound of out for bf16, bound of lse)."""
    B, hq, M, d = q.shape
    group = hq // k_perm.shape[1]
    out, lse = np.zeros_like(q), np.full((B, hq, M), -np.inf)
    bound, bound_lse = np.zeros_like(q), np.zeros((B, hq, M))
    idx = np.full((B, hq, M, k_keep), -1, dtype=np.int32)
    for b in range(B):
        n = N if lengths is None else int(lengths[b])
        nb = -(-n // block)
        for h in range(hq):
            for m in range(M):
                row = q[b, h, m]
                with np.errstate(invalid="ignore"):
                    s = k_pool[b, h // group, :nb] @ row
                s = np.where(np.isnan(s), -np.inf, s)
                kept = np.sort(np.argsort(-s, kind="stable")[:k_keep])
                idx[b, h, m, :len(kept)] = kept
                if len(kept) == 0:
                    continue
                tok = np.concatenate([np.arange(j * block, min(n, (j + 1) * block)) for j in kept])
                kk, vv = k_perm[b, h // group, tok], v_perm[b, h // group, tok]
                p, ls = _softmax(row[None], kk, np.ones((1, len(tok)), dtype=bool))
                out[b, h, m], lse[b, h, m] = (p @ vv)[0], ls[0]
                worst = (np.abs(kk) @ np.abs(row)).max() / math.sqrt(d) * 2.0 ** -17 + T
                bound[b, h, m] = 2 * worst * (p @ np.abs(vv))[0] + U * np.abs(out[b, h, m])
                bound_lse[b, h, m] = worst + 2.0 ** -20 * abs(ls[0])
    return out, idx, lse, bound, bound_lse
