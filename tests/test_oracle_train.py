"""Pins of the float64 oracle of rotary positions, of block-sparse
attention's gradients and of single-token queries (oracle/train_ref.py):
complex multiplication, relative positions, central differences, torch's
float64 autograd, explicit loops."""

import math

import numpy as np
import pytest
import torch

from oracle import paro_ref as ref
from oracle import train_ref as tr
from test_oracle_attention import random_idx

GRIDS = [((2, 3, 4), 8), ((3, 2, 5), 7)]


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_is_a_complex_product(interleaved):
    rng = np.random.default_rng(3)
    d, pairs, theta = 16, (3, 2, 2), 100.0
    pos = tr.grid_positions((2, 3, 4))
    x = rng.standard_normal((24, d))
    y = tr.rope(x, tr.rope_angles(pos, d, pairs, theta), interleaved)
    axis = [0, 0, 0, 1, 1, 2, 2, None]
    within = [0, 1, 2, 0, 1, 0, 1, None]
    for n in range(24):
        for p in range(d // 2):
            i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + d // 2)
            t = 0.0 if axis[p] is None else pos[n, axis[p]] * theta ** (-within[p] / pairs[axis[p]])
            z = complex(x[n, i], x[n, j]) * complex(math.cos(t), math.sin(t))
            assert abs(z.real - y[n, i]) < 1e-14 and abs(z.imag - y[n, j]) < 1e-14


def test_rope_keeps_relative_positions_and_turns_back():
    rng = np.random.default_rng(4)
    d, pairs = 12, (2, 2, 2)
    q, k = rng.standard_normal((2, 1, d))

    def dot(pq, pk):
        a = tr.rope(q, tr.rope_angles([pq], d, pairs, 50.0))
        b = tr.rope(k, tr.rope_angles([pk], d, pairs, 50.0))
        return (a * b).sum()

    assert abs(dot((1, 2, 3), (4, 0, 5)) - dot((11, 7, 3), (14, 5, 5))) < 1e-12
    ang = tr.rope_angles(tr.grid_positions((1, 2, 3)), d, pairs, 50.0, first=(7.5, 0, 0), step=(1, 0.5, 1))
    x = rng.standard_normal((6, d))
    assert np.abs(tr.rope(tr.rope(x, ang), ang, inverse=True) - x).max() < 1e-14
    # the inverse is the transpose: <R x, y> = <x, R^-1 y>
    y = rng.standard_normal((6, d))
    assert abs((tr.rope(x, ang) * y).sum() - (x * tr.rope(y, ang, inverse=True)).sum()) < 1e-12


def problem(seed, grid, block, nh=3, d=4):
    rng = np.random.default_rng(seed)
    N = grid[0] * grid[1] * grid[2]
    nb = -(-N // block)
    q, k, v, do = (rng.standard_normal((1, nh, N, d)) for _ in range(4))
    idx, counts = random_idx(rng, nh, nb, max(1, nb - 1))
    counts[0, 0, 0] = 0  # a query block without keys
    return q, k, v, do, rng.standard_normal((1, nh, N)), [0, 3, 5], idx, counts


@pytest.mark.parametrize("grid,block", GRIDS)
def test_forward_is_the_oracles_attention(grid, block):
    q, k, v, _, _, perms, idx, counts = problem(5, grid, block)
    out, lse = tr.attention_lse(q, k, v, grid, perms, block, idx, counts)
    assert np.abs(out - ref.attention(q, k, v, grid, perms, block, idx, counts)).max() < 1e-13
    # rows without keys, and out as the explicit sum of exp(s - lse) v
    assert (lse[0, 0] == -np.inf).sum() == block
    assert (out[0, 0][lse[0, 0] == -np.inf] == 0).all()


@pytest.mark.parametrize("grid,block", GRIDS)
def test_gradients_are_the_differences(grid, block):
    q, k, v, do, dl, perms, idx, counts = problem(6, grid, block)

    def f(q, k, v):
        out, lse = tr.attention_lse(q, k, v, grid, perms, block, idx, counts)
        fin = np.isfinite(lse)
        return (out * do).sum() + (lse[fin] * dl[fin]).sum()

    grads = tr.attention_backward(q, k, v, do, grid, perms, block, idx, counts, dl)
    rng = np.random.default_rng(7)
    for which, g in enumerate(grads):
        x = [q, k, v]
        direction = rng.standard_normal(q.shape)
        eps = 1e-5
        up, down = ([a + s * eps * direction if i == which else a for i, a in enumerate(x)]
                    for s in (1, -1))
        # the error of a central difference: eps^2 f''' / 6 + 1e-16 |f| / eps
        assert abs((f(*up) - f(*down)) / (2 * eps) - (g * direction).sum()) < 1e-6
        at = tuple(rng.integers(0, n) for n in q.shape)
        up, down = ([a.copy() for a in x] for _ in range(2))
        up[which][at] += eps
        down[which][at] -= eps
        assert abs((f(*up) - f(*down)) / (2 * eps) - g[at]) < 1e-7


def test_gradients_are_torch_autograds():
    grid, block = (2, 3, 4), 8
    q, k, v, do, dl, perms, idx, counts = problem(8, grid, block)
    counts[...] = np.maximum(counts, 1)
    t = [torch.from_numpy(x).requires_grad_() for x in (q, k, v)]
    total = 0.0
    for b, h, allowed in tr._tiles(q, grid, perms, block, idx, counts):
        s = (t[0][b, h] @ t[1][b, h].T / 2.0).masked_fill(~torch.from_numpy(allowed), -math.inf)
        lse = torch.logsumexp(s, 1)
        total = total + (torch.exp(s - lse[:, None]) @ t[2][b, h] * torch.from_numpy(do[b, h])).sum()
        total = total + (lse * torch.from_numpy(dl[b, h])).sum()
    total.backward()
    for x, g in zip(t, tr.attention_backward(q, k, v, do, grid, perms, block, idx, counts, dl)):
        assert np.abs(x.grad.numpy() - g).max() < 1e-12


def test_bounds_hold_for_the_roundings_they_count():
    """The forward and backward formulas with P, dS, out and the results
    rounded to bf16 stay within the bounds, and the bounds are no looser
    than some hundred times what such a run shows."""
    grid, block = (2, 5, 7), 16
    q, k, v, do, dl, perms, idx, counts = problem(9, grid, block, d=8)
    bf = lambda x: torch.from_numpy(x).bfloat16().double().numpy()  # noqa: E731
    q, k, v, do = (bf(x) for x in (q, k, v, do))
    bounds = tr.training_bounds(q, k, v, do, grid, perms, block, idx, counts, dl)
    out, lse = tr.attention_lse(q, k, v, grid, perms, block, idx, counts)
    dq, dk, dv = tr.attention_backward(q, k, v, do, grid, perms, block, idx, counts, dl)
    scale = 1 / math.sqrt(8)
    for b, h, allowed in tr._tiles(q, grid, perms, block, idx, counts):
        p, _ = tr._softmax(q[b, h], k[b, h], allowed)
        o = bf(bf(p) @ v[b, h])
        ds = p * (do[b, h] @ v[b, h].T - ((do[b, h] * o).sum(1) - dl[b, h])[:, None])
        got = {"out": o, "dq": bf(bf(ds) @ k[b, h] * scale), "dk": bf(bf(ds).T @ q[b, h] * scale),
               "dv": bf(bf(p).T @ do[b, h])}
        for name, want in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
            err = np.abs(got[name] - want[b, h])
            assert (err <= bounds[name][b, h] + 1e-300).all(), name
            assert bounds[name][b, h].sum() < 100 * err.sum(), name


def test_query_attention_by_loops():
    rng = np.random.default_rng(10)
    B, hk, group, M, N, block, d, keep = 2, 2, 2, 3, 27, 8, 4, 2
    nb = -(-N // block)
    q = rng.standard_normal((B, hk * group, M, d))
    k, v = (rng.standard_normal((B, hk, nb * block, d)) for _ in range(2))
    pool = rng.standard_normal((B, hk, nb, d))
    pool[0, 0, 1] = pool[0, 0, 0]  # a tie: the lower index first
    lengths = [27, 9]
    out, idx, lse, _, _ = tr.query_attention(q, k, v, pool, N, block, keep, lengths)
    for b in range(B):
        for h in range(hk * group):
            for m in range(M):
                kh = h // group
                blocks = list(range(-(-lengths[b] // block)))
                score = [sum(q[b, h, m, t] * pool[b, kh, j, t] for t in range(d)) for j in blocks]
                kept = sorted(sorted(blocks, key=lambda j: (-score[j], j))[:keep])
                assert list(idx[b, h, m]) == kept + [-1] * (keep - len(kept))
                toks = [c for j in kept for c in range(j * block, (j + 1) * block) if c < lengths[b]]
                w = [math.exp(sum(q[b, h, m, t] * k[b, kh, c, t] for t in range(d)) / 2) for c in toks]
                assert abs(lse[b, h, m] - math.log(sum(w))) < 1e-12
                for t in range(d):
                    want = sum(x * v[b, kh, c, t] for x, c in zip(w, toks)) / sum(w)
                    assert abs(out[b, h, m, t] - want) < 1e-12
    out, idx, lse, _, _ = tr.query_attention(q, k, v, pool, N, block, keep, [0, 1])
    assert (out[0] == 0).all() and (idx[0] == -1).all() and (lse[0] == -np.inf).all()
    assert np.allclose(out[1], np.repeat(v[1, :, :1], group, 0)) and (idx[1, ..., 0] == 0).all()
