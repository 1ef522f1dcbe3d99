"""GPU parity of single query tokens against a stored clip (pa_query_attn)
against the float64 oracle (oracle/train_ref.py): kept blocks equal, out and
lse within the bounds of the roundings; one row to several clusters of them,
shared key heads, lengths from none to all, garbage behind the end, ties,
scores and values that are not finite, very many blocks."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from block_sparse_attention_34_b200 import paro
from oracle import train_ref as tr

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


class Clip:
    def __init__(self, B, heads, group, M, d, block, grid, dtype=BF, seed=0):
        self.pr = pr = paro.Problem(B, heads, grid, d, block, [h % 6 for h in range(heads)])
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        k, v = (torch.randn(pr.natural, generator=g, device="cuda").to(dtype) for _ in range(2))
        self.k, self.pool = paro.reorder(k, pr, with_pool=True)
        self.v = paro.reorder(v, pr)
        self.q = torch.randn((B, heads * group, M, d), generator=g, device="cuda").to(dtype)

    def run(self, keep, lengths=None, **kw):
        B, hq, M, d = self.q.shape
        out = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda")
        idx = torch.full((B, hq, M, keep), -9, dtype=torch.int32, device="cuda")
        lse = torch.full((B, hq, M), float("nan"), device="cuda")
        ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        return paro.block_sparse_query_attn(self.q, self.k, self.v, self.pool, self.pr, keep, lengths=ln,
                                            out=out, idx=idx, lse=lse, **kw)

    def check(self, got, keep, lengths=None):
        out, idx, lse, bound, bound_lse = tr.query_attention(
            f64(self.q), f64(self.k), f64(self.v), f64(self.pool), self.pr.N, self.pr.block, keep, lengths)
        assert (got[1].cpu().numpy() == idx).all()
        if self.q.dtype == F32:  # no rounding to bf16: the result's to fp32 instead
            bound = bound - tr.U * np.abs(out) + 2.0 ** -24 * np.abs(out)
        assert (np.abs(f64(got[0]) - out) <= bound).all()
        fin = np.isfinite(lse)
        assert (f64(got[2])[~fin] == lse[~fin]).all()
        assert (np.abs(f64(got[2])[fin] - lse[fin]) <= bound_lse[fin]).all()


# rows of a key head: 1, 2, 7, 8 (one packed tile), 9, 16 (one wide tile), 17,
# 40 (several); 1 to 4 query heads a key head
SHAPES = [
    (1, 12, 1, 1, 128, 128, (5, 9, 17), 3),
    (1, 3, 1, 1, 64, 64, (4, 7, 9), 1),
    (2, 40, 2, 1, 128, 64, (3, 11, 13), 4),
    (1, 150, 1, 7, 64, 128, (3, 9, 16), 2),
    (1, 10, 2, 4, 128, 128, (6, 9, 15), 4),
    (3, 5, 1, 9, 64, 64, (4, 9, 11), 5),
    (1, 20, 4, 4, 128, 128, (6, 11, 13), 3),
    (1, 12, 1, 17, 128, 64, (3, 10, 16), 6),
    (1, 13, 2, 20, 64, 128, (5, 11, 13), 6),
    (1, 1, 1, 1, 128, 128, (1, 1, 1), 1),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,heads,group,M,d,block,grid,keep", SHAPES)
def test_against_the_oracle(B, heads, group, M, d, block, grid, keep, dtype):
    c = Clip(B, heads, group, M, d, block, grid, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.run(keep, status=status)
    assert status.item() == 0
    c.check(got, keep)
    for a, b in zip(c.run(keep), got):  # the same bits again
        assert torch.equal(a, b)
    if c.pr.NB > 1:
        c.check(c.run(c.pr.NB), c.pr.NB)  # every block


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("group,M", [(1, 1), (2, 3), (3, 5)])
def test_lengths_and_what_lies_behind_them(dtype, group, M):
    c = Clip(6, 2, group, M, 64, 64, (4, 9, 11), dtype)
    N = c.pr.N
    lengths = [0, 1, 64, 65, N - 1, N]
    want = c.run(3, lengths)
    c.check(want, 3, lengths)
    for b, n in enumerate(lengths):  # behind the end the cache may hold anything
        c.k[b, :, n:] = float("nan")
        c.v[b, :, n:] = float("inf")
        c.pool[b, :, -(-n // 64):] = float("nan")
    for a, b in zip(c.run(3, lengths), want):
        assert torch.equal(a, b)
    # a length out of range: reported, its rows left as they were
    for bad in (-1, N + 1):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, idx, lse = c.run(3, [0, bad, 64, 65, N - 1, N], status=status)
        assert status.item() == paro.PA_ERR_DEVICE_CHECK
        assert out[1].isnan().all() and (idx[1] == -9).all() and lse[1].isnan().all()
        assert torch.equal(out[2:], want[0][2:])


def test_ties_go_to_the_lower_block():
    c = Clip(1, 2, 1, 3, 64, 64, (5, 13, 16), BF)
    c.q[0, 0, 0] = 0  # every block ties
    c.pool[0, 1, 4:9] = c.pool[0, 1, 4:5]  # five equal means
    c.pool[0, 1, 4:9] *= 3
    c.q[0, 1, 1] = c.pool[0, 1, 4].to(BF)  # ... that are the best of this row
    for keep in (1, 2, 4, 7):
        c.check(c.run(keep), keep)
    big = Clip(1, 1, 1, 2, 64, 64, (4, 40, 80), BF, seed=3)  # 200 blocks in one bin
    big.q.zero_()
    for keep in (1, 33, 199):
        got = big.run(keep)
        assert (got[1].cpu() == torch.arange(keep)).all()


def test_near_ties_are_decided_beyond_32_bits():
    """Scores that differ by less than a 32-bit sum can tell."""
    c = Clip(1, 1, 1, 1, 128, 64, (1, 8, 40), BF)
    q = torch.full((128,), 1.0, device="cuda")
    q[0] = 4096.0
    c.q[0, 0, 0] = q.to(BF)
    c.pool.zero_()
    c.pool[0, 0, :, 0] = 4096.0       # 2^24 in every score
    for j, x in enumerate((0.5, 0.25, 0.75, 0.0, 0.625)):
        c.pool[0, 0, j, 1] = x         # below half a step of 2^24
    for keep, want in ((1, [2]), (2, [2, 4]), (3, [0, 2, 4]), (4, [0, 1, 2, 4])):
        assert c.run(keep)[1].flatten().tolist() == want


def test_scores_that_are_not_finite():
    c = Clip(1, 1, 1, 2, 64, 64, (2, 8, 32), BF)
    c.pool[0, 0, 2] = float("nan")  # reads as -inf: last, by index
    c.pool[0, 0, 5] = float("inf")
    c.q[0, 0] = c.q[0, 0].abs()     # +inf for both rows
    for keep in (1, 3, 7):
        idx = c.run(keep)[1][0, 0]
        assert (idx == 5).any(-1).all() and not (idx == 2).any()
    c.pool.fill_(-float("inf"))
    assert (c.run(3)[1].cpu() == torch.arange(3)).all()


@pytest.mark.parametrize("M", [2, 8, 11, 16])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_other_rows_blocks_may_hold_anything(M, value):
    """Rows that share a cluster read the union of their blocks: a value that
    is not finite reaches the rows that keep its block and no other."""
    c = Clip(1, 12, 1, M, 64, 64, (3, 16, 20), BF)
    want = c.run(3)
    j = int(want[1][0, 0, 0, 1])  # kept by row 0 at least
    c.v[0, :, j * 64 + 5, 7] = value
    c.k[0, :, j * 64 + 9] = float("nan") if value != value else c.k[0, :, j * 64 + 9]
    out, idx, lse = c.run(3)
    assert torch.equal(idx, want[1])  # the means are as they were
    hit = (idx == j).any(-1)
    assert hit.any() and (~hit).any()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[2][~hit])
    assert not out[hit][:, 7].isfinite().any()


@pytest.mark.parametrize("dtype,M", [(BF, 1), (BF, 12), (F32, 1)])
def test_very_many_blocks(dtype, M):
    """More blocks than the deep rings leave room for, up to the limit."""
    pr = paro.Problem(1, 1, (1, 1, 14528 * 64), 64, 64, [0])
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (torch.randn(pr.permuted, generator=g, device="cuda").to(dtype) for _ in range(2))
    pool = k.view(1, 1, pr.NB, 64, 64).float().mean(3)
    q = torch.randn((1, 1, M, 64), generator=g, device="cuda").to(dtype)
    out, idx, lse = paro.block_sparse_query_attn(q, k, v, pool, pr, 100)
    score = q.double() @ pool.double().transpose(-1, -2)
    want = score.sort(dim=-1, descending=True, stable=True).indices[..., :100].sort(-1).values
    assert torch.equal(idx.long(), want)
    for m in range(M):
        toks = (want[0, 0, m][:, None] * 64 + torch.arange(64, device="cuda")).flatten()
        s = k[0, 0, toks].double() @ q[0, 0, m].double() / 8
        p = torch.softmax(s, 0)
        o = p @ v[0, 0, toks].double()
        assert (out[0, 0, m].double() - o).norm() <= (tr.U if dtype == BF else 1e-5) * o.norm() + 1e-6
        assert abs(float(lse[0, 0, m]) - float(torch.logsumexp(s, 0))) < 1e-4


def test_serving_matches_the_layer():
    """A clip stored by rope_reorder, a token rotated at its place: the same
    output as that token's row of block-sparse attention over its blocks."""
    grid, d, heads = (5, 12, 16), 128, 3
    pr = paro.Problem(1, heads, grid, d, 128, [0, 3, 9])
    table = paro.RopeTable(grid, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    q, k, v = (torch.randn(pr.natural, generator=g, device="cuda").to(BF) for _ in range(3))
    kp, pool = paro.rope_reorder(k, table, pr, with_pool=True)
    vp = paro.reorder(v, pr)
    n = 777
    at = torch.tensor([[n // 192, n // 16 % 12, n % 16]], dtype=torch.int32, device="cuda")
    token = paro.rope3d(q[:, :, n:n + 1].contiguous(), table, positions=at)
    out, idx, lse = paro.block_sparse_query_attn(token, kp, vp, pool, pr, 4)
    qp = paro.rope_reorder(q, table, pr)
    every = idx[:, :, 0][:, :, None].expand(pr.per_block + (4,)).contiguous()
    full, full_lse = paro.block_sparse_attn_lse(qp, kp, vp, pr, every)
    want = f64(full[:, :, n])
    # both within their own roundings of the same value
    size = f64(vp).max() * 4 * tr.U
    assert np.abs(f64(out[:, :, 0]) - want).max() <= size
    assert np.abs(f64(lse[:, :, 0]) - f64(full_lse[:, :, n])).max() <= 1e-4


def test_captured_and_concurrent_calls():
    c = Clip(2, 4, 2, 3, 128, 128, (5, 9, 17), BF)
    want = c.run(3, [700, 400])
    ln = torch.tensor([700, 400], dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paro.block_sparse_query_attn(c.q, c.k, c.v, c.pool, c.pr, 3, lengths=ln, out=outs[0],
                                     idx=outs[1], lse=outs[2])
    graph.replay()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    ln.copy_(torch.tensor([1, 765]))  # the clip grows between replays
    graph.replay()
    for a, b in zip(outs, c.run(3, [1, 765])):
        assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(c.run(3, [700, 400]))
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("step", [1, 7, 64])
def test_a_clip_that_grows(dtype, step):
    """Keys, values and means arrive as documented, in a cache of NaN: the
    oracle of the clip so far, whose newest keys are among the kept ones."""
    c = Clip(1, 2, 2, 3, 64, 64, (3, 9, 11), dtype)
    k, v, block = c.k.clone(), c.v.clone(), c.pr.block
    for t in (c.k, c.v, c.pool):
        t.fill_(float("nan"))
    n = 0
    while n < c.pr.N:
        start, n = n, min(n + step, c.pr.N)
        c.k[:, :, start:n], c.v[:, :, start:n] = k[:, :, start:n], v[:, :, start:n]
        for j in range(start // block, (n - 1) // block + 1):
            c.pool[:, :, j] = c.k[:, :, j * block:min((j + 1) * block, n)].float().mean(2)
        if step > 1 or n % 13 in (0, 1) or n % block in (0, 1, 63) or n == c.pr.N:
            exist = -(-n // block)
            got = c.run(2, [n])
            pool = np.zeros(c.pool.shape)
            for j in range(exist):
                pool[:, :, j] = f64(k)[:, :, j * block:min((j + 1) * block, n)].mean(2)
            assert np.abs(f64(c.pool)[:, :, :exist] - pool[:, :, :exist]).max() <= 64 * 2.0 ** -24 * 8
            want = tr.query_attention(f64(c.q), f64(k), f64(v), f64(c.pool), c.pr.N, block, 2, [n])
            assert (got[1].cpu().numpy() == want[1]).all()
            c_k, c_v = c.k, c.v
            c.k, c.v = k, v  # the oracle reads nothing behind n
            c.check(got, 2, [n])
            c.k, c.v = c_k, c_v
            # the newest block, made the best by its mean, is kept and read
            q = c.q.clone()
            c.q = c.pool[:, :, exist - 1].repeat_interleave(2, 1)[:, :, None].expand(q.shape).to(dtype).contiguous() * 8
            assert (c.run(1, [n])[1] == exist - 1).all()
            c.q = q


FIRST_CALL = """
import torch
from block_sparse_attention_34_b200 import paro
pr = paro.Problem(1, 3, (5, 9, 17), 128, 128, [0, 3, 5])
for dtype in (torch.bfloat16, torch.float32):
    k = torch.randn(pr.permuted, device="cuda").to(dtype)
    pool = k.view(1, 3, pr.NB, 128, 128).float().mean(3)
    q = torch.randn(1, 6, 2, 128, device="cuda").to(dtype)
    out, idx, lse = (torch.empty_like(q), torch.empty(1, 6, 2, 3, dtype=torch.int32, device="cuda"),
                     torch.empty(1, 6, 2, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paro.block_sparse_query_attn(q, k, k, pool, pr, 3, out=out, idx=idx, lse=lse)
    graph.replay()
    for a, b in zip((out, idx, lse), paro.block_sparse_query_attn(q, k, k, pool, pr, 3)):
        assert torch.equal(a, b)
print("fine")
"""


def test_the_first_call_of_a_process_may_be_captured():
    """What the library asks the driver once a device is asked in a capture too."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert got.returncode == 0 and got.stdout.strip() == "fine", got.stderr[-2000:]
