"""GPU parity of rotary positions with three axes (pa_rope_apply,
pa_rope_reorder) against the float64 oracle (oracle/train_ref.py), element by
element within the bounds of the roundings involved: every layout, type and
head dimension, grids and given positions, axes without pairs and pairs
without an axis, in place, on views, captured, on another stream."""

import numpy as np
import pytest
import torch

from block_sparse_attention_34_b200 import autograd, paro
from block_sparse_attention_34_b200.pipeline import Pipeline
from oracle import paro_ref as ref
from oracle import pasa_ref as pasa
from oracle import selection_ref as sel
from oracle import train_ref as tr

from helpers import compare

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def random(shape, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, x, angles, interleaved, inverse=False):
    want = tr.rope(f64(x), angles, interleaved, inverse)
    bound = tr.rope_bounds(f64(x), want, interleaved, x.dtype == BF)
    assert (np.abs(f64(got) - want) <= bound).all(), np.abs(f64(got) - want).max()


# (d, pairs, grid): default splits, an axis without pairs, unrotated pairs,
# axes that share a group of four pairs two and three at a time, one token
CASES = [
    (128, (22, 21, 21), (3, 5, 7)),
    (64, (12, 10, 10), (5, 4, 9)),
    (128, (0, 30, 20), (2, 6, 11)),
    (64, (1, 1, 1), (4, 3, 2)),
    (64, (5, 0, 27), (7, 1, 5)),
    (128, (2, 1, 60), (2, 2, 33)),
    (128, (22, 21, 21), (1, 1, 1)),
]


@pytest.mark.parametrize("interleaved", [True, False], ids=["interleaved", "halves"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,pairs,grid", CASES)
def test_grid_positions(d, pairs, grid, dtype, interleaved):
    N = grid[0] * grid[1] * grid[2]
    table = paro.RopeTable(grid, d, pairs=pairs, theta=500.0, first=(9.5, 0, -3), step=(1, 0.5, 2),
                           interleaved=interleaved)
    angles = tr.rope_angles(tr.grid_positions(grid), d, pairs, 500.0, (9.5, 0, -3), (1, 0.5, 2))
    x = random((2, 11, N, d), dtype)  # 11 heads: a group of eight and a rest
    for inverse in (False, True):
        out = torch.full_like(x, float("nan"))
        assert paro.rope3d(x, table, inverse=inverse, out=out) is out
        check(out, x, angles, interleaved, inverse)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batched", [False, True])
def test_given_positions_far_ones_and_bad_ones(dtype, batched):
    d, pairs, extent = 64, (8, 12, 12), (70000, 3, 5)
    table = paro.RopeTable(extent, d, pairs=pairs)
    rng = np.random.default_rng(1)
    shape = (3, 37, 3) if batched else (37, 3)
    pos = np.stack([rng.integers(0, e, shape[:-1]) for e in extent], -1).astype(np.int32)
    pos[..., 0, 0] = extent[0] - 1  # 7e4 radians: a 32-bit angle would be off by 4e-3
    x = random((3, 2, 37, d), dtype)
    p = torch.from_numpy(pos).cuda()
    angles = tr.rope_angles(pos, d, pairs, 10000.0)
    check(paro.rope3d(x, table, positions=p), x, angles[:, None] if batched else angles, True)
    # a coordinate outside the table: reported, its rows left as they were
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for axis, value in ((0, extent[0]), (1, -1), (2, 2**31 - 1)):
        bad = p.clone()
        bad[..., 5, axis] = value
        out = torch.full_like(x, 7.0)
        paro.clear_status(status)
        paro.rope3d(x, table, positions=bad, out=out, status=status)
        assert status.item() == paro.PA_ERR_DEVICE_CHECK
        assert (out[:, :, 5] == 7).all()
        good = [n for n in range(37) if n != 5]
        assert torch.equal(out[:, :, good], paro.rope3d(x, table, positions=p)[:, :, good])


def test_layouts_views_and_in_place():
    d, grid = 128, (3, 4, 6)
    table = paro.RopeTable(grid, d)
    N = 72
    x = random((2, 5, N, d), BF)
    want = paro.rope3d(x, table)
    token_major = x.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(paro.rope3d(token_major, table), want)
    fused = random((2, N, 3, 5, d), BF)  # q, k, v of one projection
    fused[:, :, 1] = x.transpose(1, 2)
    view = fused[:, :, 1].transpose(1, 2)
    out = torch.zeros((2, N, 5, d), dtype=BF, device="cuda").transpose(1, 2)
    paro.rope3d(view, table, out=out)
    assert torch.equal(out, want) and torch.equal(view, x)
    paro.rope3d(view, table, out=view)  # in place, among its neighbours
    assert torch.equal(view, want)
    one = x[:1].expand(2, -1, -1, -1)  # a batch that shares its memory
    assert torch.equal(paro.rope3d(one, table), want[:1].expand(2, -1, -1, -1))
    with pytest.raises(ValueError, match="overlap"):
        paro.rope3d(x, table, out=x[:1].expand(2, -1, -1, -1))
    with pytest.raises(ValueError, match="16 bytes"):
        paro.rope3d(random((1, 1, N, d + 2), BF)[..., 1:d + 1], table)
    with pytest.raises(ValueError, match="contiguous"):
        paro.rope3d(random((1, 1, N, 2 * d), BF)[..., ::2], table)


REORDER = [
    # B, heads, d, block, grid, pairs, orders: ragged tails, tile orders,
    # lists of more than eight heads of one order, orders of one head each
    (1, 3, 128, 128, (5, 7, 9), None, (0, 3, 5)),
    (2, 6, 128, 128, (5, 18, 20), (20, 20, 20), (6, 7, 8, 9, 10, 11)),
    (2, 2, 64, 64, (3, 5, 7), (2, 1, 20), (1, 4)),
    (1, 5, 64, 128, (4, 8, 8), (0, 16, 16), (2, 2, 2, 2, 0)),
    (1, 19, 128, 64, (40, 21, 33), None, (5,) * 18 + (1,)),
    (1, 1, 128, 128, (1, 1, 1), None, (0,)),
]


@pytest.mark.parametrize("interleaved", [True, False], ids=["interleaved", "halves"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,heads,d,block,grid,pairs,orders", REORDER)
def test_fused_with_the_reorder(B, heads, d, block, grid, pairs, orders, dtype, interleaved):
    pr = paro.Problem(B, heads, grid, d, block, orders)
    # a table of a larger grid: the tokens' coordinates count, not its size
    table = paro.RopeTable([e + 2 for e in grid], d, pairs=pairs, interleaved=interleaved)
    x = random((B, pr.N, heads, d), dtype).transpose(1, 2)
    out = torch.full(pr.permuted, float("nan"), dtype=dtype, device="cuda")
    pool = torch.full(pr.pooled, float("nan"), device="cuda")
    paro.rope_reorder(x, table, pr, out=out, pool=pool)
    angles = tr.rope_angles(tr.grid_positions(grid), d, table.pairs, 10000.0)
    y = tr.rope(f64(x), angles, interleaved)
    want = ref.reorder(y, grid, orders, block)
    bound = ref.reorder(tr.rope_bounds(f64(x), y, interleaved, dtype == BF), grid, orders, block)
    assert (np.abs(f64(out) - want) <= bound).all()
    means = ref.block_pool(want, pr.N, block)
    size = ref.block_pool(np.abs(want), pr.N, block) + ref.block_pool(bound, pr.N, block)
    # 128 rows' sums in fp32, of unrounded rows
    exact = ref.block_pool(ref.reorder(tr.rope_bounds(f64(x), y, interleaved, False), grid, orders,
                                       block), pr.N, block)
    assert (np.abs(f64(pool) - means) <= exact + 130 * 2.0 ** -24 * size).all()
    # the rotation alone, then the reorder: the same rows
    alone = paro.rope3d(x, table, grid=grid)
    assert torch.equal(paro.reorder(alone, pr), out)
    assert torch.equal(paro.rope_reorder(x, table, pr), out)  # without the means


def test_differentiable_captured_and_on_another_stream():
    d, grid = 64, (2, 5, 8)
    table = paro.RopeTable(grid, d, interleaved=False)
    x = random((1, 3, 80, d), F32, 2).requires_grad_()
    w = random((1, 3, 80, d), F32, 3)
    y = autograd.rope3d(x, table)
    (g,) = torch.autograd.grad((y * w).sum(), x)
    angles = tr.rope_angles(tr.grid_positions(grid), d, table.pairs, 10000.0)
    check(g, w, angles, False, inverse=True)
    # the loss is linear in x: a difference along any direction is exact
    v = random((1, 3, 80, d), F32, 4)
    diff = f64((autograd.rope3d(x + v, table) - y) * w).sum()
    assert abs(diff - (f64(g) * f64(v)).sum()) <= 1e-4 * np.abs(f64(w) * f64(v)).sum()
    (g,) = torch.autograd.grad(autograd.rope3d(x, table).sum(), x)  # an expanded gradient
    check(g, torch.ones_like(x), angles, False, inverse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = paro.rope3d(x.detach(), table)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, y)
    graph, inp, out = torch.cuda.CUDAGraph(), torch.zeros_like(w), torch.empty_like(w)
    with torch.cuda.graph(graph):
        paro.rope3d(inp, table, out=out)
    inp.copy_(x.detach())
    graph.replay()
    assert torch.equal(out, y)


@pytest.mark.parametrize("kw", [{}, {"int8": True}, {"baseline": True}, {"compensate": True},
                                {"permuted": False}, {"selection": "hybrid", "top_p": 0.4}])
def test_attention_and_pipeline_rotate_first(kw):
    """attention(rope=...) is attention of the rotated q and k: the same
    selection up to the means' rounding, the same kernels after it."""
    grid, d, heads = (4, 8, 16), 128, 3
    pr_args = (grid, [0, 4, 8], 128, 1.0)  # every block kept: no near ties
    table = paro.RopeTable(grid, d)
    q, k, v = (random((1, heads, 512, d), BF, s) for s in range(3))
    got, _ = paro.attention(q, k, v, *pr_args, rope=table, **kw)
    want, _ = paro.attention(paro.rope3d(q, table), paro.rope3d(k, table), v, *pr_args, **kw)
    assert torch.equal(got, want)
    if kw in ({}, {"int8": True}, {"baseline": True}):
        pipe = Pipeline(1, heads, grid, d, 128, [0, 4, 8], 1.0, rope=table, **kw)
        assert torch.equal(pipe.run(q, k, v), want)
        assert torch.equal(pipe.run(q, k, v), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_differentiable_on_a_table_larger_than_the_clip(dtype):
    """grid=, and the gradient against the formula's and along a direction."""
    d, grid = 128, (3, 4, 6)
    table = paro.RopeTable((5, 9, 7), d)
    x, w = random((2, 3, 72, d), dtype, 1).requires_grad_(), random((2, 3, 72, d), dtype, 2)
    y = autograd.rope3d(x, table, grid=grid)
    assert torch.equal(y, paro.rope3d(x.detach(), table, grid=grid))
    (g,) = torch.autograd.grad(y, x, w)
    angles = tr.rope_angles(tr.grid_positions(grid), d, table.pairs, 10000.0)
    check(g, w, angles, True, inverse=True)
    v = np.random.default_rng(3).standard_normal(x.shape)  # the rotation is linear
    diff = (tr.rope(v, angles, True) * f64(w)).sum()
    bound = tr.rope_bounds(f64(w), tr.rope(f64(w), angles, True, True), True, dtype == BF)
    assert abs(diff - (f64(g) * v).sum()) <= (bound * np.abs(v)).sum()
    with pytest.raises(ValueError, match="grid"):
        autograd.rope3d(x, table)


@pytest.mark.parametrize("kw", [{}, {"int8": True}, {"baseline": True}, {"compensate": True},
                                {"permuted": False}, {"selection": "hybrid", "top_p": 0.8, "window": 1}])
def test_selection_sees_the_rotated_blocks(kw):
    """attention(rope=...) and Pipeline keep the blocks that the means of the
    rotated rows choose, of inputs whose scores lie more than 0.5 apart (and
    whose unrotated means choose others), and compensate by those means."""
    grid, d, heads, block, density = (6, 8, 21), 128, 3, 128, 0.3
    orders = [0, 4, 8]
    table = paro.RopeTable(grid, d)
    pr = paro.Problem(1, heads, grid, d, block, orders)
    rng = np.random.default_rng(7)
    # along the pairs that turn fastest, two of each axis: unrotated, a block's
    # rows point everywhere
    way = np.zeros((heads, 1, 1, d))
    fast = [2 * p + e for p in (0, 1, 22, 23, 43, 44) for e in (0, 1)]
    way[..., fast] = np.sign(rng.standard_normal((heads, 1, 1, 12))) / 12 ** 0.5
    way = torch.from_numpy(way).float().cuda()
    size = torch.from_numpy(np.stack([rng.permutation(pr.NB) - 3.5 for _ in range(heads)])).float().cuda()
    sign = torch.from_numpy(np.sign(rng.standard_normal((heads, pr.NB)))).float().cuda()

    def clip(each, seed):  # rows whose rotated block means are each * way
        y = 0.3 * random((heads, pr.NB, block, d), F32, seed)
        y = (y - y.mean(2, keepdim=True) + each[..., None, None] * way).to(BF)
        y = paro.inverse_reorder(y.view(pr.permuted), pr)
        return paro.rope3d(y, table, inverse=True)

    q, k, v = clip(4 * sign, 1), clip(3 * size, 2), random(pr.natural, BF, 3)
    qr, kr = paro.rope3d(q, table), paro.rope3d(k, table)
    _, _, scores = ref.pooled_scores(f64(qr), f64(kr), grid, orders, block)
    assert np.diff(np.sort(scores, -1), axis=-1).min() > 0.5
    count = ref.k_for_density(pr.NB, density)
    if "selection" in kw:
        want = sel.hybrid_select(scores, count, kw["top_p"], kw["window"])
    else:
        want = (ref.select_topk(scores, count),)

    def same(kept):
        kept = kept if isinstance(kept, tuple) else (kept,)
        return all((a.cpu().numpy() == b).all() for a, b in zip(kept, want))

    args = (grid, orders, block, density)
    out, kept = paro.attention(q, k, v, *args, rope=table, **kw)
    assert same(kept)
    assert not same(paro.attention(q, k, v, *args, **kw)[1])
    if "compensate" in kw:
        compare(out, pasa.attention_compensated(f64(qr), f64(kr), f64(v), grid, orders, block, want[0]))
        return
    rotated, _ = paro.attention(qr, kr, v, *args, **kw)
    assert torch.equal(out, rotated)
    if "permuted" not in kw:
        pipe = Pipeline(1, heads, grid, d, block, orders, density, rope=table, **kw)
        assert torch.equal(pipe.run(q, k, v), rotated)
        assert same((pipe.idx, pipe.counts) if "selection" in kw else pipe.idx)
