"""GPU parity of training attention (pa_block_sparse_attn_lse,
pa_block_sparse_attn_backward) against the float64 oracle
(oracle/train_ref.py): every element of out, lse, dq, dk and dv within the
bounds of the roundings the kernels make, at every head dimension and block
size, ragged tails, rows without keys, keys that no row keeps, one token;
malformed lists; the same bits on every run; captured, concurrent and
differentiable calls."""

import numpy as np
import pytest
import torch

from block_sparse_attention_34_b200 import autograd, paro
from oracle import train_ref as tr

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAMES = ("out", "lse", "dq", "dk", "dv")


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, B, heads, d, block, grid, orders, k, counts=None, seed=0, size=1.0):
        self.pr = pr = paro.Problem(B, heads, grid, d, block, orders)
        self.grid, self.orders, self.block = grid, list(orders), block
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.q, self.k, self.v, self.do = (
            (s * torch.randn(pr.natural, generator=g, device="cuda")).to(BF) for s in (size, size, 1, 1))
        self.dlse = torch.randn(pr.rows, generator=g, device="cuda")
        keep = np.argsort(rng.random(pr.square), -1)[..., :k]
        self.idx_np = np.sort(keep, -1).astype(np.int32)
        self.counts_np = None
        if counts == "random":
            self.counts_np = rng.integers(0, k + 1, pr.per_block).astype(np.int32)
            self.counts_np[..., 0] = 0
        self.idx = torch.from_numpy(self.idx_np).cuda()
        self.counts = None if self.counts_np is None else torch.from_numpy(self.counts_np).cuda()
        self.perm = [paro.reorder(x, pr) for x in (self.q, self.k, self.v)]

    def forward(self, **kw):
        out = torch.full(self.pr.natural, float("nan"), dtype=BF, device="cuda")
        lse = torch.full(self.pr.rows, float("nan"), device="cuda")
        return paro.block_sparse_attn_lse(*self.perm, self.pr, self.idx, self.counts, out=out, lse=lse, **kw)

    def backward(self, out, lse, dlse=None, **kw):
        grads = [torch.full(self.pr.natural, float("nan"), dtype=BF, device="cuda") for _ in range(3)]
        return paro.block_sparse_attn_backward(self.do, *self.perm, out, lse, self.pr, self.idx,
                                               self.counts, dlse=dlse, dq=grads[0], dk=grads[1],
                                               dv=grads[2], **kw)

    def oracle(self, dlse=None):
        x = [f64(t) for t in (self.q, self.k, self.v)]
        where = (self.grid, self.orders, self.block, self.idx_np, self.counts_np)
        dl = None if dlse is None else f64(dlse)
        want = dict(zip(NAMES, (*tr.attention_lse(*x, *where),
                                *tr.attention_backward(*x, f64(self.do), *where, dl))))
        return want, tr.training_bounds(*x, f64(self.do), *where, dl)


def check(got, want, bounds, names=NAMES):
    for name in names:
        g, w = f64(got[name]), want[name]
        assert (np.isfinite(g) == np.isfinite(w)).all(), name
        fin = np.isfinite(w)
        assert (g[~fin] == w[~fin]).all(), name
        err = np.abs(g[fin] - w[fin])
        assert (err <= bounds[name][fin]).all(), (name, (err - bounds[name][fin]).max())
        if name != "lse" and np.linalg.norm(w):
            # norm-wise: three roundings of at most U each (dS or P, D, the result)
            assert np.linalg.norm(g - w) <= 3 * tr.U * np.linalg.norm(w), name


CASES = {
    "d128_b128": dict(B=1, heads=3, d=128, block=128, grid=(4, 8, 16), orders=(0, 3, 5), k=2),
    "d128_b128_ragged": dict(B=2, heads=2, d=128, block=128, grid=(5, 7, 17), orders=(1, 8), k=4, counts="random"),
    "d64_b128_ragged": dict(B=1, heads=3, d=64, block=128, grid=(3, 11, 16), orders=(2, 4, 10), k=3, counts="random"),
    "d64_b64": dict(B=1, heads=2, d=64, block=64, grid=(4, 6, 10), orders=(0, 5), k=2),
    "d64_b64_ragged": dict(B=2, heads=2, d=64, block=64, grid=(3, 9, 13), orders=(9, 1), k=5, counts="random"),
    "d128_b64_ragged": dict(B=1, heads=2, d=128, block=64, grid=(2, 11, 15), orders=(3, 6), k=4, counts="random"),
    "dense_b128": dict(B=1, heads=1, d=128, block=128, grid=(3, 9, 20), orders=(4,), k=5),
    "dense_b64": dict(B=1, heads=1, d=64, block=64, grid=(3, 9, 20), orders=(2,), k=9),
    "long_lists_b64": dict(B=1, heads=1, d=64, block=64, grid=(5, 20, 23), orders=(1,), k=30),
    "one_token_b128": dict(B=1, heads=2, d=128, block=128, grid=(1, 1, 1), orders=(0, 3), k=1),
    "one_token_b64": dict(B=2, heads=1, d=64, block=64, grid=(1, 1, 1), orders=(0,), k=1),
    "sharp_b128": dict(B=1, heads=1, d=128, block=128, grid=(2, 10, 13), orders=(5,), k=2, size=3.0),
    "sharp_b64": dict(B=1, heads=1, d=64, block=64, grid=(2, 10, 13), orders=(5,), k=3, size=4.0),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("with_dlse", [False, True])
def test_forward_and_gradients(name, with_dlse):
    c = Case(**CASES[name])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.forward(status=status)
    dlse = c.dlse if with_dlse else None
    grads = c.backward(out, lse, dlse, status=status)
    assert status.item() == 0
    want, bounds = c.oracle(dlse)
    check(dict(zip(NAMES, (out, lse, *grads))), want, bounds)
    # the same bits again, on a workspace of garbage
    ws = torch.full((paro.backward_workspace(c.pr),), 0xFF, dtype=torch.uint8, device="cuda")
    for a, b in zip(c.backward(out, lse, dlse, workspace=ws), grads):
        assert torch.equal(a, b)
    if c.pr.d == 128 and c.block == 128:
        plain = paro.block_sparse_attn(*c.perm, c.pr, c.idx, c.counts, permuted=True)
        assert torch.equal(plain, out)


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 64), (64, 128)])
def test_no_keys_at_all(block, d):
    pr = paro.Problem(1, 2, (3, 7, 9), d, block, [0, 5])
    x = torch.randn(pr.permuted, device="cuda").to(BF)
    do = torch.randn(pr.natural, device="cuda").to(BF)
    counts = torch.zeros(pr.per_block, dtype=torch.int32, device="cuda")
    for width, cnt in ((0, None), (1, counts)):
        idx = torch.zeros(pr.per_block + (width,), dtype=torch.int32, device="cuda")
        out, lse = paro.block_sparse_attn_lse(x, x, x, pr, idx, cnt)
        assert (out == 0).all() and (lse == -float("inf")).all()
        for g in paro.block_sparse_attn_backward(do, x, x, x, out, lse, pr, idx, cnt):
            assert (g == 0).all()


@pytest.mark.parametrize("block,d", [(128, 128), (64, 64)])
def test_keys_that_no_row_keeps(block, d):
    c = Case(1, 1, d, block, (4, 8, 16), (0,), 1)
    c.idx.fill_(1)
    c.idx_np[...] = 1
    out, lse = c.forward()
    _, dk, dv = c.backward(out, lse)
    other = [p for p in range(512) if p // block != 1]  # order FHW: positions are tokens
    assert (dk[:, :, other] == 0).all() and (dv[:, :, other] == 0).all()
    want, bounds = c.oracle()
    check({"dk": dk, "dv": dv}, want, bounds, ("dk", "dv"))


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 64)])
def test_malformed_lists_are_reported_and_left_out(block, d):
    c = Case(1, 1, d, block, (4, 8, 16), (0,), 2)
    good_out, good_lse = c.forward()
    for bad in ([3, 1], [1, 1], [0, c.pr.NB], [-1, 2]):
        c.idx[0, 0, 1] = torch.tensor(bad, dtype=torch.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = c.forward(status=status)
        torch.cuda.synchronize()
        assert status.item() == paro.PA_ERR_DEVICE_CHECK
        rows = [p for p in range(512) if p // block != 1]
        assert out[:, :, block:2 * block].isnan().all() and lse[:, :, block:2 * block].isnan().all()
        assert torch.equal(out[:, :, rows], good_out[:, :, rows])
        paro.clear_status(status)
        dq, dk, dv = c.backward(good_out, good_lse, status=status)
        assert status.item() == paro.PA_ERR_DEVICE_CHECK
        assert dq[:, :, block:2 * block].isnan().all() and not dq[:, :, rows].isnan().any()
        # dk, dv as with an empty list there
        counts = torch.full(c.pr.per_block, 2, dtype=torch.int32, device="cuda")
        counts[0, 0, 1] = 0
        c.counts, kept = counts, c.idx.clone()
        c.idx[0, 0, 1] = torch.tensor([0, 1], dtype=torch.int32)
        _, dk2, dv2 = c.backward(good_out, good_lse)
        assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
        c.counts, c.idx = None, kept


@pytest.mark.parametrize("block,d", [(128, 128), (64, 64)])
def test_nan_stays_in_its_rows(block, d):
    """A NaN key reaches the rows that keep its block and no other."""
    c = Case(1, 1, d, block, (4, 8, 16), (0,), 1)
    c.idx[0, 0] = torch.arange(c.pr.NB, dtype=torch.int32)[:, None]  # each block its own
    c.k[0, 0, block + 3] = float("nan")
    c.perm[1] = paro.reorder(c.k, c.pr)
    out, lse = c.forward()
    dq, dk, dv = c.backward(out, lse)
    rows = [p for p in range(512) if p // block != 1]
    for t in (out, dq, dk, dv):
        assert t[:, :, rows].isfinite().all()
        assert t[:, :, block:2 * block].isnan().any()


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("up", [True, False], ids=["growing", "falling"])
def test_scores_that_grow_or_fall_along_the_list(block, d, up):
    """The running reference of a row moves at most steps, or at the first alone."""
    nb = -(-4 * 10 * 13 // block)
    c = Case(B=1, heads=2, d=d, block=block, grid=(4, 10, 13), orders=(0, 3), k=nb)
    steps = torch.linspace(-2, 3, nb).round().exp2()  # powers of two: exact in bf16
    steps = (steps if up else steps.flip(0)).to("cuda", BF)
    kp = c.perm[1].view(1, 2, nb, block, d) * steps[:, None, None]
    c.perm[1] = kp.view(c.pr.permuted)
    c.k = paro.inverse_reorder(c.perm[1], c.pr)
    out, lse = c.forward()
    grads = c.backward(out, lse, c.dlse)
    want, bounds = c.oracle(c.dlse)
    check(dict(zip(NAMES, (out, lse, *grads))), want, bounds)


def test_difference_along_a_direction():
    """The kernels' gradients against differences of the oracle's loss."""
    c = Case(**CASES["d64_b128_ragged"])
    out, lse = c.forward()
    grads = c.backward(out, lse)
    x = [f64(t) for t in (c.q, c.k, c.v)]
    _, bounds = c.oracle()
    rng = np.random.default_rng(3)
    for i, name in enumerate(("dq", "dk", "dv")):
        v = rng.standard_normal(x[i].shape)
        f = []
        for s in (1e-4, -1e-4):
            y = [a + s * v if j == i else a for j, a in enumerate(x)]
            o, _ = tr.attention_lse(*y, c.grid, c.orders, c.block, c.idx_np, c.counts_np)
            f.append((o * f64(c.do)).sum())
        assert abs((f[0] - f[1]) / 2e-4 - (f64(grads[i]) * v).sum()) <= (bounds[name] * np.abs(v)).sum() + 1e-3


def test_autograd_with_rope_selection_and_graphs():
    """rope, reorder, selection, attention and their gradients as a training
    step runs them, against the steps one by one; then captured and
    replayed."""
    grid, d, heads = (4, 8, 20), 128, 3
    pr = paro.Problem(1, heads, grid, d, 128, [0, 3, 8])
    table = paro.RopeTable((6, 8, 20), d)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    leaves = [torch.randn((1, pr.N, heads, d), generator=g, device="cuda").to(BF).requires_grad_()
              for _ in range(3)]
    do = torch.randn(pr.natural, generator=g, device="cuda").to(BF)
    dlse = torch.randn(pr.rows, generator=g, device="cuda")

    def step():
        q, k, v = (x.transpose(1, 2) for x in leaves)
        return autograd.sparse_attention(q, k, v, pr, density=0.6, rope=table)

    out, lse = step()
    grads = torch.autograd.grad((out, lse), leaves, (do, dlse), retain_graph=True)
    q, k, v = (x.detach().transpose(1, 2) for x in leaves)
    (qp, qm), (kp, km) = (paro.rope_reorder(x, table, pr, with_pool=True) for x in (q, k))
    vp = paro.reorder(v.contiguous(), pr)
    idx = paro.select_topk(paro.score_pooled(qm, km, pr), pr, paro.k_for_density(pr.NB, 0.6))
    out2, lse2 = paro.block_sparse_attn_lse(qp, kp, vp, pr, idx)
    dq, dk, dv = paro.block_sparse_attn_backward(do, qp, kp, vp, out2, lse2, pr, idx, dlse=dlse)
    dq, dk = (paro.rope3d(x, table, inverse=True, grid=grid) for x in (dq, dk))
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for a, b in zip(grads, (dq, dk, dv)):
        assert torch.equal(a, b.transpose(1, 2))
    # only lse used; only out used
    (a,) = torch.autograd.grad(lse, leaves[:1], dlse, retain_graph=True)
    b, _, _ = paro.block_sparse_attn_backward(torch.zeros_like(do), qp, kp, vp, out2, lse2, pr, idx, dlse=dlse)
    assert torch.equal(a, paro.rope3d(b, table, inverse=True, grid=grid).transpose(1, 2))
    assert torch.equal(torch.autograd.grad(out, leaves[2:], do, retain_graph=True)[0],
                       dv.transpose(1, 2))

    # captured on leaves that no eager graph holds (torch.autograd would
    # otherwise wait for the stream of that graph, which a capture forbids)
    leaves = [x.detach().clone().requires_grad_() for x in leaves]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = step()
        captured = torch.autograd.grad((o, l), leaves, (do, dlse))
    for t in captured:
        t.zero_()
    graph.replay()
    for a, b in zip(captured, grads):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two backward passes on two streams, each with its own workspace."""
    cases = [Case(**CASES[n]) for n in ("d128_b128_ragged", "d64_b64_ragged")]
    fwd = [c.forward() for c in cases]
    want = [c.backward(*f) for c, f in zip(cases, fwd)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for c, f, s in zip(cases, fwd, streams):
            with torch.cuda.stream(s):
                got.append(c.backward(*f))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_the_480p_layer_on_sampled_rows():
    """A full-size layer (three heads): lse and out on sampled rows, dq there,
    dk and dv of one key block, in 64 bits on the GPU by plain torch."""
    pr = paro.Problem(1, 3, (21, 30, 52), 128, 128, [0, 2, 5])
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q, k, v, do = (torch.randn(pr.natural, generator=g, device="cuda").to(BF) for _ in range(4))
    idx = torch.rand(pr.square, generator=g, device="cuda").argsort(-1)[..., :64].sort(-1).values.int()
    qp, kp, vp, dop = (paro.reorder(x, pr) for x in (q, k, v, do))
    out, lse = paro.block_sparse_attn_lse(qp, kp, vp, pr, idx)
    grads = paro.block_sparse_attn_backward(do, qp, kp, vp, out, lse, pr, idx)
    out, dq, dk, dv = (paro.reorder(x, pr).double() for x in (out, *grads))
    scale = 128 ** -0.5

    def rows(h, i):  # query block i of head h in 64 bits
        keys = (idx[0, h, i].long()[:, None] * 128 + torch.arange(128, device="cuda")).flatten()
        a = slice(i * 128, (i + 1) * 128)
        Q, K, V, D = qp[0, h, a].double(), kp[0, h, keys].double(), vp[0, h, keys].double(), dop[0, h, a].double()
        s = (Q @ K.T * scale).masked_fill(keys >= pr.N, -float("inf"))
        p = torch.softmax(s, 1)
        o, dp = p @ V, D @ V.T
        ds = p * (dp - (D * o).sum(1, keepdim=True)) * scale
        return keys, a, p, o, ds, K, Q, D

    def near(x, y):
        assert (x - y).norm() <= 3 * tr.U * y.norm()

    for h, i in ((0, 0), (1, 133), (2, 254)):
        _, a, _, o, ds, K, _, _ = rows(h, i)
        near(out[0, h, a], o)
        near(dq[0, h, a], ds @ K)
    h, j = 1, 77
    sk, sv = torch.zeros(128, 128, device="cuda").double(), torch.zeros(128, 128, device="cuda").double()
    for i in (idx[0, h] == j).any(-1).nonzero()[:, 0].tolist():
        keys, _, p, _, ds, _, Q, D = rows(h, i)
        cols = keys // 128 == j
        valid = torch.arange(i * 128, (i + 1) * 128, device="cuda") < pr.N
        sk += (ds[valid][:, cols]).T @ Q[valid]
        sv += (p[valid][:, cols]).T @ D[valid]
    near(dk[0, h, j * 128:(j + 1) * 128], sk)
    near(dv[0, h, j * 128:(j + 1) * 128], sv)


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 128), (64, 64)])
def test_an_expired_status_ends_every_pass(block, d):
    """A status word that already records PA_ERR_TIMEOUT: forward and backward
    return at once, write nothing and leave it as it was; a normal call
    follows on the cleared word."""
    c = Case(2, 3, d, block, (5, 16, 17), (0, 3, 5), 3, counts="random")
    out, lse = c.forward()
    want = c.backward(out, lse, c.dlse)
    status = torch.full((1,), paro.PA_ERR_TIMEOUT, dtype=torch.int32, device="cuda")
    ended = (*c.forward(status=status), *c.backward(out, lse, c.dlse, status=status))
    assert status.item() == paro.PA_ERR_TIMEOUT
    assert all(t.isnan().all() for t in ended)
    paro.clear_status(status)
    for a, b in zip((*c.forward(status=status), *c.backward(out, lse, c.dlse, status=status)),
                    (out, lse, *want)):
        assert torch.equal(a, b)
    assert status.item() == 0


def many_blocks(d, block, seed):
    """600 blocks of 40 heads, more than four for each CTA of the persistent
    backward kernel, whose lists have 0 to 7 entries, with runs of lists of
    none and of one and a head without any."""
    c = Case(1, 40, d, block, (5, 19, 4 * block // 25), [h % 12 for h in range(40)], 7, counts="random", seed=seed)
    n = c.counts_np.reshape(-1)
    assert n.size >= 4 * 148
    n[90:130] = 0
    n[300:340] = 1
    n[450:470] = np.arange(20) % 2
    c.counts_np[0, 33] = 0
    c.counts = torch.from_numpy(c.counts_np).cuda()
    return c


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 64)])
def test_many_blocks_of_many_lengths(block, d):
    c = many_blocks(d, block, 11)
    out, lse = c.forward()
    grads = c.backward(out, lse, c.dlse)
    want, bounds = c.oracle(c.dlse)
    check(dict(zip(NAMES, (out, lse, *grads))), want, bounds)
    for _ in range(6):  # whichever CTA takes a block
        for a, b in zip(c.backward(out, lse, c.dlse), grads):
            assert torch.equal(a, b)


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 64)])
def test_malformed_lists_among_many_blocks(block, d):
    """They add nothing and their rows of dq stay as they were; every other
    block's sums are as if they kept nothing."""
    c = many_blocks(d, block, 12)
    bad = [(0, 1), (0, 2), (7, 0), (13, 5), (13, 6), (13, 7), (30, 14), (39, 14)]
    for h, i in bad:
        c.counts_np[0, h, i] = 0
    c.counts = torch.from_numpy(c.counts_np).cuda()
    out, lse = c.forward()
    want, bounds = c.oracle()
    for n, (h, i) in enumerate(bad):
        c.idx[0, h, i] = torch.arange(7, dtype=torch.int32)
        c.idx[0, h, i, 1] = (0, c.pr.NB, -1, 2)[n % 4]
        c.counts[0, h, i] = (7, 3)[n % 2] if n != 5 else 8  # 8: more entries than there are
    rows = torch.zeros(c.pr.permuted, dtype=BF, device="cuda")
    for h, i in bad:
        rows[0, h, i * block:(i + 1) * block] = 1
    rows = paro.inverse_reorder(rows, c.pr)[..., 0] == 1
    first = None
    for _ in range(4):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dq, dk, dv = c.backward(out, lse, status=status)
        assert status.item() == paro.PA_ERR_DEVICE_CHECK
        assert dq[rows].isnan().all()
        dq[rows] = 0
        check({"dq": dq, "dk": dk, "dv": dv}, want, bounds, ("dq", "dk", "dv"))
        first = first or (dq, dk, dv)
        assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), first))


@pytest.mark.parametrize("rotated", [False, True])
def test_gradients_and_inputs_that_start_anywhere(rotated):
    """A part of a concatenation hands its gradient over at any address."""
    pr = paro.Problem(1, 2, (3, 8, 9), 64, 64, [0, 5])
    table = paro.RopeTable((3, 8, 9), 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    data = [torch.randn(pr.natural, generator=g, device="cuda").to(BF) for _ in range(3)]
    w = torch.randn(3 + data[0].numel(), generator=g, device="cuda").to(BF)

    def grads(join, place):
        leaves = [place(x).requires_grad_() for x in data]
        out, _ = autograd.sparse_attention(*leaves, pr, density=0.5, rope=table if rotated else None)
        x = place(data[0]).requires_grad_()
        turned = autograd.rope3d(x, table) if x.data_ptr() % 16 == 0 else None
        both = [t for t in (out, turned) if t is not None]
        for t in both:
            if join:
                t = torch.cat((torch.zeros(3, dtype=BF, device="cuda"), t.flatten()))
                (t * w).sum().backward()
            else:
                (t * w[3:].clone().view(pr.natural)).sum().backward()
        return [x.grad for x in leaves] + ([x.grad] if turned is not None else [])

    def odd(x):
        return torch.cat((x.new_zeros(1), x.flatten()))[1:].view(x.shape)

    want = grads(False, torch.clone)
    for a, b in zip(grads(True, torch.clone), want):
        assert torch.equal(a, b)
    for a, b in zip(grads(True, odd), want[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("block,d", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_an_infinity_stays_one(block, d, k):
    """An infinite value or gradient gives infinities where its weight meets
    it, for lists of odd and of even length, and touches nothing else."""
    c = Case(1, 2, d, block, (4, 13, 16), (0, 0), k, seed=k)  # order FHW: positions are tokens
    out, lse = c.forward()
    grads = c.backward(out, lse)
    keep = torch.zeros(c.pr.square, dtype=torch.bool, device="cuda").scatter_(3, c.idx.long(), True)
    of = torch.arange(c.pr.N, device="cuda") // block
    j = int(c.idx[0, 0, 1, -1])  # kept by the second block of the first head
    at = min(j * block + 9, c.pr.N - 1)

    clean = c.perm[2].clone()
    c.perm[2][0, 0, at, 5] = float("inf")
    got, same = c.forward()
    assert torch.equal(same, lse)
    want = out.clone()
    want[0, 0, :, 5] = torch.where(keep[0, 0, of, j], float("inf"), want[0, 0, :, 5].float()).to(BF)
    assert torch.equal(got, want)

    c.perm[2], at = clean, block + 3
    c.do[0, 0, at, 7] = float("inf")
    dv = c.backward(out, lse)[2]
    want = grads[2].clone()
    want[0, 0, :, 7] = torch.where(keep[0, 0, 1, of], float("inf"), want[0, 0, :, 7].float()).to(BF)
    assert torch.equal(dv, want)


@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 128), (64, 64)])
def test_a_row_whose_keys_all_score_minus_infinity(block, d):
    """It is a row without keys: zeros and -inf, no gradient of its own, and
    nothing of it in its keys' gradients."""
    c = Case(1, 1, d, block, (4, 13, 16), (0,), 3, counts="random", seed=4)  # positions are tokens
    c.counts_np[...] = 3
    c.counts = torch.from_numpy(c.counts_np).cuda()
    at = [5, block + 7, c.pr.N - 1]
    c.q[..., 0] = 0
    c.k[..., 0] = -1e20
    c.do[0, 0, at] = 0

    def run(value):
        c.q[0, 0, at, 0] = value
        c.perm[:2] = [paro.reorder(x, c.pr) for x in (c.q, c.k)]
        out, lse = c.forward()
        return out, lse, c.backward(out, lse)

    out0, lse0, want = run(0.0)
    out, lse, _ = run(1e20)  # 1e20 * -1e20 is beyond 32 bits
    assert (out[0, 0, at] == 0).all() and (lse[0, 0, at] == -float("inf")).all()
    rest = torch.ones(c.pr.N, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(out[0, 0, rest], out0[0, 0, rest]) and torch.equal(lse[0, 0, rest], lse0[0, 0, rest])
    c.do[0, 0, at] = 3.0
    dq, dk, dv = c.backward(out, lse)
    assert (dq[0, 0, at] == 0).all() and torch.equal(dq[0, 0, rest], want[0][0, 0, rest])
    assert torch.equal(dk, want[1]) and torch.equal(dv, want[2])


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("block,d", [(128, 128), (128, 64), (64, 128), (64, 64)])
def test_nan_keys_give_a_nan_log_sum(block, d, k):
    """Where out is NaN so is lse, a block of nothing but NaN included: -inf
    would say that the row has no keys."""
    c = Case(1, 1, d, block, (4, 13, 16), (0,), k, seed=k)  # order FHW: positions are tokens
    clean = c.forward()
    keep = torch.zeros(c.pr.square, dtype=torch.bool, device="cuda").scatter_(3, c.idx.long(), True)
    of = torch.arange(c.pr.N, device="cuda") // block
    j = int(c.idx[0, 0, 1, 0])
    hit = keep[0, 0, of, j]
    for rows in (slice(0, block), slice(3, 4)):  # every key of the block, one of them
        kp = c.perm[1].clone()
        c.perm[1][0, 0, j * block:(j + 1) * block][rows] = float("nan")
        out, lse = c.forward()
        c.perm[1] = kp
        assert out[0, 0, hit].isnan().all() and lse[0, 0, hit].isnan().all()
        assert torch.equal(out[0, 0, ~hit], clean[0][0, 0, ~hit])
        assert torch.equal(lse[0, 0, ~hit], clean[1][0, 0, ~hit])
