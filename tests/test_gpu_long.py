"""GPU: offsets that pass 32 bits.  33 heads of 524,288 tokens at d = 128 are
2^31 elements and one head more; what an operator makes of the last head is
what it makes of that head alone, bit for bit.  And two host threads that
call at once."""

import threading

import pytest
import torch

from block_sparse_attention_34_b200 import paro

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GRID = (32, 128, 128)
HEADS, D, ORDER = 33, 128, 4


def problem(heads, block):
    return paro.Problem(1, heads, GRID, D, block, [ORDER] * heads)


def tensor(pr, seed, dtype=BF):
    """Zeros but for the last head and, as far from zero, the first."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.zeros(pr.natural, dtype=dtype, device="cuda")
    for h in (0, HEADS - 1):
        x[:, h] = torch.randn(pr.natural[2:], generator=g, device="cuda").to(dtype)
    return x


def last(x):
    return x[:, HEADS - 1:].clone()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rotation(dtype):
    many, one = problem(HEADS, 128), problem(1, 128)
    rope = paro.RopeTable(GRID, D)
    x = tensor(many, 0, dtype)
    alone = last(x)
    assert torch.equal(last(paro.rope3d(x, rope)), paro.rope3d(alone, rope))
    # rows of a [B, N, heads, d] tensor, whose last rows lie behind 2^31
    turned = x.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(last(paro.rope3d(turned, rope)), paro.rope3d(alone, rope))
    for a, b in zip(paro.rope_reorder(turned, rope, many, with_pool=True),
                    paro.rope_reorder(alone, rope, one, with_pool=True)):
        assert torch.equal(last(a), b)


@pytest.mark.parametrize("block", [128, 64])
def test_training(block):
    many, one = problem(HEADS, block), problem(1, block)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    # three kept blocks a row, ascending, the first and the last among them
    idx = torch.randint(1, one.NB - 1, one.per_block + (3,), generator=g, device="cuda", dtype=torch.int32)
    idx[..., 0] = 0
    idx[..., 2] = one.NB - 1
    q, k, v, do = (tensor(many, s) for s in range(4))
    alone = [last(t) for t in (q, k, v, do)]

    def run(pr, q, k, v, do):
        lists = idx.expand(pr.B, pr.heads, -1, -1).contiguous()
        # (the copies are any tensors of the permuted shape here: N_p = N)
        out, lse = paro.block_sparse_attn_lse(q, k, v, pr, lists)
        return (out, lse, *paro.block_sparse_attn_backward(do, q, k, v, out, lse, pr, lists))

    for a, b in zip(run(many, q, k, v, do), run(one, *alone)):
        assert torch.equal(last(a), b)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_query_rows(dtype):
    many, one = problem(HEADS, 128), problem(1, 128)
    k, v = tensor(many, 5, dtype), tensor(many, 6, dtype)
    alone = [last(t) for t in (k, v)]
    pool = k.view(1, HEADS, many.NB, 128, D).float().mean(3)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    q = torch.randn((1, HEADS, 2, D), generator=g, device="cuda").to(dtype)
    out, idx, lse = paro.block_sparse_query_attn(q, k, v, pool, many, 40)
    o1, i1, l1 = paro.block_sparse_query_attn(last(q), *alone, last(pool), one, 40)
    assert torch.equal(last(idx), i1)
    # another number of CTAs joins the row: sums of 5120 keys in another order,
    # out by a few 2^-24 of the largest value (|v| < 8) before its rounding
    slack = 64 * 2.0 ** -24 * 8
    eps = torch.finfo(dtype).eps
    assert ((last(out) - o1).abs().double() <= eps * o1.abs().double() + slack).all()
    assert (last(lse) - l1).abs().max() <= 64 * 2.0 ** -24 * l1.abs().max()


def test_two_host_threads():
    def work(n, fail):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                grid = (1 + n, 16, 16)
                pr = paro.Problem(1, 2, grid, 128, 128, [0, 3])
                g = torch.Generator(device="cuda")
                g.manual_seed(n)
                x = [torch.randn(pr.natural, generator=g, device="cuda").to(BF) for _ in range(3)]
                rope = paro.RopeTable(grid, 128)
                want = None
                for _ in range(20):
                    qp, kp = (paro.rope_reorder(t, rope, pr, with_pool=True) for t in x[:2])
                    vp = paro.reorder(x[2], pr)
                    keep = pr.NB // 2 + 1
                    idx = paro.select_topk(paro.score_pooled(qp[1], kp[1], pr), pr, keep)
                    out, lse = paro.block_sparse_attn_lse(qp[0], kp[0], vp, pr, idx)
                    got = (out, lse, *paro.block_sparse_attn_backward(x[0], qp[0], kp[0], vp, out, lse, pr, idx),
                           *paro.block_sparse_query_attn(x[0][:, :, :5].contiguous(), kp[0], vp, kp[1], pr, keep))
                    torch.cuda.current_stream().synchronize()
                    if want is None:
                        want = got
                    assert all(torch.equal(a, b) for a, b in zip(got, want))
        except BaseException as e:  # for the main thread
            fail.append(e)

    fail = []
    threads = [threading.Thread(target=work, args=(n, fail)) for n in range(1, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fail, fail
