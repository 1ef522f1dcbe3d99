"""Host side of the differentiable operators, on host tensors and with the
library's calls replaced: which tensors reach them."""

import pytest
import torch

from block_sparse_attention_34_b200 import autograd, paro

BF = torch.bfloat16


def fine(t):
    """What the library takes: rows contiguous, each at a multiple of 16 bytes."""
    e = 16 // t.element_size()
    return t.stride(3) == 1 and t.data_ptr() % 16 == 0 and all(
        n == 1 or s % e == 0 for n, s in zip(t.shape[:3], t.stride()))


def odd(shape, dtype=BF):
    """A contiguous tensor that starts one element behind a multiple of 16 bytes."""
    n = torch.Size(shape).numel()
    return torch.randn(n + 1).to(dtype)[1:].view(shape)


def behind(y, n):
    """A loss whose gradient of ``y`` starts n elements into a larger one."""
    joined = torch.cat((torch.zeros(n, dtype=y.dtype), y.flatten()))
    return (joined * torch.randn(joined.numel()).to(y.dtype)).sum()


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as they would be made: each checks its tensors and
    gives tensors of the right shapes."""
    seen = []

    def rope3d(x, rope, out=None, **kw):
        seen.append(("rope3d", kw))
        assert fine(x)
        y = x.clone(memory_format=torch.contiguous_format)
        return y if out is None else out.copy_(y)

    def reorder(x, pr, with_pool=False):
        assert x.is_contiguous() and x.data_ptr() % 16 == 0
        y = torch.zeros(pr.permuted, dtype=x.dtype)
        return (y, torch.zeros(pr.pooled)) if with_pool else y

    def rope_reorder(x, rope, pr, with_pool=False):
        assert fine(x)
        return reorder(x.contiguous().clone(), pr, with_pool)

    def backward(dout, q, k, v, out, lse, pr, idx, counts, dlse=None, status=None):
        assert dout.is_contiguous() and dout.data_ptr() % 16 == 0 and dout.dtype == BF
        assert dlse is None or dlse.is_contiguous()
        seen.append(("backward", {}))
        return tuple(torch.ones(pr.natural, dtype=BF) for _ in range(3))

    monkeypatch.setattr(paro, "rope3d", rope3d)
    monkeypatch.setattr(paro, "reorder", reorder)
    monkeypatch.setattr(paro, "rope_reorder", rope_reorder)
    monkeypatch.setattr(paro, "score_pooled", lambda q, k, pr: torch.zeros(pr.square))
    monkeypatch.setattr(paro, "select_topk", lambda s, pr, k: torch.zeros(pr.per_block + (k,), dtype=torch.int32))
    monkeypatch.setattr(paro, "block_sparse_attn_lse", lambda q, k, v, pr, idx, counts, status=None: (
        torch.zeros(pr.natural, dtype=BF), torch.zeros(pr.rows)))
    monkeypatch.setattr(paro, "block_sparse_attn_backward", backward)
    return seen


@pytest.fixture
def problem():
    return paro.Problem(1, 2, (3, 8, 9), 64, 64, [0, 5])


def test_a_gradient_may_start_anywhere(calls, problem):
    x = torch.randn(problem.natural).to(BF).requires_grad_()
    y = autograd.rope3d(x, None)
    got = []
    y.register_hook(lambda g: got.append((g.is_contiguous(), g.data_ptr() % 16)))
    behind(y, 3).backward()
    assert got == [(True, 6)]  # as autograd hands it over
    leaves = [torch.randn(problem.natural).to(BF).requires_grad_() for _ in range(3)]
    for rope in (None, "table"):
        out, lse = autograd.sparse_attention(*leaves, problem, density=0.5, rope=rope)
        behind(out, 5).backward()
        out, lse = autograd.sparse_attention(*leaves, problem, density=0.5, rope=rope)
        behind(lse, 5).backward()


def test_inputs_may_start_anywhere(calls, problem):
    q, k, v = (odd(problem.natural).requires_grad_() for _ in range(3))
    for rope in (None, "table"):
        out, _ = autograd.sparse_attention(q, k, v, problem, density=0.5, rope=rope)
        out.sum().backward()
        # and in any layout
        t = [x.detach().transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
        autograd.sparse_attention(*t, problem, density=0.5, rope=rope)


def test_what_fits_is_not_copied():
    x = torch.zeros(2, 3, 8, 64, dtype=BF)
    for t in (x, x.transpose(1, 2), x[:, :1], x[:1].expand(2, -1, -1, -1)):
        assert autograd._rows(t) is t
    assert autograd._whole(x) is x
    assert autograd._whole(x.transpose(1, 2)).is_contiguous()
    one = torch.zeros(3 * 8 * 64 + 1, dtype=BF).as_strided((1, 3, 8, 64), (1, 512, 64, 1))
    assert autograd._rows(one) is one  # the stride of one element says nothing
    for t in (odd((2, 3, 8, 64)), torch.zeros(2, 3, 8, 66, dtype=BF)[..., :64], x[..., ::2]):
        assert fine(autograd._rows(t)) and torch.equal(autograd._rows(t), t)


def test_a_table_larger_than_the_clip(calls):
    """``grid`` places the tokens, forward and back, as in paro.rope3d."""
    x = torch.randn(1, 2, 24, 64).requires_grad_()
    autograd.rope3d(x, None, grid=(2, 3, 4)).sum().backward()
    assert [(name, kw["grid"], kw["inverse"]) for name, kw in calls] == [
        ("rope3d", (2, 3, 4), False), ("rope3d", (2, 3, 4), True)]


@pytest.mark.parametrize("need", [(True, False, False), (False, True, True), (False, False, True), (True, True, True)])
def test_only_the_gradients_asked_for(calls, problem, need):
    """What nobody asked for is neither turned back nor handed on."""
    leaves = [torch.randn(problem.natural).to(BF).requires_grad_(n) for n in need]
    out, _ = autograd.sparse_attention(*leaves, problem, density=0.5, rope="table")
    out.sum().backward()
    assert [x.grad is not None for x in leaves] == list(need)
    assert [name for name, _ in calls] == ["backward"] + ["rope3d"] * sum(need[:2])
