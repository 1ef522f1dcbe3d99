"""Host-side checks of rotary positions, training attention and single-token
queries: what the library and the binding refuse before any launch (so these
run without a GPU)."""

import copy
import ctypes
import os
import pickle

import numpy as np
import pytest
import torch

from block_sparse_attention_34_b200 import autograd, paro

FAKE = ctypes.c_void_p(4096)  # never dereferenced: every case fails validation first
OFF = ctypes.c_void_p(4100)   # not 16-byte aligned
INV, UNS = paro.PA_ERR_INVALID_ARG, paro.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(paro.LIB_PATH):
        from block_sparse_attention_34_b200 import build
        build.build()
    return paro.load()


def perms(*ids):
    a = np.array(ids, dtype=np.int8)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def rope(extent=(4, 8, 8), pairs=(12, 10, 10), inter=1):
    three = ctypes.c_int32 * 3
    return paro.PaRope(three(*extent), three(*pairs), inter)


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


SHAPE = paro.PaShape(1, 2, 4, 8, 8, 64, 64)


def test_rope_tables(lib):
    # rows of whole groups of four pairs, cosines and sines, and one row of
    # the pairs that stay
    assert lib.pa_rope_table_floats(rope()) == 8 * (4 * 3 + 8 * 3 + 8 * 3 + 8)
    assert lib.pa_rope_table_floats(rope(pairs=(0, 64, 0))) == 8 * 8 * 16
    for bad in (rope(extent=(0, 8, 8)), rope(pairs=(-1, 4, 4)), rope(pairs=(0, 0, 0)),
                rope(pairs=(30, 30, 30)), rope(inter=2), rope(extent=(2**30, 2**30, 1))):
        assert lib.pa_rope_table_floats(bad) == -1
    one = (ctypes.c_double * 3)(1, 1, 1)
    nan = (ctypes.c_double * 3)(1, float("nan"), 1)
    for args in ((rope(pairs=(0, 0, 0)), 1e4, one, one, FAKE), (rope(), 0.0, one, one, FAKE),
                 (rope(), float("inf"), one, one, FAKE), (rope(), 1e4, nan, one, FAKE),
                 (rope(), 1e4, one, nan, FAKE), (rope(), 1e4, None, one, FAKE),
                 (rope(), 1e4, one, one, None), (rope(), 1e4, one, one, OFF)):
        assert lib.pa_rope_table(*args, None) == INV


def test_rope_apply_refusals(lib):
    def call(x=FAKE, xs=None, y=OFF, ys=None, dtype=paro.PA_BF16, shape=SHAPE, r=None, table=FAKE,
             positions=None, batched=0, flags=0):
        return lib.pa_rope_apply(x, xs, y, ys, dtype, shape, r or rope(), table, positions, batched, flags,
                                 None, None)

    assert call() == INV and b"aligned" in lib.pa_last_error()
    y = ctypes.c_void_p(8192)
    assert call(dtype=paro.PA_I8, y=y) == INV
    assert call(x=None, y=y) == INV and call(y=None) == INV and call(y=y, table=OFF) == INV
    assert call(y=y, shape=paro.PaShape(1, 2, 4, 8, 8, 96, 64)) == UNS
    assert call(y=y, r=rope(pairs=(20, 10, 10))) == INV and b"d/2" in lib.pa_last_error()
    assert call(y=y, r=rope(extent=(3, 8, 8))) == INV and b"cover" in lib.pa_last_error()
    assert call(y=y, xs=strides(64, 64, 4)) == INV and b"16 bytes" in lib.pa_last_error()
    assert call(y=y, ys=strides(64, -8, 64)) == INV
    assert call(y=y, flags=2) == INV and call(y=y, batched=2) == INV
    assert call(y=FAKE, xs=strides(0, 64, 128)) == INV and b"equal strides" in lib.pa_last_error()
    assert call(y=y, shape=paro.PaShape(65536, 2, 4, 8, 8, 64, 64)) == UNS


def test_rope_reorder_refusals(lib):
    keep, pp = perms(0, 5)
    keep2, bad = perms(0, 12)

    def call(x=FAKE, xs=None, xp=FAKE, dtype=paro.PA_F32, shape=SHAPE, p=pp, r=None, table=FAKE):
        return lib.pa_rope_reorder(x, xs, xp, dtype, shape, p, r or rope(), table, None, None)

    assert call(p=bad) == INV and call(p=None) == INV and call(x=None) == INV and call(xp=OFF) == INV
    assert call(r=rope(extent=(4, 8, 7))) == INV and call(table=None) == INV
    assert call(xs=strides(64, 64, 2)) == INV
    keep3, many = perms(*[0] * 1000)
    assert call(shape=paro.PaShape(66, 1000, 4, 8, 8, 64, 64), p=many) == UNS


def test_training_refusals(lib):
    keep, pp = perms(0, 5)

    def fwd(q=FAKE, dtype=paro.PA_BF16, shape=SHAPE, idx=FAKE, k=2, out=FAKE, lse=FAKE):
        return lib.pa_block_sparse_attn_lse(q, FAKE, FAKE, dtype, shape, pp, idx, None, k, out, lse, None, None)

    assert fwd(dtype=paro.PA_F32) == UNS and b"PA_BF16" in lib.pa_last_error()
    assert fwd(q=None) == INV and fwd(q=OFF) == INV and fwd(idx=None) == INV and fwd(lse=None) == INV
    assert fwd(k=5) == INV and fwd(k=-1) == INV  # NB = 4
    assert fwd(shape=paro.PaShape(1, 2, 4, 8, 8, 64, 32)) == UNS
    assert fwd(shape=paro.PaShape(1, 2, 1, 1, 65536 * 64, 64, 64)) == UNS
    n = lib.pa_block_sparse_attn_backward_workspace(SHAPE)
    # dO permuted, two statistics a row, one bit a pair of blocks, the lists'
    # lengths, two counters
    assert n == 2 * 256 * 64 * 2 + 2 * (2 * 256 * 4) + 3 * 256
    assert lib.pa_block_sparse_attn_backward_workspace(paro.PaShape(1, 2, 4, 8, 8, 65, 64)) == -1
    assert lib.pa_block_sparse_attn_backward_workspace(paro.PaShape(70000, 1, 4, 8, 8, 64, 64)) == -1

    def bwd(dout=FAKE, dtype=paro.PA_BF16, lse=FAKE, idx=FAKE, k=2, dq=FAKE, ws=FAKE, size=n):
        return lib.pa_block_sparse_attn_backward(dout, FAKE, FAKE, FAKE, FAKE, lse, None, dtype, SHAPE, pp, idx,
                                                 None, k, dq, FAKE, FAKE, ws, size, None, None)

    assert bwd(dtype=paro.PA_F32) == UNS and bwd(dout=None) == INV and bwd(lse=None) == INV
    assert bwd(dq=OFF) == INV and bwd(idx=None) == INV and bwd(k=5) == INV
    assert bwd(ws=None) == INV and bwd(ws=ctypes.c_void_p(4096 + 16)) == INV
    assert bwd(size=n - 1) == INV and b"workspace" in lib.pa_last_error()


def test_query_refusals(lib):
    def call(q=FAKE, dtype=paro.PA_BF16, shape=SHAPE, group=1, M=1, keep=2, out=FAKE, idx=FAKE):
        return lib.pa_query_attn(q, FAKE, FAKE, FAKE, dtype, shape, group, M, keep, None, out, idx, None, None, None)

    assert call(dtype=paro.PA_I8) == INV and call(q=None) == INV and call(out=OFF) == INV
    assert call(idx=None) == INV and call(group=0) == INV and call(M=0) == INV
    assert call(keep=0) == INV and call(keep=5) == INV
    assert call(M=2**27) == UNS and call(group=2**30, M=2**30) == UNS
    assert call(shape=paro.PaShape(1, 2, 1, 1, 14529 * 64, 64, 64)) == UNS


def test_the_binding_refuses_host_tensors_and_wrong_shapes(lib):
    pr = paro.Problem(1, 2, (4, 8, 8), 64, 64, [0, 5])
    x = torch.zeros(pr.natural, dtype=torch.bfloat16)
    xp = torch.zeros(pr.permuted, dtype=torch.bfloat16)
    idx = torch.zeros(pr.per_block + (2,), dtype=torch.int32)
    lse = torch.zeros(pr.rows)
    with pytest.raises(ValueError, match="CUDA"):
        paro.RopeTable((4, 8, 8), 64, device="cpu")
    with pytest.raises(ValueError, match="malformed"):
        paro.RopeTable((4, 8, 8), 64, pairs=(20, 10, 10))
    with pytest.raises(ValueError, match="extents"):
        paro.RopeTable((0, 8, 8), 64)
    with pytest.raises(ValueError, match="per axis"):
        paro.RopeTable((8, 8), 64)
    for call in (lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx),
                 lambda: paro.block_sparse_attn_backward(x, xp, xp, xp, x, lse, pr, idx),
                 lambda: paro.block_sparse_query_attn(x[:, :, :1], xp, xp, torch.zeros(pr.pooled), pr, 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert paro.backward_workspace(pr) == lib.pa_block_sparse_attn_backward_workspace(pr.shape)
    with pytest.raises(paro.ParoError):
        paro.backward_workspace(paro.Problem(1, 2, (4, 8, 8), 65, 64, [0, 5]))
    with pytest.raises(ValueError, match="either"):
        autograd.sparse_attention(x, x, x, pr)
    with pytest.raises(ValueError, match="counts"):
        autograd.sparse_attention(x, x, x, pr, density=0.5, counts=idx)


@pytest.fixture
def device_blind(monkeypatch):
    """The binding's checks of shapes and types alone, on host tensors; the
    library must not be reached."""
    monkeypatch.setattr(paro, "_device_of", lambda t: t.get_device())
    monkeypatch.setattr(paro, "_launch", lambda *a: pytest.fail("the call reached the library"))


def test_the_binding_checks_every_tensor(lib, device_blind):
    pr = paro.Problem(1, 2, (3, 8, 9), 64, 64, [0, 5])  # 216 tokens, 4 blocks
    bf = torch.bfloat16
    x, xp = torch.zeros(pr.natural, dtype=bf), torch.zeros(pr.permuted, dtype=bf)
    idx, lse, pool = torch.zeros(pr.per_block + (2,), dtype=torch.int32), torch.zeros(pr.rows), torch.zeros(pr.pooled)
    q = torch.zeros(1, 4, 3, 64, dtype=bf)
    bad = [
        lambda: paro.block_sparse_attn_lse(x, xp, xp, pr, idx),
        lambda: paro.block_sparse_attn_lse(xp, xp.float(), xp, pr, idx),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx[:, :1]),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx.long()),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx, counts=torch.zeros(1, 2, 3, dtype=torch.int32)),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx, out=xp),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx, lse=lse.double()),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx, status=lse),
        lambda: paro.block_sparse_attn_backward(xp, xp, xp, xp, x, lse, pr, idx),
        lambda: paro.block_sparse_attn_backward(x, xp, xp, x, x, lse, pr, idx),
        lambda: paro.block_sparse_attn_backward(x, xp, xp, xp, x, lse[:, :1], pr, idx),
        lambda: paro.block_sparse_attn_backward(x, xp, xp, xp, x, lse, pr, idx, dlse=lse.bfloat16()),
        lambda: paro.block_sparse_attn_backward(x, xp, xp, xp, x, lse, pr, idx, dk=x.float()),
        lambda: paro.block_sparse_attn_backward(x, xp, xp, xp, x, lse, pr, idx, workspace=lse),
        lambda: paro.block_sparse_query_attn(q[:, :3], xp, xp, pool, pr, 2),
        lambda: paro.block_sparse_query_attn(q[..., :32], xp, xp, pool, pr, 2),
        lambda: paro.block_sparse_query_attn(q[:, :, :0], xp, xp, pool, pr, 2),
        lambda: paro.block_sparse_query_attn(q.float(), xp, xp, pool, pr, 2),
        lambda: paro.block_sparse_query_attn(q.half(), xp.half(), xp.half(), pool, pr, 2),
        lambda: paro.block_sparse_query_attn(q, x, xp, pool, pr, 2),
        lambda: paro.block_sparse_query_attn(q, xp, xp, pool.bfloat16(), pr, 2),
        lambda: paro.block_sparse_query_attn(q, xp, xp, pool, pr, 0),
        lambda: paro.block_sparse_query_attn(q, xp, xp, pool, pr, 5),
        lambda: paro.block_sparse_query_attn(q, xp, xp, pool, pr, 2, lengths=torch.zeros(2, dtype=torch.int32)),
        lambda: paro.block_sparse_query_attn(q, xp, xp, pool, pr, 2, lengths=torch.zeros(1)),
        lambda: paro.block_sparse_query_attn(q, xp, xp, pool, pr, 2, idx=torch.zeros(1, 4, 3, 3, dtype=torch.int32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was accepted")


def test_a_problem_is_copied_and_pickled(lib):
    """Copies stand alone: their pointer is to their own order ids."""
    pr = paro.Problem(1, 3, (3, 8, 9), 64, 64, [0, 5, 9])
    paro.backward_workspace(pr)
    for other in (copy.copy(pr), copy.deepcopy(pr), pickle.loads(pickle.dumps(pr)),
                  copy.deepcopy({"problem": pr})["problem"]):
        assert other.perms_ptr.value == other._perms.ctypes.data
        assert list(ctypes.cast(other.perms_ptr, ctypes.POINTER(ctypes.c_int8))[:3]) == [0, 5, 9]
        assert bytes(other.shape) == bytes(pr.shape)
        for name in ("B", "heads", "N", "NB", "N_p", "workspace", "natural", "rows", "permuted", "pooled",
                     "square", "per_block"):
            assert getattr(other, name) == getattr(pr, name)
    del pr
    assert list(ctypes.cast(other.perms_ptr, ctypes.POINTER(ctypes.c_int8))[:3]) == [0, 5, 9]


def test_a_module_that_holds_one_is_copied(lib):
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.w = torch.nn.Parameter(torch.zeros(3))
            self.problem = paro.Problem(1, 2, (4, 8, 8), 64, 64, [1, 7])

    ema = copy.deepcopy(Layer())
    assert list(ctypes.cast(ema.problem.perms_ptr, ctypes.POINTER(ctypes.c_int8))[:2]) == [1, 7]
