"""Host side of the launches: every entry runs on its tensors' device and on
that device's current stream, whichever device is current.  Host tensors
stand for tensors of a second device, and the library is a recorder: nothing
is dereferenced."""

import ctypes

import pytest
import torch

from block_sparse_attention_34_b200 import autograd, paro
from block_sparse_attention_34_b200.pipeline import Pipeline

BF, I32 = torch.bfloat16, torch.int32
STREAMS = {0: 7000, 1: 7001}  # the current stream of each device


class Recorder:
    """Every launch of the library, with the device that was current."""

    def __init__(self, current, real):
        self.current, self.real, self.calls = current, real, []

    def __getattr__(self, name):
        if name in ("pa_k_for_density", "pa_rope_table_floats", "pa_last_error",
                    "pa_block_sparse_attn_backward_workspace"):
            return getattr(self.real, name)

        def call(*args):
            stream = args[-1].value if isinstance(args[-1], ctypes.c_void_p) else args[-1]
            self.calls.append((name, self.current[0], stream))
            return paro.PA_OK

        return call


@pytest.fixture
def lib(monkeypatch):
    current = [0]

    class device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.before, current[0] = current[0], self.i

        def __exit__(self, *exc):
            current[0] = self.before

    recorder = Recorder(current, paro.load())
    # the tensors say that they are on device 1
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i=None: type(
        "S", (), {"cuda_stream": STREAMS[current[0] if i is None else i]}))
    monkeypatch.setattr(paro, "_current_device", lambda: current[0])
    monkeypatch.setattr(paro, "_raw_stream", lambda i: STREAMS[i])
    monkeypatch.setattr(paro, "load", lambda: recorder)
    return recorder


def on_device_1(lib, least=1):
    assert len(lib.calls) >= least
    assert {(dev, stream) for _, dev, stream in lib.calls} == {(1, STREAMS[1])}, lib.calls
    lib.calls.clear()


PR = dict(B=1, heads=2, grid=(4, 8, 16), d=128, block=128, perms=[0, 5])


def test_every_entry(lib, monkeypatch):
    monkeypatch.setattr(torch, "empty", torch.zeros)  # orders that index
    pr = paro.Problem(**PR)
    f32 = torch.float32
    x, xp = torch.zeros(pr.natural, dtype=BF), torch.zeros(pr.permuted, dtype=BF)
    x8, scale = torch.zeros(pr.permuted, dtype=torch.int8), torch.zeros(pr.per_block)
    pool, scores, rows = torch.zeros(pr.pooled), torch.zeros(pr.square), torch.zeros(pr.rows)
    idx, status = torch.zeros(pr.per_block + (2,), dtype=I32), torch.zeros(1, dtype=I32)
    rope = paro.RopeTable.__new__(paro.RopeTable)
    rope.extent, rope.d, rope.pairs, rope.interleaved = (4, 8, 16), 128, (22, 21, 21), True
    rope.desc = paro.PaRope((ctypes.c_int32 * 3)(4, 8, 16), (ctypes.c_int32 * 3)(22, 21, 21), 1)
    rope.table = torch.zeros(8)
    entries = [
        lambda: paro.clear_status(status),
        lambda: paro.reorder(x, pr, with_pool=True),
        lambda: paro.inverse_reorder(xp, pr),
        lambda: paro.block_score(x, x, pr),
        lambda: paro.score_pooled(pool, pool, pr),
        lambda: paro.select_topk(scores, pr, 2),
        lambda: paro.compact_mask(torch.zeros(pr.per_block + (1,), dtype=I32), pr),
        lambda: paro.select_hybrid(scores, pr, 2, 0.5, 1),
        lambda: paro.sics_scores(x, x, pr),
        lambda: paro.map_row_stats(xp, xp, pr, 0, status),
        lambda: paro.map_block_stats(xp, xp, pr, 0, rows, rows, status=status),
        lambda: paro.paro_offline(x, x, (4, 8, 16), 128),
        lambda: paro.quantize_int8(x, pr, with_pool=True),
        lambda: paro.quantize_int8(x, pr, bits=4),
        lambda: paro.block_sparse_attn(x, x, x, pr, idx, status=status),
        lambda: paro.block_sparse_attn(x, x, x, pr, idx, baseline=True),
        lambda: paro.block_sparse_attn(x8, x8, x8, pr, idx, scales=(scale,) * 3),
        lambda: paro.block_sparse_attn_compensated(xp, xp, xp, pr, idx, pool, pool, permuted=True),
        lambda: paro.round_bf16(pool),
        lambda: paro.rope3d(x, rope),
        lambda: paro.rope_reorder(x, rope, pr, with_pool=True),
        lambda: paro.block_sparse_attn_lse(xp, xp, xp, pr, idx),
        lambda: paro.block_sparse_attn_backward(x, xp, xp, xp, x, rows, pr, idx),
        lambda: paro.block_sparse_query_attn(x[:, :, :1].contiguous(), xp, xp, pool, pr, 2),
    ]
    for entry in entries:
        entry()
        on_device_1(lib)


@pytest.mark.parametrize("kw", [{}, {"int8": True}, {"baseline": True}, {"compensate": True},
                                {"permuted": False}, {"selection": "hybrid", "top_p": 0.4}])
def test_whole_calls(lib, kw):
    pr = paro.Problem(**PR)
    x = torch.zeros(pr.natural, dtype=BF)
    paro.attention(x, x, x, PR["grid"], PR["perms"], 128, 0.5, **kw)
    on_device_1(lib, 3)
    if "compensate" not in kw and "permuted" not in kw:
        pipe = Pipeline(1, 2, PR["grid"], 128, 128, PR["perms"], 0.5, device="cpu", **kw)
        pipe.run(x, x, x)
        on_device_1(lib, 4)


def test_a_training_step(lib):
    pr = paro.Problem(**PR)
    leaves = [torch.zeros(pr.natural, dtype=BF).requires_grad_() for _ in range(3)]
    out, _ = autograd.sparse_attention(*leaves, pr, density=0.5)
    out.sum().backward()
    on_device_1(lib, 7)
