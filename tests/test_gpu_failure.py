"""The failure path of the tcgen05 attention kernel, driven on the GPU
without a fault: a host-set test hook (pa_test_inject_v_stall) makes the
V-tile loader of one CTA skip one kept tile, so the MMA issuer's bounded
wait for it runs out after a host-set limit of 1 ms.  The kernel must record
PA_ERR_TIMEOUT, unwind (every role leaves its loop, copies and MMAs drained,
tensor memory released), return quickly, and leave the context usable: a
normal call afterwards on the same context is checked against the oracle.
No trap, no bad address, nothing left waiting."""

import time

import numpy as np
import pytest
import torch

from block_sparse_attention_34_b200 import paro
from block_sparse_attention_34_b200.synth import as_f64
from oracle import paro_ref as ref

from helpers import compare, custom, inputs, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("permuted", [True, False], ids=["tma_tiles", "gathered_rows"])
def test_bounded_wait_runs_out_and_context_stays_usable(permuted):
    w = custom("stall_1024", 1, 2, 128, (4, 16, 16), 128, "bf16", 1.0, perms=(0, 3))
    q, k, v, perms = inputs(w)
    pr = paro.Problem(w.B, w.heads, (w.F, w.H, w.W), w.d, w.block, perms)
    qd, kd, vd = to_dev(q, k, v)
    if permuted:
        qd, kd, vd = (paro.reorder(x, pr) for x in (qd, kd, vd))
    idx = torch.arange(w.NB, dtype=torch.int32, device="cuda").expand(1, w.heads, w.NB, w.NB)
    idx = idx.contiguous()
    want = ref.attention(as_f64(q), as_f64(k), as_f64(v), (w.F, w.H, w.W), perms, w.block,
                         idx.cpu().numpy())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        out = paro.block_sparse_attn(qd, kd, vd, pr, idx, status=status, permuted=permuted)
        torch.cuda.synchronize()
        return out

    out = call()  # warm: module load, attribute set-up
    assert status.item() == 0
    compare(out, want)

    paro.test_inject_v_stall(query_block=3, batch_head=1, tile=2, wait_limit_ns=1_000_000)
    try:
        t0 = time.perf_counter()
        call()
        elapsed = time.perf_counter() - t0
    finally:
        paro.test_inject_v_stall(-1, -1, -1, 0)
    assert status.item() == paro.PA_ERR_TIMEOUT
    assert elapsed < 1.0, elapsed

    # the same context, the hook off, the status cleared: a normal call
    paro.clear_status(status)
    out = call()
    assert status.item() == 0
    compare(out, want)



@pytest.mark.parametrize("form", ["tma_tiles", "gathered_rows", "compensated", "int8", "int8_p_tile", "map"])
def test_an_expired_status_ends_the_launch(form):
    """A status word that already records PA_ERR_TIMEOUT: every kernel with
    bounded waits returns at once, writes nothing and leaves the word."""
    pr = paro.Problem(1, 3, (5, 16, 17), 128, 128, [0, 3, 5])
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn(pr.natural, generator=g, device="cuda").bfloat16()
    xp, pool = paro.reorder(x, pr, with_pool=True)
    idx = torch.arange(pr.NB, dtype=torch.int32, device="cuda").expand(pr.square).contiguous()
    status = torch.full((1,), paro.PA_ERR_TIMEOUT, dtype=torch.int32, device="cuda")
    out = torch.full(pr.natural, float("nan"), dtype=torch.bfloat16, device="cuda")
    if form == "tma_tiles":
        paro.block_sparse_attn(xp, xp, xp, pr, idx, out=out, status=status, permuted=True)
    elif form == "gathered_rows":
        paro.block_sparse_attn(x, x, x, pr, idx, out=out, status=status)
    elif form == "compensated":
        paro.block_sparse_attn_compensated(xp, xp, xp, pr, idx[..., :2].contiguous(), pool, pool, out=out,
                                           status=status, permuted=True)
    elif form == "map":
        paro.map_row_stats(xp, xp, pr, 0, status)
    else:
        x8, scale = paro.quantize_int8(x, pr)
        paro.block_sparse_attn(x8, x8, x8, pr, idx, scales=(scale,) * 3, out=out, status=status,
                               p_tile=form == "int8_p_tile")
    assert status.item() == paro.PA_ERR_TIMEOUT
    assert out.isnan().all()
