"""Differentiable forms of the library's operators, for training a video
DiT: rotary positions and block-sparse attention as torch.autograd functions.

Argument handling only, as in :mod:`paro`: every forward and backward step
runs in the library's kernels on the current torch stream.  The choice of the
kept blocks is not differentiated.  A step captured into a CUDA graph needs
leaves that no eager autograd graph still holds, as everywhere in
torch.autograd: it would wait for that graph's stream, which a capture
forbids.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import paro


def _rows(t):
    """``t``, or a copy, as the library takes it with strides: rows contiguous,
    each at a multiple of 16 bytes.  (A gradient lies where autograd put it: that
    of a part of a concatenation may start anywhere, contiguous or not.)"""
    e = 16 // t.element_size()
    fine = t.stride(3) == 1 and t.data_ptr() % 16 == 0 and all(
        t.shape[i] == 1 or t.stride(i) % e == 0 for i in range(3))
    return t if fine else t.clone(memory_format=torch.contiguous_format)


def _whole(t):
    """``t``, or a copy, as the library takes it without: contiguous from a
    multiple of 16 bytes on."""
    fine = t.is_contiguous() and t.data_ptr() % 16 == 0
    return t if fine else t.clone(memory_format=torch.contiguous_format)


class _Rope3d(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rope, positions, inverse, status, grid):
        ctx.rope, ctx.inverse, ctx.status, ctx.grid = rope, inverse, status, grid
        ctx.save_for_backward(positions)
        return paro.rope3d(x, rope, positions=positions, inverse=inverse, status=status, grid=grid)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (positions,) = ctx.saved_tensors
        return paro.rope3d(_rows(g), ctx.rope, positions=positions, inverse=not ctx.inverse,
                           status=ctx.status, grid=ctx.grid), None, None, None, None, None


def rope3d(x, rope, positions=None, inverse=False, status=None, grid=None):
    """:func:`paro.rope3d`, differentiable in x."""
    return _Rope3d.apply(x, rope, positions, inverse, status, grid)


class _SparseAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, pr, idx, counts, density, rope, status):
        if rope is None:
            qp, kp = (paro.reorder(_whole(x), pr, with_pool=idx is None) for x in (q, k))
        else:
            qp, kp = (paro.rope_reorder(_rows(x), rope, pr, with_pool=idx is None) for x in (q, k))
        vp = paro.reorder(_whole(v), pr)
        if idx is None:
            (qp, q_pool), (kp, k_pool) = qp, kp
            idx = paro.select_topk(paro.score_pooled(q_pool, k_pool, pr), pr,
                                   paro.k_for_density(pr.NB, density))
        out, lse = paro.block_sparse_attn_lse(qp, kp, vp, pr, idx, counts, status=status)
        ctx.pr, ctx.rope, ctx.status = pr, rope, status
        ctx.save_for_backward(qp, kp, vp, out, lse, idx, counts)
        ctx.set_materialize_grads(False)
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dlse):
        qp, kp, vp, out, lse, idx, counts = ctx.saved_tensors
        if dout is None and dlse is None:
            return (None,) * 9
        dout = torch.zeros_like(out) if dout is None else _whole(dout)
        dlse = None if dlse is None else dlse.contiguous()
        dq, dk, dv = paro.block_sparse_attn_backward(dout, qp, kp, vp, out, lse, ctx.pr, idx, counts,
                                                     dlse=dlse, status=ctx.status)
        # (one call computes the three: what nobody asked for goes no further)
        grads = [g if need else None for g, need in zip((dq, dk, dv), ctx.needs_input_grad)]
        if ctx.rope is not None:
            grid = (ctx.pr.F, ctx.pr.H, ctx.pr.W)
            for g in grads[:2]:
                if g is not None:
                    paro.rope3d(g, ctx.rope, grid=grid, inverse=True, out=g)
        return (*grads, None, None, None, None, None, None)


def sparse_attention(q, k, v, pr, idx=None, counts=None, density=None, rope=None, status=None):
    """Block-sparse attention of bf16 q, k, v [B, heads, N, d], natural token
    order, differentiable in the three: returns (out, lse).

    ``idx`` (and ``counts``): the kept blocks of every query block, or, with
    ``density`` instead, the library's top-k of the pooled block scores.
    ``rope`` (:class:`paro.RopeTable`): q and k are rotated on the way into
    their heads' orders, and their gradients back."""
    if (idx is None) == (density is None):
        raise ValueError("give either idx or density")
    if idx is None and counts is not None:
        raise ValueError("counts go with idx")
    return _SparseAttention.apply(q, k, v, pr, idx, counts, density, rope, status)
