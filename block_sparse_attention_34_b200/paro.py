"""Thin Python binding of libparo (include/paro.h).

Argument marshalling only: every step runs in the library's CUDA kernels on
the current torch stream of its tensors' device, whichever device is current.
Torch supplies device memory and streams.  There is no CPU fallback: if the
library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import functools
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libparo.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_TIMEOUT, PA_ERR_DEVICE_CHECK = range(6)
ABI_VERSION = 8  # the pa_abi_version() these signatures describe
PA_F32, PA_BF16, PA_I8 = 0, 1, 2
PA_ATTN_PERMUTED = 1
PA_ATTN_P4 = 2  # with int8 inputs: 4-bit P codes (INT4 PV)
PA_ROPE_INVERSE = 1  # pa_rope_apply: the transposed rotation
PA_ATTN_P_TILE = 4  # with int8 inputs: normalised P, one scale per tile (two passes)
STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_CUDA",
                4: "PA_ERR_TIMEOUT", 5: "PA_ERR_DEVICE_CHECK"}
ORDER_IDS = {"FHW": 0, "FWH": 1, "HFW": 2, "HWF": 3, "WFH": 4, "WHF": 5}
# ids 6-11: 3D tile blockings (tf, th, tw) of the block size (include/paro.h)
TILE_IDS = {128: {"T1x8x16": 6, "T1x16x8": 7, "T2x8x8": 8, "T4x4x8": 9, "T8x4x4": 10,
                  "T16x2x4": 11},
            64: {"T1x8x8": 6, "T1x4x16": 7, "T2x4x8": 8, "T4x4x4": 9, "T8x2x4": 10,
                 "T16x2x2": 11}}
N_ORDERS = 12


class PaShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "heads", "F", "H", "W", "d", "block")]


class PaRope(ctypes.Structure):
    _fields_ = [("extent", ctypes.c_int32 * 3), ("pairs", ctypes.c_int32 * 3),
                ("interleaved", ctypes.c_int32)]


class ParoError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int32


def load():
    """Load libparo.so (built by ``python -m block_sparse_attention_34_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m block_sparse_attention_34_b200.build` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "pa_abi_version": ([], _I),
        "pa_last_error": ([], ctypes.c_char_p),
        "pa_clear_status": ([_P, _P], _I),
        "pa_test_inject_v_stall": ([_I, _I, _I, ctypes.c_uint64], _I),
        "pa_num_blocks": ([PaShape], _I),
        "pa_k_for_density": ([_I, ctypes.c_double], _I),
        "pa_reorder": ([_P, _P, _I, PaShape, _P, _P, _P], _I),
        "pa_inverse_reorder": ([_P, _P, _I, PaShape, _P, _P], _I),
        "pa_block_score": ([_P, _P, _I, PaShape, _P, _P, _P, _P, _P], _I),
        "pa_score_pooled": ([_P, _P, PaShape, _P, _P], _I),
        "pa_select_topk": ([_P, PaShape, _I, _P, _P], _I),
        "pa_compact_mask": ([_P, PaShape, _P, _P, _P], _I),
        "pa_select_hybrid": ([_P, PaShape, _I, ctypes.c_double, _I, _P, _P, _P], _I),
        "pa_sics_scores": ([_P, _P, _I, PaShape, _P, _P, _P], _I),
        "pa_map_row_stats": ([_P, _P, PaShape, _I, _P, _P, _P, _P], _I),
        "pa_map_block_stats": ([_P, _P, PaShape, _I, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P,
                                _P], _I),
        "pa_paro_metric": ([_P, _P, _P, PaShape, _I, ctypes.c_float, _P, _P, _P], _I),
        "pa_paro_choose": ([_P, _P, PaShape, ctypes.c_float, _P, _P, _P], _I),
        "pa_quantize_int8": ([_P, _I, PaShape, _P, _P, _P, _P, _P], _I),
        "pa_quantize_int4": ([_P, _I, PaShape, _P, _P, _P, _P, _P], _I),
        "pa_block_sparse_attn": ([_P, _P, _P, _I, ctypes.c_uint32, PaShape, _P, _P, _P, _I, _P, _P, _P,
                                  _P, _P, _P], _I),
        "pa_block_sparse_attn_mma": ([_P, _P, _P, _I, ctypes.c_uint32, PaShape, _P, _P, _P, _I, _P, _P,
                                      _P], _I),
        "pa_block_sparse_attn_compensated": ([_P, _P, _P, _I, ctypes.c_uint32, PaShape, _P, _P, _P, _I,
                                              _P, _P, _I, _P, _P, _P], _I),
        "pa_round_bf16": ([_P, _P, ctypes.c_int64, _P], _I),
        "pa_rope_table_floats": ([PaRope], ctypes.c_int64),
        "pa_rope_table": ([PaRope, ctypes.c_double, _P, _P, _P, _P], _I),
        "pa_rope_apply": ([_P, _P, _P, _P, _I, PaShape, PaRope, _P, _P, _I, ctypes.c_uint32, _P,
                           _P], _I),
        "pa_rope_reorder": ([_P, _P, _P, _I, PaShape, _P, PaRope, _P, _P, _P], _I),
        "pa_block_sparse_attn_lse": ([_P, _P, _P, _I, PaShape, _P, _P, _P, _I, _P, _P, _P, _P], _I),
        "pa_block_sparse_attn_backward_workspace": ([PaShape], ctypes.c_int64),
        "pa_block_sparse_attn_backward": ([_P] * 7 + [_I, PaShape, _P, _P, _P, _I, _P, _P, _P, _P,
                                                      ctypes.c_int64, _P, _P], _I),
        "pa_query_attn": ([_P, _P, _P, _P, _I, PaShape, _I, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    }
    lib.pa_abi_version.restype = _I
    if lib.pa_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{LIB_PATH} has ABI version {lib.pa_abi_version()}, this binding "
                           f"needs {ABI_VERSION}: rebuild it with "
                           "`python -m block_sparse_attention_34_b200.build`")
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int):
    if status != PA_OK:
        raise ParoError(status, load().pa_last_error().decode())


def _addr(t):
    return None if t is None else t.data_ptr()


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream():
    """The current stream of the current device."""
    return _raw_stream(_current_device())


def _launch(t, fn, *args):
    """fn(*args, stream) on the device of ``t`` and that device's current
    stream, as torch's own operators run: the one way every entry launches, so
    that the steps of a call stay in order whichever device is current."""
    i = t.get_device()
    if i < 0 or i == _current_device():  # (host tensors end at every entry's checks)
        status = fn(*args, _stream())
    else:
        with torch.cuda.device(i):
            status = fn(*args, _stream())
    _check(status)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return PA_F32
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.int8:
        return PA_I8
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need_cuda(*ts):
    dev = None
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i < 0:
                raise ValueError("tensors must be on a CUDA device (no CPU path)")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            if dev is None:
                dev = i
            elif i != dev:
                raise ValueError(f"tensors on different devices (cuda:{dev} and cuda:{i})")


_FLOAT = (torch.float32, torch.bfloat16)


def _expect(t, name, shape, dtypes):
    """Raise ValueError unless tensor ``t`` has exactly ``shape`` and one of
    ``dtypes``: the library reads and writes whole buffers of the sizes the
    shape implies, so a smaller buffer must never reach it."""
    if t is None:
        return
    if t.shape != shape and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if isinstance(dtypes, torch.dtype):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")


def _same_dtype(*named):
    ts = [(n, t) for n, t in named if t is not None]
    for n, t in ts[1:]:
        if t.dtype != ts[0][1].dtype:
            raise ValueError(f"{n}: dtype {t.dtype} differs from {ts[0][0]}'s {ts[0][1].dtype}")


class Problem:
    """Sizes of one attention call plus the per-head order ids."""

    def __init__(self, B, heads, grid, d, block, perms):
        self.B, self.heads, self.d, self.block = int(B), int(heads), int(d), int(block)
        self.F, self.H, self.W = (int(x) for x in grid)
        self.N = self.F * self.H * self.W
        self.NB = -(-self.N // self.block)
        self.N_p = self.NB * self.block
        p = np.asarray(perms, dtype=np.int8)
        if p.shape != (self.heads,):
            raise ValueError(f"perms must have one order id per head ({self.heads})")
        self._perms = np.ascontiguousarray(p)
        self.shape = PaShape(self.B, self.heads, self.F, self.H, self.W, self.d, self.block)
        self.perms_ptr = self._perms.ctypes.data_as(ctypes.c_void_p)
        self.workspace = None  # bytes of the backward pass's workspace, once asked for
        # tensor shapes of the call
        self.natural = (self.B, self.heads, self.N, self.d)
        self.rows = (self.B, self.heads, self.N)
        self.permuted = (self.B, self.heads, self.N_p, self.d)
        self.pooled = (self.B, self.heads, self.NB, self.d)
        self.square = (self.B, self.heads, self.NB, self.NB)
        self.per_block = (self.B, self.heads, self.NB)

    # a copy or a pickle carries the order ids, and points to its own
    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "perms_ptr"}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._perms = np.ascontiguousarray(self._perms)
        self.perms_ptr = self._perms.ctypes.data_as(ctypes.c_void_p)

    @classmethod
    def from_qkv(cls, q, grid, perms, block):
        B, h, N, d = q.shape
        return cls(B, h, grid, d, block, perms)


def clear_status(status):
    """Enqueue status[0] = PA_OK on the current stream (a memset)."""
    _need_cuda(status)
    _expect_status(status)
    _launch(status, load().pa_clear_status, _addr(status))


def test_inject_v_stall(query_block: int, batch_head: int, tile: int, wait_limit_ns: int):
    """Failure-path test hook (pa_test_inject_v_stall): the V loader of one
    CTA of the tcgen05 bf16 kernel skips one kept tile, so a bounded wait
    runs out after ``wait_limit_ns``; ``tile < 0`` switches it off."""
    _check(load().pa_test_inject_v_stall(int(query_block), int(batch_head), int(tile),
                                         int(wait_limit_ns)))


def k_for_density(nb: int, density: float) -> int:
    return int(load().pa_k_for_density(int(nb), float(density)))


def reorder(x, pr: Problem, out=None, pool=None, with_pool=False):
    """Permuted copy [B, heads, N_p, d] of natural-order x; with
    ``with_pool`` (or a given ``pool`` buffer) also the block means, from
    the same read: returns (x_perm, pool)."""
    _need_cuda(x, out, pool)
    if x.shape != pr.natural or x.dtype not in _FLOAT:
        raise ValueError(f"x: {tuple(x.shape)} {x.dtype}, expected {pr.natural} and one of {_FLOAT}")
    _expect(out, "out", pr.permuted, x.dtype)
    _expect(pool, "pool", pr.pooled, torch.float32)
    out = out if out is not None else x.new_empty(pr.permuted)
    if with_pool and pool is None:
        pool = x.new_empty(pr.pooled, dtype=torch.float32)
    _launch(x, load().pa_reorder, x.data_ptr(), out.data_ptr(), _dtype_code(x), pr.shape,
            pr.perms_ptr, _addr(pool))
    return (out, pool) if (with_pool or pool is not None) else out


def inverse_reorder(xp, pr: Problem, out=None):
    _need_cuda(xp, out)
    _expect(xp, "xp", pr.permuted, _FLOAT)
    _expect(out, "out", pr.natural, xp.dtype)
    out = out if out is not None else torch.empty((pr.B, pr.heads, pr.N, pr.d), dtype=xp.dtype,
                                                  device=xp.device)
    _launch(xp, load().pa_inverse_reorder, _addr(xp), _addr(out), _dtype_code(xp), pr.shape, pr.perms_ptr)
    return out


def block_score(q, k, pr: Problem, q_pool=None, k_pool=None, scores=None):
    _need_cuda(q, k, q_pool, k_pool, scores)
    _expect(q, "q", pr.natural, _FLOAT)
    _expect(k, "k", pr.natural, q.dtype)
    _expect(q_pool, "q_pool", pr.pooled, torch.float32)
    _expect(k_pool, "k_pool", pr.pooled, torch.float32)
    _expect(scores, "scores", pr.square, torch.float32)
    dev = q.device
    q_pool = q_pool if q_pool is not None else torch.empty((pr.B, pr.heads, pr.NB, pr.d), dtype=torch.float32, device=dev)
    k_pool = k_pool if k_pool is not None else torch.empty_like(q_pool)
    scores = scores if scores is not None else torch.empty((pr.B, pr.heads, pr.NB, pr.NB), dtype=torch.float32, device=dev)
    _launch(q, load().pa_block_score, _addr(q), _addr(k), _dtype_code(q), pr.shape, pr.perms_ptr,
            _addr(q_pool), _addr(k_pool), _addr(scores))
    return q_pool, k_pool, scores


def score_pooled(q_pool, k_pool, pr: Problem, scores=None):
    _need_cuda(q_pool, k_pool, scores)
    _expect(q_pool, "q_pool", pr.pooled, torch.float32)
    _expect(k_pool, "k_pool", pr.pooled, torch.float32)
    _expect(scores, "scores", pr.square, torch.float32)
    scores = scores if scores is not None else torch.empty((pr.B, pr.heads, pr.NB, pr.NB), dtype=torch.float32, device=q_pool.device)
    _launch(q_pool, load().pa_score_pooled, _addr(q_pool), _addr(k_pool), pr.shape, _addr(scores))
    return scores


def select_topk(scores, pr: Problem, k: int, idx=None):
    _need_cuda(scores, idx)
    _expect(scores, "scores", pr.square, torch.float32)
    _expect(idx, "idx", pr.per_block + (int(k),), torch.int32)
    idx = idx if idx is not None else torch.empty((pr.B, pr.heads, pr.NB, k), dtype=torch.int32, device=scores.device)
    _launch(scores, load().pa_select_topk, _addr(scores), pr.shape, int(k), _addr(idx))
    return idx


def compact_mask(bitmask, pr: Problem, idx=None, counts=None):
    _need_cuda(bitmask, idx, counts)
    _expect(bitmask, "bitmask", pr.per_block + (-(-pr.NB // 32),), (torch.int32, torch.uint32))
    _expect(idx, "idx", pr.square, torch.int32)
    _expect(counts, "counts", pr.per_block, torch.int32)
    dev = bitmask.device
    idx = idx if idx is not None else torch.empty((pr.B, pr.heads, pr.NB, pr.NB), dtype=torch.int32, device=dev)
    counts = counts if counts is not None else torch.empty((pr.B, pr.heads, pr.NB), dtype=torch.int32, device=dev)
    _launch(bitmask, load().pa_compact_mask, _addr(bitmask), pr.shape, _addr(idx), _addr(counts))
    return idx, counts


def select_hybrid(scores, pr: Problem, k: int, top_p: float, window: int, idx=None, counts=None):
    """Union of the diagonal, a local window, Top-K and Top-P per query-block
    row -> (idx [B,h,NB,NB] ascending, -1 padded; counts [B,h,NB])."""
    _need_cuda(scores, idx, counts)
    _expect(scores, "scores", pr.square, torch.float32)
    _expect(idx, "idx", pr.square, torch.int32)
    _expect(counts, "counts", pr.per_block, torch.int32)
    dev = scores.device
    idx = idx if idx is not None else torch.empty((pr.B, pr.heads, pr.NB, pr.NB), dtype=torch.int32, device=dev)
    counts = counts if counts is not None else torch.empty((pr.B, pr.heads, pr.NB), dtype=torch.int32, device=dev)
    _launch(scores, load().pa_select_hybrid, _addr(scores), pr.shape, int(k), float(top_p), int(window),
            _addr(idx), _addr(counts))
    return idx, counts


def sics_scores(q, k, pr: Problem, scores=None, orders=None):
    """Blocking scores of the 12 candidates (six axis orders, six 3D tile
    blockings): SICS of q's and k's blocks -> (scores [B,h,12], orders
    [heads] int8, each head's pick by the library: the largest score summed
    over the batch, ties to the lower id)."""
    _need_cuda(q, k, scores, orders)
    _expect(q, "q", pr.natural, _FLOAT)
    _expect(k, "k", pr.natural, q.dtype)
    _expect(scores, "scores", (pr.B, pr.heads, N_ORDERS), torch.float32)
    _expect(orders, "orders", (pr.heads,), torch.int8)
    scores = scores if scores is not None else torch.empty((pr.B, pr.heads, N_ORDERS), dtype=torch.float32, device=q.device)
    orders = orders if orders is not None else torch.empty((pr.heads,), dtype=torch.int8, device=q.device)
    _launch(q, load().pa_sics_scores, _addr(q), _addr(k), _dtype_code(q), pr.shape, _addr(scores),
            _addr(orders))
    return scores, orders


def map_row_stats(q_perm, k_perm, pr: Problem, order: int, status=None):
    """Row softmax (log2 max, sum) of every token of the dense map, from
    copies of q, k permuted by ``order`` -> ([B,h,N], [B,h,N])."""
    _need_cuda(q_perm, k_perm, status)
    _expect_status(status)
    _expect(q_perm, "q_perm", pr.permuted, torch.bfloat16)
    _expect(k_perm, "k_perm", pr.permuted, torch.bfloat16)
    dev = q_perm.device
    m = torch.empty((pr.B, pr.heads, pr.N), dtype=torch.float32, device=dev)
    l = torch.empty_like(m)
    _launch(q_perm, load().pa_map_row_stats, _addr(q_perm), _addr(k_perm), pr.shape, int(order), _addr(m),
            _addr(l), _addr(status))
    return m, l


def map_block_stats(q_perm, k_perm, pr: Problem, order: int, row_max, row_sum, eps=1e-3,
                    with_log=True, status=None):
    """Per block of the map in ``order``: dict of [B,h,NB,NB] count / total
    / peak (and log_total)."""
    _need_cuda(q_perm, k_perm, row_max, row_sum, status)
    _expect_status(status)
    _expect(q_perm, "q_perm", pr.permuted, torch.bfloat16)
    _expect(k_perm, "k_perm", pr.permuted, torch.bfloat16)
    _expect(row_max, "row_max", (pr.B, pr.heads, pr.N), torch.float32)
    _expect(row_sum, "row_sum", (pr.B, pr.heads, pr.N), torch.float32)
    dev = q_perm.device
    out = {key: torch.empty((pr.B, pr.heads, pr.NB, pr.NB), dtype=torch.float32, device=dev)
           for key in ("count", "total", "peak")}
    out["log_total"] = torch.empty_like(out["total"]) if with_log else None
    _launch(q_perm, load().pa_map_block_stats, _addr(q_perm), _addr(k_perm), pr.shape, int(order),
            _addr(row_max), _addr(row_sum), float(eps), _addr(out["count"]), _addr(out["total"]),
            _addr(out["peak"]), _addr(out["log_total"]), _addr(status))
    return out


def paro_offline(q, k, grid, block, eps=1e-3, rho=0.9, alpha=0.5, sigma=0.9, status=None):
    """PAROAttention's offline stage for natural-order q, k (bf16, d = 128,
    block = 128): the six orders' block statistics of the dense map, the
    per-head metric and order, and the static mask of each head's chosen
    order by block-sum thresholding at ``sigma``.  Returns a dict: orders
    [B,h] int8, metric / sparse_frac / incoherence [B,h,6], idx [B,h,NB,NB]
    and counts [B,h,NB] (the chosen order's mask, per head)."""
    B, heads = q.shape[:2]
    dev = q.device
    probs = [Problem(B, heads, grid, q.shape[-1], block, [o] * heads) for o in range(6)]
    pr0 = probs[0]
    sf = torch.empty((B, heads, 6), dtype=torch.float32, device=dev)
    inc = torch.empty_like(sf)
    idx_all = torch.empty((6, B, heads, pr0.NB, pr0.NB), dtype=torch.int32, device=dev)
    cnt_all = torch.empty((6, B, heads, pr0.NB), dtype=torch.int32, device=dev)
    row_max = row_sum = None
    for o, pr in enumerate(probs):
        qp, kp = reorder(q, pr), reorder(k, pr)
        if row_max is None:
            row_max, row_sum = map_row_stats(qp, kp, pr, o, status)
        st = map_block_stats(qp, kp, pr, o, row_max, row_sum, eps, True, status)
        _launch(sf, load().pa_paro_metric, _addr(st["count"]), _addr(st["total"]), _addr(st["peak"]),
                pr.shape, o, float(rho), _addr(sf), _addr(inc))
        select_hybrid(st["log_total"], pr, 0, sigma, -1, idx_all[o], cnt_all[o])
        del qp, kp, st
    metric = torch.empty_like(sf)
    orders = torch.empty((B, heads), dtype=torch.int8, device=dev)
    _launch(sf, load().pa_paro_choose, _addr(sf), _addr(inc), pr0.shape, float(alpha), _addr(metric),
            _addr(orders))
    # each head's mask in its chosen order (a gather of the six candidates)
    pick = orders.long()
    bi = torch.arange(B, device=dev)[:, None]
    hi = torch.arange(heads, device=dev)[None, :]
    return {"orders": orders, "metric": metric, "sparse_frac": sf, "incoherence": inc,
            "idx": idx_all[pick, bi, hi], "counts": cnt_all[pick, bi, hi]}


def quantize_int8(x, pr: Problem, with_pool=False, x_q=None, scales=None, pool=None, bits=8):
    """Per-block symmetric quantisation in the permuted order: 8-bit codes
    (levels +-127), or ``bits=4`` (levels +-7, one code per byte)."""
    _need_cuda(x, x_q, scales, pool)
    _expect(x, "x", pr.natural, _FLOAT)
    _expect(x_q, "x_q", pr.permuted, torch.int8)
    _expect(scales, "scales", pr.per_block, torch.float32)
    _expect(pool, "pool", pr.pooled, torch.float32)
    dev = x.device
    x_q = x_q if x_q is not None else torch.empty((pr.B, pr.heads, pr.N_p, pr.d), dtype=torch.int8, device=dev)
    scales = scales if scales is not None else torch.empty((pr.B, pr.heads, pr.NB), dtype=torch.float32, device=dev)
    if with_pool and pool is None:
        pool = torch.empty((pr.B, pr.heads, pr.NB, pr.d), dtype=torch.float32, device=dev)
    if bits not in (4, 8):
        raise ValueError(f"bits={bits}: 4 or 8")
    fn = load().pa_quantize_int8 if bits == 8 else load().pa_quantize_int4
    _launch(x, fn, _addr(x), _dtype_code(x), pr.shape, pr.perms_ptr, _addr(x_q), _addr(scales),
            _addr(pool))
    return (x_q, scales, pool) if with_pool else (x_q, scales)


def _check_lists(idx, counts, pr: Problem):
    """idx [B,h,NB,k_max] int32 with 0 <= k_max <= NB; counts [B,h,NB] int32."""
    if idx is None:
        raise ValueError("idx is required")
    if idx.dim() != 4 or tuple(idx.shape[:3]) != pr.per_block or idx.shape[3] > pr.NB:
        raise ValueError(f"idx: shape {tuple(idx.shape)}, expected {pr.per_block + ('k<=NB',)}")
    _expect(idx, "idx", tuple(idx.shape), torch.int32)
    _expect(counts, "counts", pr.per_block, torch.int32)


def _expect_status(status):
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status: an int32 tensor of at least one element")


def block_sparse_attn(q, k, v, pr: Problem, idx, counts=None, scales=None, out=None,
                      status=None, baseline=False, permuted=False, p4=False, p_tile=False):
    """O = block-sparse attention over the kept tiles, natural token order.

    ``permuted``: q, k, v are [B, heads, N_p, d] from :func:`reorder`.
    ``scales`` = (q_scale, k_scale, v_scale) for int8 q/k/v from
    :func:`quantize_int8` (output bf16); with them ``p4`` quantises P to 4
    bits and ``p_tile`` quantises the normalised P with one scale per tile
    (two passes over the kept tiles) instead of the one-pass fixed scale.
    ``baseline=True`` runs the mma.sync comparison kernel instead of the
    tcgen05 one."""
    _need_cuda(q, k, v, idx, counts, out, status, *(scales or ()))
    code = _dtype_code(q)
    _same_dtype(("q", q), ("k", k), ("v", v))
    rows = pr.permuted if (permuted or code == PA_I8) else pr.natural
    for name, t in (("q", q), ("k", k), ("v", v)):
        _expect(t, name, rows, (torch.float32, torch.bfloat16, torch.int8))
    _check_lists(idx, counts, pr)
    if code == PA_I8:
        if scales is None or len(scales) != 3:
            raise ValueError("int8 q, k, v need scales=(q_scale, k_scale, v_scale)")
        for name, t in zip(("q_scale", "k_scale", "v_scale"), scales):
            _expect(t, name, pr.per_block, torch.float32)
    out_dtype = torch.bfloat16 if code == PA_I8 else q.dtype
    _expect(out, "out", pr.natural, out_dtype)
    _expect_status(status)
    out = out if out is not None else torch.empty((pr.B, pr.heads, pr.N, pr.d), dtype=out_dtype, device=q.device)
    k_max = int(idx.shape[-1])
    flags = ((PA_ATTN_PERMUTED if permuted else 0) | (PA_ATTN_P4 if p4 else 0)
             | (PA_ATTN_P_TILE if p_tile else 0))
    if baseline:
        _launch(q, load().pa_block_sparse_attn_mma, _addr(q), _addr(k), _addr(v), code, flags,
                pr.shape, pr.perms_ptr, _addr(idx), _addr(counts), k_max, _addr(out), _addr(status))
    else:
        qs, ks, vs = scales if scales is not None else (None, None, None)
        _launch(q, load().pa_block_sparse_attn, _addr(q), _addr(k), _addr(v), code, flags, pr.shape,
                pr.perms_ptr, _addr(idx), _addr(counts), k_max, _addr(qs), _addr(ks), _addr(vs),
                _addr(out), _addr(status))
    return out


def block_sparse_attn_compensated(q, k, v, pr: Problem, idx, k_pool, v_pool, counts=None,
                                  out=None, status=None, permuted=False):
    """Block-sparse attention in which every unselected key block still
    enters the softmax as one pooled key row (mean key, mean value, weight
    = its valid keys): PASA's grouped first-order compensation.  k_pool,
    v_pool [B, heads, NB, d] block means (from :func:`reorder` with
    ``with_pool`` or :func:`block_score`), both float32, or both bfloat16
    (:func:`round_bf16`; bf16 q, k, v with d = block = 128 only, the faster
    form).  bf16 or fp32 q, k, v; output natural order, q's dtype."""
    _need_cuda(q, k, v, idx, counts, k_pool, v_pool, out, status)
    _same_dtype(("q", q), ("k", k), ("v", v))
    rows = pr.permuted if permuted else pr.natural
    for name, t in (("q", q), ("k", k), ("v", v)):
        _expect(t, name, rows, _FLOAT)
    _check_lists(idx, counts, pr)
    pool_dt = k_pool.dtype if k_pool is not None else torch.float32
    if pool_dt not in (torch.float32, torch.bfloat16):
        raise ValueError(f"k_pool dtype {pool_dt}: float32 or bfloat16")
    _expect(k_pool, "k_pool", pr.pooled, pool_dt)
    _expect(v_pool, "v_pool", pr.pooled, pool_dt)
    _expect(out, "out", pr.natural, q.dtype)
    _expect_status(status)
    out = out if out is not None else torch.empty((pr.B, pr.heads, pr.N, pr.d), dtype=q.dtype,
                                                  device=q.device)
    _launch(q, load().pa_block_sparse_attn_compensated, _addr(q), _addr(k), _addr(v),
            _dtype_code(q), PA_ATTN_PERMUTED if permuted else 0, pr.shape, pr.perms_ptr, _addr(idx),
            _addr(counts), int(idx.shape[-1]), _addr(k_pool), _addr(v_pool), _dtype_code(k_pool),
            _addr(out), _addr(status))
    return out


def round_bf16(x, out=None):
    """x (float32, CUDA, contiguous) rounded to bfloat16 by the library's
    kernel: the bf16 block means :func:`block_sparse_attn_compensated`
    loads with the K and V tiles' copy engine."""
    _need_cuda(x, out)
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    elif out.dtype != torch.bfloat16 or out.shape != x.shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bfloat16 tensor of shape {tuple(x.shape)}")
    _launch(x, load().pa_round_bf16, _addr(x), _addr(out), x.numel())
    return out


def _device_of(t):
    i = t.get_device()
    if i < 0:
        raise ValueError("tensors must be on a CUDA device (no CPU path)")
    return i


def _need(i, name, t, shape, dtype):
    """Raise ValueError unless ``t`` is contiguous, on device ``i``, and of
    that shape and type: the library reads and writes whole buffers of the
    sizes the problem implies."""
    if t.get_device() == i and t.shape == shape and t.dtype == dtype and t.is_contiguous():
        return
    if t.get_device() != i:
        raise ValueError(f"{name}: on {t.device}, expected device {i}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype}, expected {tuple(shape)} {dtype}")


def _need_status(i, status):
    if status is not None:
        _need(i, "status", status, status.shape, torch.int32)
        _expect_status(status)


def _need_lists(i, idx, counts, pr):
    """idx [B,h,NB,k_max] int32 with 0 <= k_max <= NB; counts [B,h,NB] int32."""
    if idx.dim() != 4 or idx.shape[3] > pr.NB:
        raise ValueError(f"idx: shape {tuple(idx.shape)}, expected {pr.per_block + ('k<=NB',)}")
    _need(i, "idx", idx, pr.per_block + (idx.shape[3],), torch.int32)
    if counts is not None:
        _need(i, "counts", counts, pr.per_block, torch.int32)


@functools.lru_cache(maxsize=256)
def _row_shape(B, heads, F, H, W, d):
    return PaShape(B, heads, F, H, W, d, 64)


class RopeTable:
    """Rotary positions with three axes (time, height, width): the cosines
    and sines of every coordinate of ``extent`` = (frames, height, width),
    made once, on the device and its current stream, and kept by the caller.

    ``pairs``: how many of the head dimension's d/2 pairs turn with each axis,
    in that order (the rest stay); default: a third of them each to height
    and width, the rest to time.  Pair i of axis a turns by
    ``(first[a] + step[a] * position) * theta ** (-i / pairs[a])``; ``first``
    places a clip that continues another one, ``step`` stretches an axis.
    ``interleaved``: pair p is elements (2p, 2p + 1), else (p, p + d/2)."""

    def __init__(self, extent, d, pairs=None, theta=10000.0, first=(0.0, 0.0, 0.0),
                 step=(1.0, 1.0, 1.0), interleaved=True, device="cuda"):
        self.extent = tuple(int(x) for x in extent)
        self.d = int(d)
        if pairs is None:
            third = self.d // 6
            pairs = (self.d // 2 - 2 * third, third, third)
        self.pairs = tuple(int(x) for x in pairs)
        self.interleaved = bool(interleaved)
        if not len(self.extent) == len(self.pairs) == len(first) == len(step) == 3:
            raise ValueError("extent, pairs, first and step have one value per axis (3)")
        if any(not 1 <= x < 1 << 31 for x in self.extent) or any(not 0 <= x <= 64 for x in self.pairs):
            raise ValueError(f"extent {self.extent}, pairs {self.pairs}: extents >= 1, pairs 0 .. 64")
        self.desc = PaRope((ctypes.c_int32 * 3)(*self.extent), (ctypes.c_int32 * 3)(*self.pairs),
                           int(self.interleaved))
        lib = load()
        n = lib.pa_rope_table_floats(self.desc)
        if n < 0 or sum(self.pairs) > self.d // 2:
            raise ValueError(f"extent {self.extent}, pairs {self.pairs}: malformed for d = {self.d}")
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError("tensors must be on a CUDA device (no CPU path)")
        self.table = torch.empty(n, dtype=torch.float32, device=dev)
        three = ctypes.c_double * 3
        _launch(self.table, lib.pa_rope_table, self.desc, float(theta), three(*map(float, first)),
                three(*map(float, step)), _addr(self.table))


def _row_strides(t, name):
    """Element strides (batch, head, token) of a [B, heads, N, d] tensor with
    contiguous rows, as the library takes them (None: contiguous)."""
    if t.data_ptr() % 16 == 0 and t.is_contiguous():
        return None
    if t.stride(3) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    e = 16 // t.element_size()
    # the stride of a dimension of one element says nothing
    s = [0 if t.shape[i] == 1 else t.stride(i) for i in range(3)]
    if any(x % e for x in s) or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows must start at multiples of 16 bytes (strides {t.stride()})")
    return (ctypes.c_int64 * 3)(*s)


def _rope_checks(x, rope, d):
    i = _device_of(x)
    if x.dim() != 4 or x.dtype not in _FLOAT or x.numel() == 0:
        raise ValueError(f"x: [B, heads, N, d] of float32 or bfloat16, got {tuple(x.shape)} {x.dtype}")
    if rope.d != d or x.shape[3] != d or rope.table.get_device() != i:
        raise ValueError(f"rope: a table for d = {rope.d} on {rope.table.device}, x has d = {x.shape[3]} "
                         f"on {x.device}")
    return i


def _dense_rows(t):
    """Whether no two elements of ``t`` share memory (dimensions sorted by
    stride each step over the whole of the smaller ones)."""
    at = 1
    for stride, n in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < at:
            return False
        at = stride * (n - 1) + at
    return True


def rope3d(x, rope: RopeTable, positions=None, inverse=False, out=None, status=None, grid=None):
    """Rotary positions with three axes of x [B, heads, N, d].

    Rows must be contiguous and start at multiples of 16 bytes; batch, head
    and token strides are free, so the projection's [B, N, heads, d] goes in
    as ``.transpose(1, 2)``.  Token n sits at its place in ``grid`` (frames,
    height, width; by default ``rope.extent``, which has to cover it), or at
    ``positions`` (int32 [N, 3] or [B, N, 3], contiguous; a coordinate
    outside the table is reported on ``status`` and its rows stay unwritten).
    ``inverse`` turns back: the gradient's rotation.  ``out``: any non-overlapping strides, or
    x itself (not a tensor that shares only part of x's memory); contiguous
    by default."""
    i = _rope_checks(x, rope, rope.d)
    B, heads, N, d = x.shape
    if positions is None:
        F, H, W = rope.extent if grid is None else grid
        if F * H * W != N:
            raise ValueError(f"x has {N} tokens, the grid {(F, H, W)}: give grid or positions")
        batched = 0
    else:
        if grid is not None:
            raise ValueError("grid or positions, not both")
        F, H, W = 1, 1, N
        batched = int(positions.dim() == 3)
        _need(i, "positions", positions, (B, N, 3) if batched else (N, 3), torch.int32)
    _need_status(i, status)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        out_strides = None
    else:
        _expect(out, "out", x.shape, x.dtype)
        if out.get_device() != i:
            raise ValueError(f"out: on {out.device}, x is on {x.device}")
        if not (out.is_contiguous() or _dense_rows(out)):
            raise ValueError("out: rows overlap")
        out_strides = _row_strides(out, "out")
    _launch(x, load().pa_rope_apply, x.data_ptr(), _row_strides(x, "x"), out.data_ptr(), out_strides,
            _dtype_code(x), _row_shape(B, heads, F, H, W, d), rope.desc, rope.table.data_ptr(),
            _addr(positions), batched, PA_ROPE_INVERSE if inverse else 0, _addr(status))
    return out


def rope_reorder(x, rope: RopeTable, pr: Problem, out=None, pool=None, with_pool=False):
    """:func:`rope3d` and :func:`reorder` in one pass: the permuted copy
    [B, heads, N_p, d] of the rotated x and, with ``with_pool`` (or a given
    ``pool``), the block means of the rotated rows (taken before they are
    rounded): returns (x_perm, pool).  x as for :func:`rope3d`, token n at
    its place in pr's grid, which ``rope.extent`` has to cover."""
    i = _rope_checks(x, rope, pr.d)
    if x.shape != pr.natural:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected {pr.natural}")
    if rope.extent[0] < pr.F or rope.extent[1] < pr.H or rope.extent[2] < pr.W:
        raise ValueError(f"rope.extent {rope.extent} does not cover the grid {(pr.F, pr.H, pr.W)}")
    if out is None:
        out = x.new_empty(pr.permuted)
    else:
        _need(i, "out", out, pr.permuted, x.dtype)
    if pool is not None:
        _need(i, "pool", pool, pr.pooled, torch.float32)
    elif with_pool:
        pool = x.new_empty(pr.pooled, dtype=torch.float32)
    _launch(x, load().pa_rope_reorder, x.data_ptr(), _row_strides(x, "x"), out.data_ptr(),
            _dtype_code(x), pr.shape, pr.perms_ptr, rope.desc, rope.table.data_ptr(), _addr(pool))
    return (out, pool) if pool is not None else out


def block_sparse_attn_lse(q, k, v, pr: Problem, idx, counts=None, out=None, lse=None, status=None):
    """:func:`block_sparse_attn` for bf16 permuted copies q, k, v
    [B, heads, N_p, d] (:func:`reorder` or :func:`rope_reorder`), which also
    returns the natural log-sum-exp of every row, [B, heads, N] float32 (-inf
    for a row without kept blocks): the forward pass of training."""
    i = _device_of(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(i, name, t, pr.permuted, torch.bfloat16)
    _need_lists(i, idx, counts, pr)
    _need_status(i, status)
    if out is None:
        out = q.new_empty(pr.natural)
    else:
        _need(i, "out", out, pr.natural, torch.bfloat16)
    if lse is None:
        lse = q.new_empty(pr.rows, dtype=torch.float32)
    else:
        _need(i, "lse", lse, pr.rows, torch.float32)
    _launch(q, load().pa_block_sparse_attn_lse, q.data_ptr(), k.data_ptr(), v.data_ptr(), PA_BF16,
            pr.shape, pr.perms_ptr, _addr(idx), _addr(counts), idx.shape[3], out.data_ptr(),
            lse.data_ptr(), _addr(status))
    return out, lse


def block_sparse_attn_backward(dout, q, k, v, out, lse, pr: Problem, idx, counts=None, dlse=None,
                               dq=None, dk=None, dv=None, workspace=None, status=None):
    """Gradients (dq, dk, dv) [B, heads, N, d] of :func:`block_sparse_attn_lse`
    in natural token order.  q, k, v: the permuted copies of the forward
    pass; dout, out natural order; ``dlse``: the gradient of lse, if it was
    used.  The same bits on every run.  ``workspace``: a uint8 tensor of at
    least :func:`backward_workspace` bytes that no call in flight uses (by
    default allocated here)."""
    i = _device_of(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(i, name, t, pr.permuted, torch.bfloat16)
    _need(i, "dout", dout, pr.natural, torch.bfloat16)
    _need(i, "out", out, pr.natural, torch.bfloat16)
    _need(i, "lse", lse, pr.rows, torch.float32)
    if dlse is not None:
        _need(i, "dlse", dlse, pr.rows, torch.float32)
    _need_lists(i, idx, counts, pr)
    _need_status(i, status)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None:
            _need(i, name, t, pr.natural, torch.bfloat16)
    dq = torch.empty_like(out) if dq is None else dq
    dk = torch.empty_like(out) if dk is None else dk
    dv = torch.empty_like(out) if dv is None else dv
    if workspace is None:
        workspace = q.new_empty(backward_workspace(pr), dtype=torch.uint8)
    else:
        _need(i, "workspace", workspace, workspace.shape, torch.uint8)
    _launch(q, load().pa_block_sparse_attn_backward, dout.data_ptr(), q.data_ptr(), k.data_ptr(),
            v.data_ptr(), out.data_ptr(), lse.data_ptr(), _addr(dlse), PA_BF16, pr.shape,
            pr.perms_ptr, _addr(idx), _addr(counts), idx.shape[3], dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), workspace.data_ptr(), workspace.numel(), _addr(status))
    return dq, dk, dv


def backward_workspace(pr: Problem) -> int:
    """Bytes of workspace of :func:`block_sparse_attn_backward`."""
    if pr.workspace is None:
        n = load().pa_block_sparse_attn_backward_workspace(pr.shape)
        if n < 0:
            raise ParoError(PA_ERR_UNSUPPORTED, load().pa_last_error().decode())
        pr.workspace = n
    return pr.workspace


def block_sparse_query_attn(q, k, v, k_pool, pr: Problem, k_keep: int, lengths=None, out=None,
                            idx=None, lse=None, status=None):
    """Single query tokens against a stored clip (serving): every row of q
    [B, q_heads, M, d] keeps the ``k_keep`` blocks with the largest
    q . k_pool, ties to the lower index, and attends to their tokens.

    k, v [B, heads, N_p, d]: the clip in the permuted order, k_pool
    [B, heads, NB, d] float32 its block means (:func:`reorder` or
    :func:`rope_reorder` with ``with_pool``, for a whole clip); q_heads a
    multiple of heads (query head h reads key head h // (q_heads / heads)).
    ``lengths`` [B] int32: how many positions of the order exist so far
    (0 .. N).  A clip that still grows has its means kept by the caller, over
    the keys that exist: once position n - 1 is written, block j = (n - 1) //
    block has ``k_pool[b, :, j] = k[b, :, j * block:n].float().mean(1)``.
    float32 or bfloat16.  Returns (out [B, q_heads, M, d], idx [B, q_heads, M, k_keep]
    ascending with -1 behind the last, lse [B, q_heads, M]); a row without
    keys gives zeros and -inf."""
    i = _device_of(q)
    if q.dim() != 4 or q.dtype not in _FLOAT:
        raise ValueError(f"q: {tuple(q.shape)} {q.dtype}, expected four dimensions and one of {_FLOAT}")
    B, heads, M, d = q.shape
    if B != pr.B or heads < 1 or heads % pr.heads or M < 1 or d != pr.d or not q.is_contiguous():
        raise ValueError(f"q: shape {tuple(q.shape)}, expected ({pr.B}, a multiple of {pr.heads}, M, {pr.d}) "
                         "and contiguous")
    k_keep = int(k_keep)
    if not 1 <= k_keep <= pr.NB:
        raise ValueError(f"k_keep={k_keep} must be in [1, {pr.NB}]")
    _need(i, "k", k, pr.permuted, q.dtype)
    _need(i, "v", v, pr.permuted, q.dtype)
    _need(i, "k_pool", k_pool, pr.pooled, torch.float32)
    if lengths is not None:
        _need(i, "lengths", lengths, (B,), torch.int32)
    _need_status(i, status)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(i, "out", out, q.shape, q.dtype)
    if idx is None:
        idx = q.new_empty((B, heads, M, k_keep), dtype=torch.int32)
    else:
        _need(i, "idx", idx, (B, heads, M, k_keep), torch.int32)
    if lse is None:
        lse = q.new_empty((B, heads, M), dtype=torch.float32)
    else:
        _need(i, "lse", lse, (B, heads, M), torch.float32)
    _launch(q, load().pa_query_attn, q.data_ptr(), k.data_ptr(), v.data_ptr(), k_pool.data_ptr(),
            _dtype_code(q), pr.shape, heads // pr.heads, M, k_keep, _addr(lengths),
            out.data_ptr(), idx.data_ptr(), lse.data_ptr(), _addr(status))
    return out, idx, lse


def choose_orders_sics(q, k, grid, block):
    """SPADE's blocking choice per head, made by the library: the candidate
    (axis order or 3D tile blocking) whose blocks have the largest SICS of q
    and k -> list of order ids (copied to the host: the calls that follow
    take the order ids as host data)."""
    B, heads = q.shape[:2]
    pr = Problem(B, heads, grid, q.shape[-1], block, [0] * heads)
    _, orders = sics_scores(q, k, pr)
    return [int(o) for o in orders.cpu().tolist()]


def attention(q, k, v, grid, perms, block, density, int8=False, baseline=False, status=None,
              permuted=True, int4_pv=False, selection="topk", top_p=0.0, window=-1,
              compensate=False, p_tile=None, rope=None):
    """The whole path for one call: reorder with block means (one read of
    q, k, v) -> pooled block scores -> kept blocks -> block-sparse attention
    over the permuted tiles, stored back in natural order.

    ``perms``: one axis-order id per head, or "sics" to pick each head's
    order by the SICS blocking score (SPADE).  ``selection``: "topk" (the
    diagonal plus the k-1 best blocks, k from ``density``) or "hybrid" (the
    union of that Top-K, the Top-P set at ``top_p`` and the local window
    |i - j| <= ``window``, with per-row counts).  ``int8`` runs the INT8
    kernel (``int4_pv``: 4-bit P and V; ``p_tile``: P normalised and
    quantised per tile, the pages' reading, by default with ``int4_pv``
    only, since at 8 bits the one-pass form stays within the INT8
    tolerance of it).  ``permuted=False`` skips the
    reorder pass (the kernel gathers token rows); ``baseline=True`` runs the
    mma.sync comparison kernel.  ``compensate`` adds PASA's grouped
    first-order compensation of the unselected blocks (bf16 / fp32 only;
    :func:`block_sparse_attn_compensated`).  ``rope`` (:class:`RopeTable`):
    q and k are rotated first, on the way into the heads' orders where the
    path reorders them.  Returns (out, idx) — with the hybrid filter, idx is
    (idx, counts)."""
    if rope is not None and (isinstance(perms, str) or int8 or baseline or not (permuted or compensate)):
        # the step that comes first reads q and k in their natural order
        q, k = (rope3d(x, rope, grid=grid) for x in (q, k))
        rope = None
    if isinstance(perms, str):
        if perms != "sics":
            raise ValueError(f"perms={perms!r}: order ids or 'sics'")
        perms = choose_orders_sics(q, k, grid, block)
    pr = Problem.from_qkv(q, grid, perms, block)
    kk = k_for_density(pr.NB, density)

    def into_order(x):
        if rope is None:
            return reorder(x, pr, with_pool=True)
        return rope_reorder(x, rope, pr, with_pool=True)

    def select(scores):
        if selection == "hybrid":
            return select_hybrid(scores, pr, kk, top_p, window)
        if selection != "topk":
            raise ValueError(f"selection={selection!r}: topk or hybrid")
        return select_topk(scores, pr, kk), None

    if compensate:
        if int8:
            raise ValueError("compensate runs on bf16 / fp32 inputs")
        qp, q_pool = into_order(q)
        kp, k_pool = into_order(k)
        vp, v_pool = reorder(v, pr, with_pool=True)
        idx, counts = select(score_pooled(q_pool, k_pool, pr))
        if q.dtype == torch.bfloat16 and pr.d == 128 and pr.block == 128:
            # the tcgen05 kernel loads bf16 means like K and V tiles
            k_pool, v_pool = round_bf16(k_pool), round_bf16(v_pool)
        out = block_sparse_attn_compensated(qp, kp, vp, pr, idx, k_pool, v_pool, counts,
                                            status=status, permuted=True)
    elif int8:
        q8, qs, qp = quantize_int8(q, pr, with_pool=True)
        k8, ks, kp = quantize_int8(k, pr, with_pool=True)
        v8, vs = quantize_int8(v, pr, bits=4 if int4_pv else 8)
        idx, counts = select(score_pooled(qp, kp, pr))
        out = block_sparse_attn(q8, k8, v8, pr, idx, counts, scales=(qs, ks, vs), status=status,
                                p4=int4_pv, p_tile=int4_pv if p_tile is None else p_tile)
    elif permuted and not baseline:
        qp, q_pool = into_order(q)
        kp, k_pool = into_order(k)
        vp = reorder(v, pr)
        idx, counts = select(score_pooled(q_pool, k_pool, pr))
        out = block_sparse_attn(qp, kp, vp, pr, idx, counts, status=status, permuted=True)
    else:
        _, _, scores = block_score(q, k, pr)
        idx, counts = select(scores)
        out = block_sparse_attn(q, k, v, pr, idx, counts, baseline=baseline, status=status)
    return out, (idx if counts is None else (idx, counts))
