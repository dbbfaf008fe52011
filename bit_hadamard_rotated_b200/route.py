"""Tokens sorted by expert and back (include/hq.h, hq_moe_sort and the row movers).

As everywhere in this package: checks of devices, types and shapes, pointer
marshalling and the tensors' own device's current stream.  Nothing is computed
here.  hq_moe_gather and hq_moe_combine take part in autograd.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import check, lib
from .hq import _DT, _need_cuda, _need_workspace, _new, _on, _raw_stream


class MoePlan:
    """Where the pairs of a routing go: pos int32 [T][k] (row of each pair, -1
    without one), offsets int32 [n_experts + 1], counts int32 [n_experts];
    n_rows: rows that hold every possible routing of these sizes."""

    def __init__(self, buf, T, k, n_experts, ends, n_rows, align):
        self._buf, self._ends = buf, ends  # pos at its start, offsets and counts from `ends` on
        self.T, self.k, self.n_experts, self.n_rows, self.align = T, k, n_experts, n_rows, align
        self.device, self._pos = buf.device, buf.data_ptr()

    @property
    def pos(self):
        return self._buf.as_strided((self.T, self.k), (self.k, 1), 0)

    @property
    def offsets(self):
        return self._buf[self._ends:self._ends + self.n_experts + 1]

    @property
    def counts(self):
        return self._buf[self._ends + self.n_experts + 1:self._ends + 2 * self.n_experts + 1]


def hq_moe_sort(topk_ids: torch.Tensor, n_experts: int, align: int = 1, workspace: torch.Tensor | None = None,
                stream=None) -> MoePlan:
    """Sort the (token, slot) pairs of topk_ids (int32 [T][k]) by expert: each
    expert's rows in the pairs' order, its first row a multiple of align; ids
    outside [0, n_experts) get no row."""
    _need_cuda(topk_ids, workspace)
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 [T][k] tensor")
    if workspace is not None:
        _need_workspace(workspace, topk_ids.device)
    return _on(topk_ids.device, stream, _sort, topk_ids, int(n_experts), int(align), workspace)


def _sort(ids, E, align, ws):
    dev, (T, k) = ids.device, ids.shape
    L = lib()
    need = int(L.hq_moe_sort_workspace_size(T, k, E))
    # one allocation: pos, then offsets and counts, then the workspace, 256-byte aligned
    ends = (T * k + 63) // 64 * 64
    at = ends + (2 * max(E, 0) + 64) // 64 * 64
    buf = torch.empty_strided((at + (need // 4 if ws is None else 0),), (1,), dtype=torch.int32, device=dev)
    plan = MoePlan(buf, T, k, E, ends, T * k + min(E, T * k) * (align - 1), align)
    p = plan._pos
    wp, wn = (p + 4 * at, need) if ws is None else (ws.data_ptr(), ws.numel())
    st = L.hq_moe_sort(ids.data_ptr(), T, k, E, align, p, p + 4 * ends, p + 4 * (ends + E + 1), wp, wn,
                       _raw_stream(None, dev.index))
    if st:
        check(st, "hq_moe_sort")
    return plan


def _need_like(t, what, shape, dtype, dev):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {tuple(shape)} on {dev}")


def _need_rows(x, what, plan, tokens):
    """x [T][H] (tokens) or [n_rows][H], of a type the kernels take, on the plan's device."""
    if x.dtype not in _DT or x.dim() != 2 or not x.is_contiguous() or x.device != plan.device:
        raise ValueError(f"{what} must be a contiguous fp16, bf16 or fp32 matrix on the plan's device")
    if tokens and x.shape[0] != plan.T:
        raise ValueError(f"{what} must have one row per token, {plan.T}")


def _need_weights(topk_w, plan):
    _need_like(topk_w, "topk_w", (plan.T, plan.k), torch.float32, plan.device)


def _recorded(out):
    """Whether autograd records a call on tensors that require a gradient."""
    if out is not None and torch.is_grad_enabled():
        raise ValueError("a call whose gradient is recorded takes no out")
    return torch.is_grad_enabled()


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return _gather(x, plan, x.new_zeros((plan.n_rows, x.shape[1])))

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        return hq_moe_gather_grad(g.contiguous(), ctx.plan), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, topk_w, plan, out_dtype):
        ctx.plan = plan
        ctx.save_for_backward(rows, topk_w)
        return _combine(rows, plan, topk_w, out_dtype, None, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        rows, topk_w = ctx.saved_tensors
        dt = rows.dtype
        if g.dtype != dt:  # fp32 from 16-bit rows or the other way round: nothing is rounded before the products
            rows, g = rows.float(), g.float()
        drows, dw = hq_moe_combine_grad(g.contiguous(), rows, ctx.plan, topk_w, out=torch.zeros_like(rows))
        return drows.to(dt), dw, None, None


def hq_moe_gather(x: torch.Tensor, plan: MoePlan, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's row x[t] to the rows of its pairs: [n_rows][H] (rows without
    a pair are left as they are in `out`; a new tensor's are not initialised, or
    zero where x's gradient is recorded)."""
    _need_rows(x, "x", plan, True)
    if x.requires_grad and _recorded(out):
        return _on(x.device, stream, _Gather.apply, x, plan)
    if out is not None:
        _need_like(out, "out", (out.shape[0], x.shape[1]), x.dtype, x.device)
    return _on(x.device, stream, _gather, x, plan, out)


def _gather(x, plan, out):
    T, k = plan.T, plan.k
    if out is None:
        out = _new(plan.n_rows, x.shape[1], x.dtype, x.device)
    st = lib().hq_moe_gather(x.data_ptr(), _DT[x.dtype], plan._pos, T, k, x.shape[1], out.data_ptr(),
                             out.shape[0], _raw_stream(None, x.device.index))
    if st:
        check(st, "hq_moe_gather")
    return out


def _combine(rows, plan, topk_w, out_dtype, out, stream):
    _need_rows(rows, "rows", plan, False)
    T, H = plan.T, rows.shape[1]
    dt = (rows.dtype if out is None else out.dtype) if out_dtype is None else out_dtype
    if dt not in _DT:
        raise ValueError("the output must be fp16, bf16 or fp32")
    if out is not None:
        _need_like(out, "out", (T, H), dt, rows.device)
    return _on(rows.device, stream, _launch_combine, rows, plan, topk_w, dt, out)


def _launch_combine(rows, plan, topk_w, dt, out):
    T, k = plan.T, plan.k
    if out is None:
        out = _new(T, rows.shape[1], dt, rows.device)
    st = lib().hq_moe_combine(rows.data_ptr(), _DT[rows.dtype], rows.shape[0], plan._pos,
                              None if topk_w is None else topk_w.data_ptr(), T, k, rows.shape[1], out.data_ptr(),
                              _DT[out.dtype], _raw_stream(None, rows.device.index))
    if st:
        check(st, "hq_moe_combine")
    return out


def hq_moe_combine(rows: torch.Tensor, plan: MoePlan, topk_w: torch.Tensor, out_dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j topk_w[t][j] rows[pos[t][j]] (fp32 sums, slots ascending), of rows' type unless out_dtype says
    otherwise."""
    _need_weights(topk_w, plan)
    if (rows.requires_grad or topk_w.requires_grad) and _recorded(out):
        return _on(rows.device, stream, _Combine.apply, rows, topk_w, plan, out_dtype)
    return _combine(rows, plan, topk_w, out_dtype, out, stream)


def hq_moe_gather_grad(drows: torch.Tensor, plan: MoePlan, out_dtype: torch.dtype | None = None,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of hq_moe_gather: dx[t] = sum_j drows[pos[t][j]]."""
    return _combine(drows, plan, None, out_dtype, out, stream)


def hq_moe_combine_grad(dy: torch.Tensor, rows: torch.Tensor, plan: MoePlan, topk_w: torch.Tensor,
                        out: torch.Tensor | None = None, stream=None):
    """(drows, dtopk_w), the gradients of hq_moe_combine: drows[pos[t][j]] =
    topk_w[t][j] dy[t] (rows without a pair are left as they are in `out`; a new
    tensor's are not initialised) and dtopk_w[t][j] = <dy[t], rows[pos[t][j]]>
    in fp32."""
    _need_rows(dy, "dy", plan, True)
    _need_rows(rows, "rows", plan, False)
    _need_weights(topk_w, plan)
    if rows.dtype != dy.dtype or rows.shape[1] != dy.shape[1]:
        raise ValueError("dy and rows must have one type and width")
    if out is not None:
        _need_like(out, "out", rows.shape, rows.dtype, rows.device)
    return _on(dy.device, stream, _combine_grad, dy, rows, plan, topk_w, out)


def _combine_grad(dy, rows, plan, topk_w, out):
    T, k = plan.T, plan.k
    if out is None:
        out = torch.empty_like(rows)
    dw = torch.empty_like(topk_w)
    st = lib().hq_moe_combine_grad(dy.data_ptr(), _DT[dy.dtype], rows.data_ptr(), rows.shape[0], plan._pos,
                                   topk_w.data_ptr(), T, k, rows.shape[1], out.data_ptr(), dw.data_ptr(),
                                   _raw_stream(None, dy.device.index))
    if st:
        check(st, "hq_moe_combine_grad")
    return out, dw


__all__ = ["MoePlan", "hq_moe_sort", "hq_moe_gather", "hq_moe_gather_grad", "hq_moe_combine", "hq_moe_combine_grad"]
