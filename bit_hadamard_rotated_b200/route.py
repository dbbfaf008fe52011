"""Tokens sorted by expert and back (include/hq.h, hq_moe_sort and the row movers).

As everywhere in this package: checks of devices, types and shapes, pointer
marshalling and the tensors' own device's current stream.  Nothing is computed
here.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import check, lib
from .hq import _DT, _need_cuda, _ptr, _raw_stream


def _on(t: torch.Tensor):
    """The device of t as the current one, for the launches of a call."""
    return torch.cuda.device(t.device)


def _st(stream, t):
    return _raw_stream(stream, t.device.index)


class MoePlan:
    """Where the pairs of a routing go: pos int32 [T][k] (row of each pair, -1
    without one), offsets int32 [n_experts + 1], counts int32 [n_experts];
    n_rows: rows that hold every possible routing of these sizes."""

    def __init__(self, pos, offsets, counts, n_rows, align):
        self.pos, self.offsets, self.counts, self.n_rows, self.align = pos, offsets, counts, n_rows, align


def hq_moe_sort(topk_ids: torch.Tensor, n_experts: int, align: int = 1, workspace: torch.Tensor | None = None,
                stream=None) -> MoePlan:
    """Sort the (token, slot) pairs of topk_ids (int32 [T][k]) by expert: each
    expert's rows in the pairs' order, its first row a multiple of align; ids
    outside [0, n_experts) get no row."""
    _need_cuda(topk_ids, workspace)
    if topk_ids.dtype != torch.int32 or topk_ids.dim() != 2 or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 [T][k] tensor")
    T, k = topk_ids.shape
    dev = topk_ids.device
    with _on(topk_ids):
        need = int(lib().hq_moe_sort_workspace_size(T, k, n_experts))
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        pos = torch.empty((T, k), dtype=torch.int32, device=dev)
        ends = torch.empty(max(2 * n_experts + 1, 1), dtype=torch.int32, device=dev)
        offsets, counts = ends[:n_experts + 1], ends[n_experts + 1:]
        check(lib().hq_moe_sort(_ptr(topk_ids), T, k, n_experts, align, _ptr(pos), _ptr(offsets), _ptr(counts),
                                _ptr(workspace), workspace.numel(), _st(stream, topk_ids)), "hq_moe_sort")
    return MoePlan(pos, offsets, counts, T * k + min(n_experts, T * k) * (align - 1), align)


def _need_like(t, what, shape, dtype, dev):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {tuple(shape)} on {dev}")


def _need_rows(x, what, plan, tokens):
    """x [T][H] (tokens) or [n_rows][H], of a type the kernels take, on the plan's device."""
    _need_cuda(x, plan.pos)
    if x.dtype not in _DT or x.dim() != 2 or not x.is_contiguous() or x.device != plan.pos.device:
        raise ValueError(f"{what} must be a contiguous fp16, bf16 or fp32 matrix on the plan's device")
    if tokens and x.shape[0] != plan.pos.shape[0]:
        raise ValueError(f"{what} must have one row per token, {plan.pos.shape[0]}")


def _need_weights(topk_w, plan):
    _need_like(topk_w, "topk_w", plan.pos.shape, torch.float32, plan.pos.device)


def hq_moe_gather(x: torch.Tensor, plan: MoePlan, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Each token's row x[t] to the rows of its pairs: [n_rows][H] (rows without
    a pair are left as they are in `out`; a new tensor's are not initialised)."""
    _need_rows(x, "x", plan, True)
    T, H = x.shape
    if out is None:
        out = torch.empty((plan.n_rows, H), dtype=x.dtype, device=x.device)
    else:
        _need_like(out, "out", (out.shape[0], H), x.dtype, x.device)
    with _on(x):
        check(lib().hq_moe_gather(_ptr(x), _DT[x.dtype], _ptr(plan.pos), T, plan.pos.shape[1], H, _ptr(out),
                                  out.shape[0], _st(stream, x)), "hq_moe_gather")
    return out


def _combine(rows, plan, topk_w, out_dtype, out, stream):
    _need_rows(rows, "rows", plan, False)
    T, k = plan.pos.shape
    H = rows.shape[1]
    dt = (rows.dtype if out is None else out.dtype) if out_dtype is None else out_dtype
    if dt not in _DT:
        raise ValueError("the output must be fp16, bf16 or fp32")
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=rows.device)
    else:
        _need_like(out, "out", (T, H), dt, rows.device)
    with _on(rows):
        check(lib().hq_moe_combine(_ptr(rows), _DT[rows.dtype], rows.shape[0], _ptr(plan.pos), _ptr(topk_w), T, k, H,
                                   _ptr(out), _DT[dt], _st(stream, rows)), "hq_moe_combine")
    return out


def hq_moe_combine(rows: torch.Tensor, plan: MoePlan, topk_w: torch.Tensor, out_dtype: torch.dtype | None = None,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = sum_j topk_w[t][j] rows[pos[t][j]] (fp32 sums, slots ascending), of rows' type unless out_dtype says
    otherwise."""
    _need_weights(topk_w, plan)
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
    T, H = dy.shape
    if out is None:
        out = torch.empty_like(rows)
    else:
        _need_like(out, "out", rows.shape, rows.dtype, rows.device)
    dw = torch.empty(plan.pos.shape, dtype=torch.float32, device=dy.device)
    with _on(dy):
        check(lib().hq_moe_combine_grad(_ptr(dy), _DT[dy.dtype], _ptr(rows), rows.shape[0], _ptr(plan.pos),
                                        _ptr(topk_w), T, plan.pos.shape[1], H, _ptr(out), _ptr(dw), _st(stream, dy)),
              "hq_moe_combine_grad")
    return out, dw


__all__ = ["MoePlan", "hq_moe_sort", "hq_moe_gather", "hq_moe_gather_grad", "hq_moe_combine", "hq_moe_combine_grad"]
