"""Microscaled 4-bit floating-point matrices (include/hq.h, hq_fp4_*).

As everywhere in this package: checks of devices, types and shapes, pointer
marshalling and the tensors' own device's current stream.  Nothing is computed
here.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import HQ_FP4_MX, HQ_FP4_NV, HqFp4Matrix, check, lib
from .hq import _DT, _need_cuda, _need_workspace, _new, _on, _ptr, _raw_stream

_FMT = {"nv": HQ_FP4_NV, "mx": HQ_FP4_MX}
_ZEROED = 8448  # bytes at a workspace's start, the status word and the counters: all of it that has to be zero


def _scale_shape(fmt: str, rows: int, K: int):
    """Scale tiles [row tiles][K tiles][32][4][4] (include/hq.h)."""
    return (rows + 127) // 128, -(-K // (64 if fmt == "nv" else 128)), 32, 4, 4


def _need_scale(t, dev, n=1):
    if t is not None and (t.dtype != torch.float32 or t.numel() not in (1, n) or not t.is_contiguous()
                          or t.device != dev):
        raise ValueError(f"a tensor scale must be fp32 with {'one value' if n == 1 else f'1 or {n} values'} on {dev}")


class Fp4Matrix:
    """A packed matrix: codes uint8 [rows][K/2], scales uint8 tiles [row
    tiles][K tiles][32][4][4], fmt "nv" or "mx", tensor_scale fp32 (one value,
    or one per expert) or None.  values: the rounded values, where
    hq_fp4_quantize was asked for them."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, fmt: str = "nv",
                 tensor_scale: torch.Tensor | None = None, values: torch.Tensor | None = None):
        _need_cuda(codes, scales, tensor_scale)
        if fmt not in _FMT:
            raise ValueError('fmt must be "nv" or "mx"')
        if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
            raise ValueError("codes must be a contiguous uint8 [rows][K/2] tensor")
        rows, K = codes.shape[0], codes.shape[1] * 2
        if (scales.dtype != torch.uint8 or tuple(scales.shape) != _scale_shape(fmt, rows, K)
                or not scales.is_contiguous() or scales.device != codes.device):
            raise ValueError(f"scales must be contiguous uint8 tiles {_scale_shape(fmt, rows, K)} on {codes.device}")
        if tensor_scale is not None and (fmt != "nv" or tensor_scale.dtype != torch.float32 or tensor_scale.numel() < 1
                                         or not tensor_scale.is_contiguous() or tensor_scale.device != codes.device):
            raise ValueError(f'tensor_scale must be contiguous fp32 on {codes.device}, and only for "nv"')
        self._set(codes, scales, fmt, tensor_scale, values)

    def _set(self, codes, scales, fmt, tensor_scale, values):
        self.codes, self.scales, self.fmt, self.tensor_scale, self.values = codes, scales, fmt, tensor_scale, values
        self.c = HqFp4Matrix(_FMT[fmt], codes.shape[0], codes.shape[1] * 2, codes.data_ptr(), scales.data_ptr(),
                             None if tensor_scale is None else tensor_scale.data_ptr(),
                             0 if tensor_scale is None else tensor_scale.numel())
        self._ref = ctypes.byref(self.c)
        return self

    @property
    def rows(self):
        return self.c.rows

    @property
    def K(self):
        return self.c.K


def _need_rows(x, K=None):
    if x.dtype not in _DT or x.dim() != 2 or (K is not None and x.shape[1] != K):
        raise ValueError(f"x must be fp16, bf16 or fp32 [rows][{'K' if K is None else K}]")


def _rows_in(x):
    """x as rows the kernels read: unit stride along K and rows on 16-byte
    boundaries (copied if they are not), and its row stride (of a contiguous x
    its width: torch keeps any stride for a single row)."""
    if x.is_contiguous():
        return x if x.data_ptr() % 16 == 0 else x.clone(), x.shape[1]
    if x.stride(1) != 1 or x.stride(0) < x.shape[1] or x.stride(0) * x.element_size() % 16 or x.data_ptr() % 16:
        return x.contiguous(), x.shape[1]
    return x, x.stride(0)


def hq_fp4_tensor_scale(x: torch.Tensor, stream=None) -> torch.Tensor:
    """max |x| / 2688 as an fp32 scalar tensor: the tensor scale that puts x's
    largest block at the end of the "nv" format's range (1 for zeros)."""
    _need_cuda(x)
    _need_rows(x)
    return _on(x.device, stream, _tensor_scale, x)


def _tensor_scale(x):
    dev = x.device
    x, ldx = _rows_in(x)
    out = torch.empty_strided((), (), dtype=torch.float32, device=dev)
    ws = _new(1, 256, torch.uint8, dev)
    check(lib().hq_fp4_tensor_scale(x.data_ptr(), _DT[x.dtype], ldx, x.shape[0], x.shape[1],
                                    out.data_ptr(), ws.data_ptr(), 256, _raw_stream(None, dev.index)),
          "hq_fp4_tensor_scale")
    return out


def hq_fp4_quantize(x: torch.Tensor, fmt: str = "nv", tensor_scale: torch.Tensor | None = None, values=False,
                    stream=None) -> Fp4Matrix:
    """Pack rows x [rows][K] (fp16/bf16/fp32, K a multiple of 32).  values: True,
    or a tensor like x to write into, for the rounded values in x's type too."""
    if not x.is_cuda:
        _need_cuda(x)
    if fmt not in _FMT:
        raise ValueError('fmt must be "nv" or "mx"')
    _need_rows(x)
    if tensor_scale is not None:
        if fmt != "nv":
            raise ValueError('only "nv" takes a tensor scale')
        _need_scale(tensor_scale, x.device)
    if values is not True and values is not False and values is not None and (
            values.dtype != x.dtype or values.shape != x.shape or not values.is_contiguous() or values.device != x.device):
        raise ValueError("values must be a contiguous tensor of x's type and shape")
    return _on(x.device, stream, _quantize, x, fmt, tensor_scale, values)


def _quantize(x, fmt, tensor_scale, values):
    dev, (rows, K) = x.device, x.shape
    x, ldx = _rows_in(x)
    kb = -(-K // (64 if fmt == "nv" else 128))
    if values is True:
        values = _new(rows, K, x.dtype, dev)
    elif values is False:
        values = None
    q = Fp4Matrix.__new__(Fp4Matrix)._set(
        _new(rows, K // 2, torch.uint8, dev),
        torch.empty_strided(_scale_shape(fmt, rows, K), (512 * kb, 512, 16, 4, 1), dtype=torch.uint8, device=dev), fmt,
        tensor_scale, values)
    if K & 1:
        q.c.K = K  # as given: an odd K is refused below
    st = lib().hq_fp4_quantize(x.data_ptr(), _DT[x.dtype], ldx, q._ref,
                               None if values is None else values.data_ptr(), _raw_stream(None, dev.index))
    if st:
        check(st, "hq_fp4_quantize")
    return q


def _out(out, rows, M, dtype, dev):
    """The output and its row stride (rows may be strided, columns not)."""
    if dtype not in _DT:
        raise ValueError("the output must be fp16, bf16 or fp32")
    if out is None:
        return _new(rows, M, dtype, dev), M
    if out.dtype != dtype or tuple(out.shape) != (rows, M) or out.device != dev or (M > 1 and out.stride(1) != 1) \
            or (rows > 1 and out.stride(0) < M):
        raise ValueError(f"out must be {dtype} [{rows}][{M}] on {dev} with unit column stride")
    return out, max(out.stride(0), M)


def _workspace(need, dev):
    ws = torch.empty(max(need, _ZEROED), dtype=torch.uint8, device=dev)
    ws[:_ZEROED].zero_()
    return ws


def hq_fp4_matmul(w: Fp4Matrix, a: Fp4Matrix, out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[n][m] = sum_k w[m][k] a[n][k] of two packed matrices, [a.rows][w.rows]."""
    dev = w.codes.device
    if a.codes.device != dev:
        raise ValueError(f"a is on {a.codes.device}, the weights on {dev}")
    if workspace is not None:
        _need_workspace(workspace, dev)
    return _on(dev, stream, _matmul, w, a, out_dtype, out, workspace)


def _matmul(w, a, out_dtype, out, workspace):
    dev = w.codes.device
    out, ldy = _out(out, a.rows, w.rows, out_dtype if out is None else out.dtype, dev)
    ws = _workspace(int(lib().hq_fp4_matmul_workspace_size(w._ref, a.rows)), dev) if workspace is None else workspace
    check(lib().hq_fp4_matmul(w._ref, a._ref, out.data_ptr(), _DT[out.dtype], ldy, ws.data_ptr(), ws.numel(),
                              _raw_stream(None, dev.index)), "hq_fp4_matmul")
    return out


def hq_fp4_linear(w: Fp4Matrix, x: torch.Tensor, x_scale: torch.Tensor | None = None,
                  out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = W q(x): x [N][K] (fp16/bf16/fp32) quantised row by row in w's format
    (x_scale: its tensor scale), times the packed weights; [N][w.rows] of x's
    type unless out_dtype says otherwise."""
    _need_cuda(x, x_scale)
    dev = w.codes.device
    _need_rows(x, w.K)
    if x.device != dev:
        raise ValueError(f"x is on {x.device}, the weights on {dev}")
    _need_scale(x_scale, dev)
    if workspace is not None:
        _need_workspace(workspace, dev)
    dtype = out_dtype or (x.dtype if out is None else out.dtype)
    return _on(dev, stream, _linear, w, x, x_scale, dtype, out, workspace)


def _linear(w, x, x_scale, dtype, out, workspace):
    dev, N = w.codes.device, x.shape[0]
    x, ldx = _rows_in(x)
    out, ldy = _out(out, N, w.rows, dtype, dev)
    ws = _workspace(int(lib().hq_fp4_linear_workspace_size(w._ref, N)), dev) if workspace is None else workspace
    st = lib().hq_fp4_linear(w._ref, x.data_ptr(), _DT[x.dtype], ldx, N,
                             None if x_scale is None else x_scale.data_ptr(), out.data_ptr(), _DT[dtype], ldy,
                             ws.data_ptr(), ws.numel(), _raw_stream(None, dev.index))
    if st:
        check(st, "hq_fp4_linear")
    return out


class _Layer:
    """A layer's workspace.  It grows with the calls.  One that a graph was
    captured on is kept when it is outgrown, and its successor is at least
    twice as large; any other is given back."""

    def __init__(self):
        self._ws, self._captured, self._outgrown = None, False, []

    def _grow(self, need, dev):
        if self._ws is not None and need <= self._ws.numel():
            return
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("call the layer once at this size before capturing it: its workspace has to grow")
        old = self._ws
        if old is not None and self._captured:
            self._outgrown.append(old)
            need = max(need, 2 * old.numel())
        self._ws = _workspace(need, dev)
        if old is not None and not self._captured:
            self._ws[:4].copy_(old[:4])  # the status of earlier calls
            old.record_stream(torch.cuda.current_stream(dev))  # they may still be running
        self._captured = False

    def _room_for_call(self):
        """The workspace as a call uses it."""
        if not self._captured and torch.cuda.is_current_stream_capturing():
            self._captured = True
        return self._ws

    def check_status(self, stream=None):
        """Raise HqError if a call on this layer, or a graph captured of one,
        recorded a device error; the layer is ready for the next call then."""
        for ws in (*self._outgrown, self._ws):
            if ws is not None:
                _on(ws.device, stream, self._check, ws)

    @staticmethod
    def _check(ws):
        st = lib().hq_check_status(ws.data_ptr(), _raw_stream(None, ws.device.index))
        if st:
            ws[:_ZEROED].zero_()  # counters that the failed call left
            check(st, "device status")


class Fp4Linear(_Layer):
    """A packed linear layer with its workspace: y = W q(x) (hq_fp4_linear).
    x_scale: the activations' tensor scale ("nv"), or None.  One layer, captured
    graphs of it included, serves one stream at a time."""

    def __init__(self, w: Fp4Matrix, x_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None):
        super().__init__()
        self.w, self.x_scale, self.out_dtype = w, x_scale, out_dtype
        _need_scale(x_scale, w.codes.device)
        self._batch = -1  # a workspace for a batch serves every smaller one

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        dev = self.w.codes.device
        if x.device != dev:
            raise ValueError(f"x is on {x.device}, the weights on {dev}")
        _need_rows(x, self.w.K)
        return _on(dev, stream, self._call, x, out)

    def _call(self, x, out):
        w, N = self.w, x.shape[0]
        if N > self._batch:
            need = int(lib().hq_fp4_linear_workspace_size(w._ref, N))
            self._grow(need, w.codes.device)
            if need:  # else the call below is refused
                self._batch = N
        return _linear(w, x, self.x_scale, self.out_dtype or (x.dtype if out is None else out.dtype), out,
                       self._room_for_call())


class Fp4Experts(_Layer):
    """The routed-expert layer on packed weights with its workspace
    (hq_fp4_experts): gate, up [n_experts * inter rows], down [n_experts *
    hidden rows].  x_scale, h_scale: tensor scales of the activations and of
    h ("nv"), or None.  One layer, captured graphs of it included, serves one
    stream at a time."""

    def __init__(self, gate: Fp4Matrix, up: Fp4Matrix, down: Fp4Matrix, n_experts: int,
                 x_scale: torch.Tensor | None = None, h_scale: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None):
        super().__init__()
        dev = gate.codes.device
        if up.codes.device != dev or down.codes.device != dev:
            raise ValueError(f"the three matrices must be on one device, {dev}")
        _need_scale(x_scale, dev)
        _need_scale(h_scale, dev)
        self.gate, self.up, self.down, self.n_experts = gate, up, down, int(n_experts)
        self.x_scale, self.h_scale, self.out_dtype = x_scale, h_scale, out_dtype
        self.hidden = gate.K
        self._room = (-1, 0, None)
        if not self._need(1, 1, torch.float32):
            raise ValueError("unsupported expert layer: formats, sizes or tensor scales do not fit together")

    def _need(self, T, k, dtype):
        return int(lib().hq_fp4_experts_workspace_size(self.gate._ref, self.up._ref, self.down._ref, self.n_experts, T, k,
                                                       _DT[dtype]))

    def __call__(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
        """y [T][hidden] of x [T][hidden], topk_ids int32 [T][k], topk_w fp32 [T][k]."""
        dev = self.gate.codes.device
        _need_rows(x, self.hidden)
        T = x.shape[0]
        if topk_ids.dtype != torch.int32 or topk_w.dtype != torch.float32 or topk_ids.dim() != 2 \
                or topk_ids.shape[0] != T or topk_w.shape != topk_ids.shape:
            raise ValueError(f"topk_ids and topk_w must be int32 and fp32 [{T}][k]")
        for t in (x, topk_ids, topk_w):
            if t.device != dev:
                raise ValueError(f"a tensor is on {t.device}, the weights on {dev}")
        dtype = self.out_dtype or (x.dtype if out is None else out.dtype)
        if out is not None and (out.dtype != dtype or tuple(out.shape) != (T, self.hidden) or not out.is_contiguous()
                                or out.device != dev):
            raise ValueError(f"out must be contiguous {dtype} [{T}][{self.hidden}] on {dev}")
        return _on(dev, stream, self._call, x, topk_ids, topk_w, dtype, out)

    def _call(self, x, ids, w, dtype, out):
        dev, (T, k) = x.device, ids.shape
        x, ldx = _rows_in(x)
        ids, w = ids.contiguous(), w.contiguous()
        if out is None:
            out = _new(T, self.hidden, dtype, dev)
        room = self._room
        if T > room[0] or k != room[1] or dtype != room[2]:
            need = self._need(T, k, dtype)
            self._grow(need, dev)
            if need:  # else the call below is refused
                self._room = (T, k, dtype)
        ws = self._room_for_call()
        st = lib().hq_fp4_experts(self.gate._ref, self.up._ref, self.down._ref, self.n_experts, x.data_ptr(),
                                  _DT[x.dtype], ldx, T, ids.data_ptr(), w.data_ptr(), k,
                                  _ptr(self.x_scale), _ptr(self.h_scale), out.data_ptr(), _DT[dtype],
                                  ws.data_ptr(), ws.numel(), _raw_stream(None, dev.index))
        if st:
            check(st, "hq_fp4_experts")
        return out


__all__ = ["Fp4Experts", "Fp4Matrix", "Fp4Linear", "hq_fp4_tensor_scale", "hq_fp4_quantize", "hq_fp4_matmul", "hq_fp4_linear"]
