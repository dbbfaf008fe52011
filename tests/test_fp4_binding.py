"""The Python binding's own checks of the 4-bit floating-point and routing calls, on CPU tensors with a stand-in for the
library that records what reaches it."""
from types import SimpleNamespace

import pytest
import torch

from bit_hadamard_rotated_b200 import HqError, fp4, hq, route


class Recorder:
    """Answers every size with 512 and every call with success."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 512
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    for mod in (fp4, route):
        monkeypatch.setattr(mod, "lib", lambda: r)
        monkeypatch.setattr(mod, "_need_cuda", lambda *ts: None)
        monkeypatch.setattr(mod, "_raw_stream", lambda *a: 0)
        monkeypatch.setattr(mod, "_on", lambda dev, stream, fn, *a: fn(*a))
    return r


def bytes_(n):
    return torch.zeros(n, dtype=torch.uint8)


BAD = {
    "expanded": lambda: bytes_(1).expand(1 << 16),
    "strided": lambda: bytes_(1 << 17)[::2],
    "of another type": lambda: torch.zeros(1 << 16, dtype=torch.int32),
    "of another device": lambda: torch.zeros(1 << 16, dtype=torch.uint8, device="meta"),
}


@pytest.mark.parametrize("how", BAD)
def test_sort_refuses_workspaces(rec, how):
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        route.hq_moe_sort(ids, 8, workspace=BAD[how]())
    assert rec.calls == []
    route.hq_moe_sort(ids, 8, workspace=bytes_(1 << 16))
    assert [n for n, _ in rec.calls] == ["hq_moe_sort"]


def matrix(rows, K):
    return fp4.Fp4Matrix(torch.zeros(rows, K // 2, dtype=torch.uint8), torch.zeros(fp4._scale_shape("nv", rows, K), dtype=torch.uint8))


@pytest.mark.parametrize("how", BAD)
def test_products_refuse_workspaces(rec, how):
    w, a = matrix(128, 64), matrix(4, 64)
    for call in (lambda ws: fp4.hq_fp4_linear(w, torch.zeros(4, 64), workspace=ws), lambda ws: fp4.hq_fp4_matmul(w, a, workspace=ws)):
        rec.calls.clear()
        with pytest.raises(ValueError):
            call(BAD[how]())
        assert rec.calls == []
        call(bytes_(1 << 16))
        assert len(rec.calls) == 1


def test_a_stream_of_another_device_is_refused():
    """It would not be the one that the call runs on: launches go to the current stream of the tensors' device."""
    ran = []
    with pytest.raises(ValueError):
        hq._on(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)), ran.append, 1)
    assert ran == []


class Sized(Recorder):
    """Sizes that go by the batch, 0 (refused) beyond 1000; calls are refused with a workspace too small for them."""

    def __getattr__(self, name):
        def size(*a):
            n = a[1] if name.startswith("hq_fp4_linear") else a[4]
            return 0 if n > 1000 else 10000 + 100 * n

        def call(*a):
            self.calls.append((name, a))
            n, room = (a[4], a[10]) if name == "hq_fp4_linear" else (a[7], a[16])
            return 2 if n > 1000 else 3 if room < 10000 + 100 * n else 0
        return size if name.endswith("workspace_size") else call


def test_a_refused_batch_leaves_the_layer_as_it_was(rec, monkeypatch):
    """A batch beyond the library's limits is refused; smaller ones still get their workspace."""
    r = Sized()
    monkeypatch.setattr(fp4, "lib", lambda: r)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    lin = fp4.Fp4Linear(matrix(128, 64))
    exp = fp4.Fp4Experts(matrix(256, 128), matrix(256, 128), matrix(256, 128), 2)

    def experts(T):
        return exp(torch.zeros(T, 128), torch.zeros(T, 2, dtype=torch.int32), torch.zeros(T, 2))
    for call in (lambda n: lin(torch.zeros(n, 64)), experts):
        call(4)
        with pytest.raises(HqError):
            call(2000)
        for n in (3, 900, 500):
            assert call(n).shape[0] == n
