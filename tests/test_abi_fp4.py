"""Host-only checks of the 4-bit floating-point and routing entry points: bad
arguments are rejected before anything is launched (these calls never reach the
GPU, so they run on a CPU-only box)."""
import ctypes

import pytest

from bit_hadamard_rotated_b200 import _lib
from bit_hadamard_rotated_b200._lib import (HQ_BF16, HQ_ERR_INVALID_ARG, HQ_ERR_UNSUPPORTED, HQ_ERR_WORKSPACE, HQ_F16,
                                            HQ_F32, HQ_FP4_MX, HQ_FP4_NV, HQ_OK, HqFp4Matrix)

FAKE = 0x100000  # aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    from bit_hadamard_rotated_b200 import build
    build.build()
    return _lib.lib()


def mat(format=HQ_FP4_NV, rows=256, K=512, codes=FAKE, scales=FAKE, ts=None, n=0):
    return HqFp4Matrix(format, rows, K, codes, scales, ts, n)


def ref(m):
    return None if m is None else ctypes.byref(m)


BAD = [
    (dict(format=2), HQ_ERR_INVALID_ARG), (dict(format=-1), HQ_ERR_INVALID_ARG), (dict(rows=-1), HQ_ERR_INVALID_ARG),
    (dict(rows=(1 << 28) + 1), HQ_ERR_INVALID_ARG), (dict(K=0), HQ_ERR_INVALID_ARG), (dict(K=-32), HQ_ERR_INVALID_ARG),
    (dict(K=48), HQ_ERR_UNSUPPORTED), (dict(K=(1 << 17) + 32), HQ_ERR_UNSUPPORTED), (dict(codes=None), HQ_ERR_INVALID_ARG),
    (dict(codes=FAKE + 8), HQ_ERR_INVALID_ARG), (dict(scales=None), HQ_ERR_INVALID_ARG), (dict(scales=FAKE + 4), HQ_ERR_INVALID_ARG),
    (dict(ts=FAKE + 2, n=1), HQ_ERR_INVALID_ARG), (dict(ts=FAKE, n=0), HQ_ERR_INVALID_ARG),
    (dict(format=HQ_FP4_MX, ts=FAKE, n=1), HQ_ERR_INVALID_ARG),
]


@pytest.fixture(autouse=True)
def nothing_launched(L):
    before = L.hq_launch_count()
    yield
    assert L.hq_launch_count() == before


def quant(L, m, x=FAKE, xd=HQ_BF16, ldx=512, values=None):
    return L.hq_fp4_quantize(x, xd, ldx, ref(m), values, None)


def test_scale_bytes(L):
    assert L.hq_fp4_scale_bytes(HQ_FP4_NV, 128, 64) == 512
    assert L.hq_fp4_scale_bytes(HQ_FP4_NV, 129, 96) == 4 * 512
    assert L.hq_fp4_scale_bytes(HQ_FP4_MX, 1, 160) == 2 * 512
    assert L.hq_fp4_scale_bytes(HQ_FP4_MX, 1, 40) == 0 and L.hq_fp4_scale_bytes(3, 1, 64) == 0


@pytest.mark.parametrize("kw,want", BAD)
def test_bad_matrices(L, kw, want):
    assert quant(L, mat(**kw)) == want
    assert L.hq_fp4_matmul(ref(mat(**kw)), ref(mat()), FAKE, HQ_F32, 1 << 29, FAKE, 1 << 40, None) == want
    assert L.hq_fp4_linear(ref(mat(**kw)), FAKE, HQ_F16, 1 << 18, 4, None, FAKE, HQ_F32, 1 << 29, FAKE, 1 << 40, None) == want
    assert L.hq_fp4_matmul_workspace_size(ref(mat(**kw)), 4) == 0
    assert L.hq_fp4_linear_launches(ref(mat(**kw)), 4) == 0


def test_quantize_rejects(L):
    assert L.hq_fp4_quantize(FAKE, HQ_BF16, 512, None, None, None) == HQ_ERR_INVALID_ARG
    assert quant(L, mat(), x=None) == HQ_ERR_INVALID_ARG
    assert quant(L, mat(), x=FAKE + 8) == HQ_ERR_INVALID_ARG
    assert quant(L, mat(), xd=3) == HQ_ERR_INVALID_ARG
    assert quant(L, mat(), ldx=511) == HQ_ERR_INVALID_ARG         # less than K
    assert quant(L, mat(), ldx=513) == HQ_ERR_INVALID_ARG         # rows off 16-byte boundaries
    assert quant(L, mat(), xd=HQ_F32, ldx=514) == HQ_ERR_INVALID_ARG
    assert quant(L, mat(), values=FAKE + 4) == HQ_ERR_INVALID_ARG
    assert quant(L, mat(ts=FAKE, n=2)) == HQ_ERR_UNSUPPORTED      # one tensor scale per matrix here
    assert quant(L, mat(rows=0, codes=None, scales=None)) == HQ_OK


def test_tensor_scale_rejects(L):
    f = lambda x=FAKE, xd=HQ_F16, ldx=512, rows=4, K=512, out=FAKE, ws=FAKE, n=256: L.hq_fp4_tensor_scale(  # noqa: E731
        x, xd, ldx, rows, K, out, ws, n, None)
    assert f(rows=0) == HQ_ERR_INVALID_ARG and f(x=None) == HQ_ERR_INVALID_ARG and f(out=None) == HQ_ERR_INVALID_ARG
    assert f(K=500) == HQ_ERR_UNSUPPORTED and f(ldx=500) == HQ_ERR_INVALID_ARG and f(out=FAKE + 2) == HQ_ERR_INVALID_ARG
    assert f(ws=None) == HQ_ERR_WORKSPACE and f(ws=FAKE + 64) == HQ_ERR_WORKSPACE and f(n=255) == HQ_ERR_WORKSPACE


def test_matmul_rejects(L):
    w = mat()
    need = L.hq_fp4_matmul_workspace_size(ref(w), 4)
    f = lambda a=mat(rows=4), y=FAKE, yd=HQ_F32, ldy=256, ws=FAKE, n=need: L.hq_fp4_matmul(  # noqa: E731
        ref(w), ref(a), y, yd, ldy, ws, n, None)
    assert f(a=None) == HQ_ERR_INVALID_ARG and f(a=mat(rows=4, K=544)) == HQ_ERR_INVALID_ARG
    assert f(a=mat(rows=4, format=HQ_FP4_MX)) == HQ_ERR_INVALID_ARG and f(a=mat(rows=4, codes=FAKE + 1)) == HQ_ERR_INVALID_ARG
    assert f(a=mat(rows=4, ts=FAKE, n=3)) == HQ_ERR_UNSUPPORTED
    assert f(y=None) == HQ_ERR_INVALID_ARG and f(y=FAKE + 2) == HQ_ERR_INVALID_ARG and f(yd=9) == HQ_ERR_INVALID_ARG
    assert f(ldy=255) == HQ_ERR_INVALID_ARG and f(ws=None) == HQ_ERR_WORKSPACE and f(n=need - 1) == HQ_ERR_WORKSPACE
    assert f(a=mat(rows=0)) == HQ_OK
    assert L.hq_fp4_matmul(ref(mat(rows=0)), ref(mat()), FAKE, HQ_F32, 256, FAKE, 1 << 40, None) == HQ_ERR_INVALID_ARG


def test_linear_rejects(L):
    w = mat()
    need = L.hq_fp4_linear_workspace_size(ref(w), 4)
    f = lambda x=FAKE, xd=HQ_BF16, ldx=512, N=4, xs=None, y=FAKE, yd=HQ_BF16, ldy=256, ws=FAKE, n=need, w=w: L.hq_fp4_linear(  # noqa: E731
        ref(w), x, xd, ldx, N, xs, y, yd, ldy, ws, n, None)
    assert f(N=-1) == HQ_ERR_INVALID_ARG and f(x=None) == HQ_ERR_INVALID_ARG and f(x=FAKE + 2) == HQ_ERR_INVALID_ARG
    assert f(ldx=500) == HQ_ERR_INVALID_ARG and f(ldx=516) == HQ_ERR_INVALID_ARG and f(y=FAKE + 1) == HQ_ERR_INVALID_ARG
    assert f(xs=FAKE + 2) == HQ_ERR_INVALID_ARG and f(w=mat(format=HQ_FP4_MX), xs=FAKE) == HQ_ERR_INVALID_ARG
    assert f(ws=FAKE + 128) == HQ_ERR_WORKSPACE and f(n=need - 1) == HQ_ERR_WORKSPACE
    assert f(w=mat(ts=FAKE, n=2)) == HQ_ERR_UNSUPPORTED and f(N=(1 << 22) + 1) == HQ_ERR_UNSUPPORTED
    assert f(N=0) == HQ_OK


def test_workspace_serves_smaller_batches(L):
    """Sizes never shrink as the batch grows, whatever the weights' shape."""
    for fmt in (HQ_FP4_NV, HQ_FP4_MX):
        for K in (32, 512, 4096, 8192, 32768):
            for rows in (1, 128, 4096, 28672):
                w = mat(format=fmt, rows=rows, K=K)
                sizes = [L.hq_fp4_linear_workspace_size(ref(w), n) for n in list(range(1, 300)) + [1000, 5000]]
                assert all(s > 0 for s in sizes) and all(b >= a for a, b in zip(sizes, sizes[1:]))
                sizes = [L.hq_fp4_matmul_workspace_size(ref(w), n) for n in range(0, 300)]
                assert all(s > 0 for s in sizes) and all(b >= a for a, b in zip(sizes, sizes[1:]))
    g, d = mat(rows=8 * 256, K=512), mat(rows=8 * 512, K=256)
    sizes = [L.hq_fp4_experts_workspace_size(ref(g), ref(g), ref(d), 8, T, 4, HQ_BF16) for T in range(0, 3000, 7)]
    assert all(s > 0 for s in sizes) and all(b >= a for a, b in zip(sizes, sizes[1:]))
    sizes = [L.hq_moe_sort_workspace_size(T, 8, 256) for T in range(0, 20000, 13)]
    assert all(s > 0 for s in sizes) and all(b >= a for a, b in zip(sizes, sizes[1:]))


def test_linear_launches(L):
    assert L.hq_fp4_linear_launches(ref(mat(K=8192)), 1) == 1 and L.hq_fp4_linear_launches(ref(mat(K=8192)), 2) == 2
    assert L.hq_fp4_linear_launches(ref(mat(K=1024)), 8) == 1 and L.hq_fp4_linear_launches(ref(mat(K=32)), 9) == 2
    assert L.hq_fp4_linear_launches(ref(mat()), 0) == 0
    assert L.hq_fp4_experts_launches(32, 8) == 5 and L.hq_fp4_experts_launches(4096, 8) == 6
    assert L.hq_fp4_experts_launches(0, 8) == 0


def experts(L, **kw):
    a = dict(g=mat(rows=8 * 256), u=mat(rows=8 * 256), d=mat(rows=8 * 512, K=256), E=8, x=FAKE, xd=HQ_BF16, ldx=512, T=4, ids=FAKE,
             w=FAKE, k=2, xs=None, hs=None, y=FAKE, yd=HQ_BF16, ws=FAKE, n=1 << 40)
    a.update(kw)
    return L.hq_fp4_experts(ref(a["g"]), ref(a["u"]), ref(a["d"]), a["E"], a["x"], a["xd"], a["ldx"], a["T"], a["ids"], a["w"],
                            a["k"], a["xs"], a["hs"], a["y"], a["yd"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), HQ_ERR_INVALID_ARG), (dict(E=0), HQ_ERR_INVALID_ARG), (dict(E=3), HQ_ERR_INVALID_ARG), (dict(k=0), HQ_ERR_INVALID_ARG),
    (dict(T=-1), HQ_ERR_INVALID_ARG), (dict(u=mat(rows=8 * 128)), HQ_ERR_INVALID_ARG), (dict(d=mat(rows=8 * 512, K=512)), HQ_ERR_INVALID_ARG),
    (dict(d=mat(rows=8 * 256, K=256)), HQ_ERR_INVALID_ARG), (dict(u=mat(rows=8 * 256, format=HQ_FP4_MX)), HQ_ERR_INVALID_ARG),
    (dict(g=mat(rows=8 * 256, ts=FAKE, n=5)), HQ_ERR_INVALID_ARG), (dict(xd=4), HQ_ERR_INVALID_ARG), (dict(yd=-1), HQ_ERR_INVALID_ARG),
    (dict(x=None), HQ_ERR_INVALID_ARG), (dict(ldx=511), HQ_ERR_INVALID_ARG), (dict(ids=None), HQ_ERR_INVALID_ARG), (dict(w=FAKE + 1), HQ_ERR_INVALID_ARG),
    (dict(y=FAKE + 8), HQ_ERR_INVALID_ARG), (dict(xs=FAKE + 1), HQ_ERR_INVALID_ARG), (dict(hs=FAKE + 1), HQ_ERR_INVALID_ARG),
    (dict(k=33), HQ_ERR_UNSUPPORTED), (dict(T=(1 << 20) + 1), HQ_ERR_UNSUPPORTED), (dict(ws=None), HQ_ERR_WORKSPACE), (dict(n=1000), HQ_ERR_WORKSPACE),
    (dict(g=mat(rows=8 * 64), u=mat(rows=8 * 64), d=mat(rows=8 * 512, K=64)), HQ_ERR_UNSUPPORTED),
    (dict(g=mat(rows=2048 * 128), u=mat(rows=2048 * 128), d=mat(rows=2048 * 512, K=128), E=2048), HQ_ERR_UNSUPPORTED),
    (dict(T=0), HQ_OK),
])
def test_experts_rejects(L, kw, want):
    assert experts(L, **kw) == want


def test_routing_rejects(L):
    def sort(ids=FAKE, T=4, k=2, E=8, align=1, pos=FAKE, off=FAKE, cnt=FAKE, ws=FAKE, n=1 << 30):
        return L.hq_moe_sort(ids, T, k, E, align, pos, off, cnt, ws, n, None)
    for kw in (dict(T=-1), dict(k=0), dict(E=0), dict(align=0), dict(ids=None), dict(pos=FAKE + 2), dict(off=None), dict(cnt=FAKE + 1)):
        assert sort(**kw) == HQ_ERR_INVALID_ARG, kw
    for kw in (dict(k=33), dict(E=16385), dict(align=4097), dict(T=1 << 23)):
        assert sort(**kw) == HQ_ERR_UNSUPPORTED, kw
    assert sort(ws=None) == HQ_ERR_WORKSPACE and sort(n=255) == HQ_ERR_WORKSPACE
    assert L.hq_moe_sort_workspace_size(4, 33, 8) == 0 and L.hq_moe_sort_workspace_size(1 << 23, 2, 8) == 0

    def gather(x=FAKE, d=HQ_BF16, pos=FAKE, T=4, k=2, H=64, rows=FAKE, n=8):
        return L.hq_moe_gather(x, d, pos, T, k, H, rows, n, None)
    for kw in (dict(d=3), dict(T=-1), dict(k=0), dict(H=0), dict(n=-1), dict(x=None), dict(x=FAKE + 1), dict(pos=FAKE + 2), dict(rows=FAKE + 1)):
        assert gather(**kw) == HQ_ERR_INVALID_ARG, kw
    assert gather(k=33) == HQ_ERR_UNSUPPORTED and gather(H=(1 << 24) + 1) == HQ_ERR_UNSUPPORTED
    assert gather(T=0) == HQ_OK and gather(n=0) == HQ_OK

    def combine(z=FAKE, d=HQ_BF16, n=8, pos=FAKE, w=FAKE, T=4, k=2, H=64, y=FAKE, yd=HQ_BF16):
        return L.hq_moe_combine(z, d, n, pos, w, T, k, H, y, yd, None)
    for kw in (dict(z=None), dict(z=FAKE + 1), dict(pos=None), dict(w=FAKE + 2), dict(y=None), dict(yd=7), dict(yd=HQ_F32, y=FAKE + 2)):
        assert combine(**kw) == HQ_ERR_INVALID_ARG, kw
    assert combine(yd=HQ_F16) == HQ_ERR_UNSUPPORTED and combine(T=0) == HQ_OK

    def grad(dy=FAKE, d=HQ_F32, z=FAKE, n=8, pos=FAKE, w=FAKE, T=4, k=2, H=64, dz=FAKE, dw=FAKE):
        return L.hq_moe_combine_grad(dy, d, z, n, pos, w, T, k, H, dz, dw, None)
    for kw in (dict(dy=None), dict(z=FAKE + 2), dict(pos=None), dict(w=None), dict(dz=None), dict(dw=FAKE + 1), dict(n=-1)):
        assert grad(**kw) == HQ_ERR_INVALID_ARG, kw
    assert grad(T=0) == HQ_OK
