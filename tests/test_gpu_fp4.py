"""GPU parity of the microscaled 4-bit matrices (hq_fp4_*) against the 64-bit
oracle.

Codes and scales are decided in IEEE single precision on both sides and must
match bit for bit.  A product's operands are exact (codes times scales have at
most 6 significant bits, so every product of two is exact in fp32), which
leaves the sums: K terms in fp32, each addition off by at most an ulp of the
partial sum (the tensor cores may truncate, 2^-23), the two tensor scales
(3 roundings of 2^-24) and one rounding of the result to y's type:
  tol = ((K + 64) 2^-23 + 3 2^-24) sum_k |w_k a_k| + eps(y) / 2 (|y| + that) + tiny(y)
with tiny half a step of y's smallest numbers (2^-25 in fp16).
"""
import numpy as np
import pytest
import torch

from bit_hadamard_rotated_b200 import (Fp4Linear, Fp4Matrix, HqError, hq_fp4_linear, hq_fp4_matmul, hq_fp4_quantize,
                                       hq_fp4_tensor_scale, hq_launch_count, hq_rotate)
from oracle import fp4

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_hadamard_rotated_b200 import build
    build.build()


def rows(R, K, dtype, seed, scale=1.0):
    """N(0, 1) rows, 1 % of the channels x 20, a zero row, a zero block, exact
    multiples of small steps (ties between codes and between scales)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, K)) * scale
    x[:, rng.choice(K, max(1, K // 100), replace=False)] *= 20
    if R > 2:
        x[1] = 0
        x[2] = rng.integers(-24, 25, K) / 4 * scale
    x[0, :32] = 0
    return torch.from_numpy(x).to(dtype)


def bits(t):
    return t.cpu().numpy()


def check_quantised(q, x, fmt, ts=None):
    R, K = x.shape
    c, s, v = fp4.quantize(x.double().numpy(), fmt, ts)
    assert np.array_equal(bits(q.codes), fp4.pack(c))
    assert np.array_equal(bits(q.scales), fp4.tile(s))
    if q.values is not None:
        want = torch.from_numpy(v)
        got = q.values.cpu().double()
        # one rounding to x's type, after the fp32 product code * e (2^-24)
        tol = (torch.finfo(x.dtype).eps / 2 + 2.0**-24) * want.abs() * (1 + 2.0**-10) + 2.0**-149
        if x.dtype == torch.float16:
            tol = tol + 2.0**-25
        ok = ((got - want).abs() <= tol) | (torch.isnan(got) & torch.isnan(want))
        assert bool(ok.all())


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K", [(1, 32), (1, 8192), (3, 96), (33, 4128), (130, 160), (257, 1024), (5, 16384), (2501, 4096), (20001, 288)])
def test_quantize_bit_exact(fmt, dtype, R, K):
    x = rows(R, K, dtype, R + K)
    check_quantised(hq_fp4_quantize(x.cuda(), fmt, values=True), x, fmt)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ts", [1.0, 0.0073, 3.1e-5, 2.0**-40, 2.0**90])
def test_quantize_tensor_scale_bit_exact(dtype, ts):
    x = rows(40, 512, dtype, 7, scale=min(ts * 50, 1000.0))
    t = torch.tensor(ts, dtype=torch.float32, device="cuda")
    q = hq_fp4_quantize(x.cuda(), "nv", tensor_scale=t, values=dtype == torch.float32)
    check_quantised(q, x, "nv", ts)


def test_quantize_every_tie_and_neighbour():
    """fp32 values on and one ulp beside every border between codes, for every
    E4M3 block scale: the quotient's last bit decides."""
    mids = (fp4.GRID[1:] + fp4.GRID[:-1]) / 2
    x = np.zeros((126, 32), dtype=np.float32)
    for r, s in enumerate(fp4._E4M3[1:]):
        m = (mids * s).astype(np.float32)
        x[r, 0] = x[r, 16] = 6 * s
        x[r, 1:8], x[r, 8:15] = m, np.nextafter(m, np.float32(np.inf))
        x[r, 17:24], x[r, 24:31] = -m, -np.nextafter(m, np.float32(0))
    t = torch.from_numpy(x)
    check_quantised(hq_fp4_quantize(t.cuda(), "nv"), t, "nv")
    u = t * 1.37e-3
    ts = 1.37e-3
    check_quantised(hq_fp4_quantize(u.cuda(), "nv", tensor_scale=torch.tensor(ts, device="cuda")), u, "nv", ts)


def test_quantize_extremes():
    """Subnormals, the largest values, infinities, NaN, negative zeros."""
    x = np.zeros((8, 64), dtype=np.float32)
    x[0, :16] = 2.0**-149
    x[1] = np.linspace(-3.4e38, 3.4e38, 64)
    x[2, 5], x[3, 40], x[4, 63] = np.inf, -np.inf, np.nan
    x[2, 20:], x[5] = 1.0, -0.0
    x[6, :32], x[6, 32:] = 2.0**-126, 1e-30
    x[7] = np.linspace(-1e-3, 1e-3, 64)
    t = torch.from_numpy(x)
    for fmt in ("nv", "mx"):
        check_quantised(hq_fp4_quantize(t.cuda(), fmt, values=True), t, fmt)


def test_quantize_strided_rows_and_refusals():
    big = rows(20, 512, torch.bfloat16, 3).cuda()
    part = big[:, 128:416]
    a, b = hq_fp4_quantize(part, "mx"), hq_fp4_quantize(part.contiguous(), "mx")
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    odd = big[:, 1:129]  # rows off 16-byte boundaries: copied by the binding
    assert torch.equal(hq_fp4_quantize(odd).codes, hq_fp4_quantize(odd.contiguous()).codes)
    with pytest.raises(HqError):
        hq_fp4_quantize(big[:, :48].contiguous())
    with pytest.raises(ValueError):
        hq_fp4_quantize(big, "mx", tensor_scale=torch.ones((), device="cuda"))
    with pytest.raises(ValueError):
        hq_fp4_quantize(big.double())
    n0 = hq_launch_count()
    q = hq_fp4_quantize(big[:0])
    assert q.codes.shape == (0, 256) and q.scales.shape[0] == 0 and hq_launch_count() == n0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K", [(1, 32), (77, 4128), (3000, 2048)])
def test_tensor_scale(dtype, R, K):
    x = rows(R, K, dtype, R, 0.02).cuda()
    want = np.float32(x.double().abs().max().item() / 2688.0 or 1)
    assert hq_fp4_tensor_scale(x).item() == want
    assert hq_fp4_tensor_scale(torch.zeros_like(x)).item() == 1.0
    assert hq_fp4_tensor_scale(x[:, :32]).item() == np.float32(x[:, :32].double().abs().max().item() / 2688.0 or 1)


# ------------------------------------------------------------------ products


def weight(M, K, fmt, seed, scaled):
    w = rows(M, K, torch.float32, seed, K**-0.5).cuda()
    ts = hq_fp4_tensor_scale(w) if scaled else None
    return hq_fp4_quantize(w, fmt, tensor_scale=ts)


def dense(q):
    ts = None if q.tensor_scale is None else q.tensor_scale.cpu().numpy()
    return fp4.values(bits(q.codes), bits(q.scales), q.fmt, ts)


def check_product(y, W, A, K):
    want, base = A @ W.T, np.abs(A) @ np.abs(W).T
    eps = torch.finfo(y.dtype).eps
    sums = ((K + 64) * 2.0**-23 + 3 * 2.0**-24) * base
    tol = sums + eps / 2 * (np.abs(want) + sums) + (2.0**-25 if y.dtype == torch.float16 else 2.0**-149)
    got = y.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= tol), f"worst err/tol {np.max(err / tol):.3g} at {np.unravel_index(np.argmax(err / tol), err.shape)}"


SHAPES = [  # M, K, N
    (128, 256, 16), (128, 256, 1), (1, 32, 1), (128, 64, 32), (128, 32, 8), (300, 96, 5), (128, 1024, 64), (384, 512, 33),
    (4100, 4128, 2), (640, 8192, 1), (128, 2048, 128), (257, 1056, 129), (512, 512, 256), (1000, 736, 333), (2304, 4096, 70),
    (129, 16384, 3), (256, 288, 1025), (20000, 256, 7),
    (9473, 544, 400), (4000, 1312, 1025), (19200, 64, 300),  # tiles of two CTAs
    (512, 8192, 100), (300, 6432, 40), (200, 3872, 20), (130, 32768, 1),  # parts of K
]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_matmul_parity(fmt, M, K, N):
    w = weight(M, K, fmt, M + K, fmt == "nv")
    x = rows(N, K, torch.bfloat16, N).cuda()
    a = hq_fp4_quantize(x, fmt)
    y = hq_fp4_matmul(w, a)
    torch.cuda.synchronize()
    check_product(y, dense(w), dense(a), K)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out", DTYPES)
def test_linear_types(fmt, dtype, out):
    M, K, N = 520, 1312, 37
    w = weight(M, K, fmt, 5, fmt == "nv")
    x = rows(N, K, dtype, 6)
    xs = 0.031 if fmt == "nv" else None
    t = None if xs is None else torch.tensor(xs, device="cuda")
    y = hq_fp4_linear(w, x.cuda(), x_scale=t, out_dtype=out)
    assert y.dtype == out
    check_product(y, dense(w), fp4.quantize(x.double().numpy(), fmt, xs)[2], K)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_equals_quantise_then_matmul(fmt, M, K, N):
    """The layer's early weight reads change nothing; one layer and workspace for falling and rising batches."""
    w = weight(M, K, fmt, M + K + 1, False)
    layer = Fp4Linear(w, out_dtype=torch.float32)
    x = rows(max(N, 3), K, torch.float16, N).cuda()
    for n in (N, 1, N, min(N, 3)):
        got = layer(x[:n])
        assert torch.equal(got, hq_fp4_matmul(w, hq_fp4_quantize(x[:n], fmt)))
    layer.check_status()


def test_weights_packed_just_before_the_call():
    """Packing and multiplying back to back, over and over on one stream, with the weights' buffers reused."""
    ws = [rows(512, 2048, torch.float32, s, 0.03).cuda() for s in range(6)]
    x = rows(4, 2048, torch.float32, 9).cuda()
    want = [hq_fp4_matmul(hq_fp4_quantize(w), hq_fp4_quantize(x)).clone() for w in ws]
    torch.cuda.synchronize()
    for _ in range(5):
        for w, y in zip(ws, want):
            assert torch.equal(hq_fp4_linear(hq_fp4_quantize(w), x), y)


def test_nan_and_infinity_reach_their_rows_only():
    w = weight(200, 512, "nv", 1, False)
    x = rows(40, 512, torch.float32, 2)
    x[7, 100], x[9, 3], x[20, 511] = float("nan"), float("inf"), -float("inf")
    y = hq_fp4_linear(w, x.cuda()).cpu()
    bad = torch.isnan(y).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 9, 20]
    assert bool(torch.isfinite(y[~bad]).all())


def test_strided_output_and_rows():
    w = weight(300, 512, "mx", 3, False)
    big = rows(50, 1024, torch.bfloat16, 4).cuda()
    out = torch.full((50, 400), 7.0, device="cuda")
    y = hq_fp4_linear(w, big[:, 256:768], out=out[:, 50:350])
    assert torch.equal(y, hq_fp4_linear(w, big[:, 256:768].contiguous(), out_dtype=torch.float32))
    assert bool((out[:, :50] == 7).all()) and bool((out[:, 350:] == 7).all())


def test_repeats_are_equal_and_streams_are_kept():
    w = weight(2048, 4096, "nv", 8, True)
    x = rows(5, 4096, torch.bfloat16, 9).cuda()
    want = hq_fp4_linear(w, x)
    layers = [Fp4Linear(w), Fp4Linear(w)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for lay, st in zip(layers, streams):
            with torch.cuda.stream(st):
                got.append(lay(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_captured_and_replayed():
    w = weight(1024, 2048, "nv", 10, True)
    layer = Fp4Linear(w)
    x = rows(3, 2048, torch.bfloat16, 11).cuda()
    y = torch.empty(3, 1024, dtype=torch.bfloat16, device="cuda")
    layer(x, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, out=y)
    for s in range(4):
        x.copy_(rows(3, 2048, torch.bfloat16, 20 + s))
        g.replay()
        assert torch.equal(y, hq_fp4_linear(w, x))


def test_captured_graph_outlives_a_larger_batch():
    """A graph of a small batch, then larger eager batches of the same layer (its workspace grows), then the graph again."""
    w = weight(1024, 8192, "nv", 12, True)
    layer = Fp4Linear(w)
    x = rows(3, 8192, torch.bfloat16, 13).cuda()
    y = layer(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, out=y)
    want = hq_fp4_linear(w, x)
    for n in (40, 100, 700):
        big = rows(n, 8192, torch.bfloat16, n).cuda()
        assert torch.equal(layer(big), hq_fp4_linear(w, big))
        junk = [torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]  # would take freed memory
        y.zero_()
        g.replay()
        assert torch.equal(y, want)
        del junk
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            Fp4Linear(w)(x, out=y)
    assert torch.equal(layer(x), want)


def test_layer_is_ready_again_after_a_device_error():
    """A status word and counters as a call whose wait ran out leaves them, in the workspace in use and in one that a
    captured graph still uses: reported, and the next call and replay are right."""
    w = weight(512, 8192, "nv", 14, True)  # parts of K: arrivals are counted
    layer = Fp4Linear(w)
    x = rows(100, 8192, torch.bfloat16, 15).cuda()
    small = layer(x[:30])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x[:30], out=small)
    want, want_small = layer(x), hq_fp4_linear(w, x[:30])
    layer.check_status()
    assert len(layer._outgrown) == 1
    for ws in (layer._ws, layer._outgrown[0]):
        ws[:4].view(torch.int32).fill_(1)
        ws[256:8448].view(torch.int32).fill_(1)
        with pytest.raises(HqError):
            layer.check_status()
        layer.check_status()
        small.zero_()
        g.replay()
        assert torch.equal(layer(x), want) and torch.equal(small, want_small)


def test_two_layers_at_once():
    """Pairs of CTAs, parts of K, one launch and two, on two streams."""
    ws = [weight(4096, 8192, "nv", 16, True), weight(9600, 2048, "mx", 17, False)]
    xs = [rows(n, w.K, torch.bfloat16, n).cuda() for w in ws for n in (1, 20, 700)]
    want = [hq_fp4_linear(ws[i // 3], x) for i, x in enumerate(xs)]
    layers = [Fp4Linear(w) for w in ws]
    for i in (2, 5):
        layers[i // 3](xs[i])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, x in enumerate(xs):
            got.append((i, layers[i // 3](x, stream=streams[i // 3])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
    for lay in layers:
        lay.check_status()


def test_given_stream():
    """Calls on a stream that is not the current one: their copies, allocations and zeroed workspaces belong to it."""
    w = weight(512, 8192, "mx", 14, False)
    big = rows(6, 8200, torch.float32, 15).cuda()
    x = big[:, 1:8193]  # rows off 16-byte boundaries: copied
    want = hq_fp4_linear(w, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [hq_fp4_linear(w, x, stream=s) for _ in range(20)]
    q = hq_fp4_quantize(x, "mx", stream=s)
    got += [hq_fp4_matmul(w, q, stream=s)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_rotated_basis():
    """Rotate, pack and multiply: (H W)(H x) = W x, so the packed product in the rotated basis is near W x."""
    M, K, N = 256, 2048, 4
    rng = np.random.default_rng(0)
    s = torch.from_numpy((rng.integers(0, 2, K) * 2 - 1).astype(np.int8)).cuda()
    W, x = rows(M, K, torch.float32, 1, K**-0.5).cuda(), rows(N, K, torch.float32, 2).cuda()
    wr, xr = hq_rotate(W, s), hq_rotate(x, s)
    w = hq_fp4_quantize(wr, "nv", tensor_scale=hq_fp4_tensor_scale(wr))
    a = hq_fp4_quantize(xr)
    y = hq_fp4_matmul(w, a)
    check_product(y, dense(w), dense(a), K)
    # each factor is off by at most half a step: 1/4 of its block's effective scale below 2, 1/2 below 4, 1 below 6,
    # so by at most 1/6 of the block's largest magnitude and the scale's own rounding (2^-4) on saturated values
    want = (x.double() @ W.double().T).cpu().numpy()
    Wd, Ad = dense(w), dense(a)
    dW, dA = np.abs(Wd - wr.double().cpu().numpy()), np.abs(Ad - xr.double().cpu().numpy())
    bound = dA @ np.abs(Wd).T + np.abs(xr.double().cpu().numpy()) @ dW.T
    rot = (14 * 2.0**-24) * (np.abs(x.double().cpu().numpy()).sum(1)[:, None] * np.abs(W.double().cpu().numpy()).sum(1)[None])
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= bound * (1 + 1e-6) + rot + 1e-4)


def test_matmul_refusals():
    w = weight(128, 256, "nv", 1, False)
    a = hq_fp4_quantize(rows(4, 256, torch.float32, 2).cuda())
    with pytest.raises(HqError):
        hq_fp4_matmul(w, hq_fp4_quantize(rows(4, 256, torch.float32, 2).cuda(), "mx"))
    with pytest.raises(HqError):
        hq_fp4_matmul(w, hq_fp4_quantize(rows(4, 512, torch.float32, 2).cuda()))
    with pytest.raises(HqError):
        hq_fp4_matmul(w, a, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        hq_fp4_matmul(w, a, out=torch.empty(4, 100, device="cuda"))
    with pytest.raises(ValueError):
        hq_fp4_linear(w, torch.zeros(4, 128, device="cuda"))
    with pytest.raises(ValueError):
        Fp4Matrix(w.codes, w.scales[:, :1].contiguous())
    n0 = hq_launch_count()
    assert hq_fp4_linear(w, torch.zeros(0, 256, device="cuda")).shape == (0, 128) and hq_launch_count() == n0


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^32, against the same rows on their own."""
    R, K = 140000, 32768
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    last = rows(300, K, torch.bfloat16, 18).cuda()
    x[-300:] = last
    x[5, 7] = 1.0
    ts = hq_fp4_tensor_scale(x)
    assert torch.equal(ts, hq_fp4_tensor_scale(last))
    q, want = hq_fp4_quantize(x, tensor_scale=ts, values=True), hq_fp4_quantize(last, tensor_scale=ts, values=True)
    assert torch.equal(q.codes[-300:], want.codes) and torch.equal(q.values[-300:], want.values)
    w = weight(256, K, "nv", 19, True)  # codes and scales of tokens past 2^31 bytes
    y = hq_fp4_matmul(w, q)
    check_product(y[-300:], dense(w), dense(want), K)  # (300 rows on their own are summed in parts of K)
    assert bool((y[6:-300] == 0).all())
    del x, q, y

    w, N = weight(16000, 64, "mx", 20, False), 300000
    x = torch.zeros(N, 64, dtype=torch.bfloat16, device="cuda")
    x[-300:] = rows(300, 64, torch.bfloat16, 21).cuda()
    y = hq_fp4_linear(w, x)
    assert torch.equal(y[-300:], hq_fp4_linear(w, x[-300:])) and bool((y[-500:-300] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("amax,ts", [(1e30, 1e-10), (1e25, 1e-15), (2.0**122, 1e-5), (2.0**120, 2.0**-20), (2.0**100, 2.0**-99),
                                     (3e38, 2.0**-30), (2.0**127, 2.0**-126), (2.0**60, 2.0**-90), (1e30, 1e-6)])
def test_quantize_with_a_tensor_scale_far_too_small(dtype, amax, ts):
    """Quotients past fp32's range: block scales end at 448, codes at 6 with the sign of x."""
    ts = float(np.float32(ts))
    x = np.zeros((5, 64))
    x[0] = np.linspace(-1, 1, 64) * amax
    x[1], x[1, 3], x[1, 40] = 0.0, -amax, amax  # one large value beside zeros
    x[2] = np.linspace(1, -1, 64) * 2000 * ts    # within the scale's range
    x[3, ::2], x[3, 1::2] = -amax, 3 * ts
    x[4] = -amax * np.exp2(-np.arange(64.0))
    x = torch.from_numpy(x).to(dtype)
    q = hq_fp4_quantize(x.cuda(), "nv", tensor_scale=torch.tensor(ts, device="cuda"), values=dtype == torch.float32)
    check_quantised(q, x, "nv", ts)
    w = hq_fp4_quantize(rows(130, 64, torch.float32, 30, 0.1).cuda())
    for n in (5, 2):  # quantised by the product's own CTAs, and by a kernel before it
        big = x[:n].repeat(40 if n == 5 else 1, 1)
        y = hq_fp4_linear(w, big.cuda(), x_scale=torch.tensor(ts, device="cuda"), out_dtype=torch.float32)
        check_product(y, dense(w), fp4.quantize(big.double().numpy(), "nv", ts)[2], 64)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ts", [None, 0.01])
def test_zeros_keep_their_sign(fmt, dtype, ts):
    """Negative zeros, and negative values that round to zero, beside values that do not."""
    if fmt == "mx" and ts is not None:
        pytest.skip("a tensor scale is NV's")
    x = torch.zeros(6, 96, dtype=dtype)
    x[0, ::3], x[0, 1::3] = -0.0, 1.5
    x[1] = -0.0
    x[1, 17] = -2.0
    x[2, 1::2], x[2, ::2] = -1e-7, 3.0
    x[3, ::2], x[3, 5] = -torch.finfo(dtype).tiny, 700.0
    x[4] = -x[0]
    x[5, 40] = 1.0
    t = None if ts is None else torch.tensor(ts, device="cuda")
    q = hq_fp4_quantize(x.cuda(), fmt, tensor_scale=t, values=True)
    check_quantised(q, x, fmt, None if ts is None else float(np.float32(ts)))
    got, want = q.values.cpu(), fp4.quantize(x.double().numpy(), fmt, ts)[2]
    assert np.array_equal(torch.signbit(got).numpy(), np.signbit(want))


@pytest.mark.parametrize("M,K,N", [(130, 64, 3), (300, 288, 40), (512, 16384, 100), (9473, 96, 400)])  # every kind of launch
@pytest.mark.parametrize("ew,ea", [(66, 66), (-75, -75), (-100, -40), (100, -100), (-60, 120)])
def test_tensor_scales_whose_product_leaves_fp32(M, K, N, ew, ea):
    """Two tensor scales 2^ew and 2^ea, results within fp32's normal range, and rows of zeros, which stay zeros."""
    size = 2.0**-9 if ew + ea > 100 else 256.0 if ew + ea < -100 else 1.0  # so that the results fit
    rng = np.random.default_rng(M + N)
    W = rng.integers(-4, 5, (M, K)) * 2.0**ew * size
    X = rng.integers(-4, 5, (N, K)) * 2.0**ea * size
    if ew + ea > 100:
        W[:, 8:], X[:, 8:] = 0, 0
    X[N // 2], W[M // 2] = 0, 0
    tw, ta = (torch.tensor(2.0**e, dtype=torch.float32, device="cuda") for e in (ew, ea))
    w = hq_fp4_quantize(torch.from_numpy(W).float().cuda(), tensor_scale=tw)
    x = torch.from_numpy(X).float().cuda()
    A = fp4.quantize(x.double().cpu().numpy(), "nv", 2.0**ea)[2]
    want = A @ dense(w).T
    y = hq_fp4_linear(w, x, x_scale=ta)
    a = hq_fp4_quantize(x, tensor_scale=ta)
    for got in (y, hq_fp4_matmul(w, a)):
        got = got.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        sums = (K + 64) * 2.0**-23 * (np.abs(A) @ np.abs(dense(w)).T)
        assert np.all(np.abs(got - want) <= sums + 3 * 2.0**-24 * np.abs(want) + 3 * 2.0**-150)
        assert np.any(got != 0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_row_of_an_odd_pitch(dtype):
    """A single row of a wider buffer, whose pitch is no multiple of 16 bytes, on and off 16-byte boundaries; a row of a
    narrower one."""
    w = weight(260, 512, "nv", 31, False)
    big = rows(4, 513, dtype, 32).cuda()
    for x in (big[:1, :512], big[1:2, :512], big[:1, 1:], big[3:, 1:], big.t().contiguous().t()[2:3, :512]):
        c = x.clone(memory_format=torch.contiguous_format).reshape(-1).clone().reshape(1, 512)
        a, b = hq_fp4_quantize(x), hq_fp4_quantize(c)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        assert torch.equal(hq_fp4_tensor_scale(x), hq_fp4_tensor_scale(c))
        want = hq_fp4_matmul(w, b)
        assert torch.equal(hq_fp4_linear(w, x, out_dtype=torch.float32), want)
        assert torch.equal(Fp4Linear(w, out_dtype=torch.float32)(x), want)
        flat = torch.as_strided(c, (1, 512), (1, 1))  # a pitch of 1
        assert torch.equal(hq_fp4_linear(w, flat, out_dtype=torch.float32), want)


def test_outgrown_workspaces_are_given_back():
    """Without a captured graph a layer holds the workspace of its largest call and no other, also when it grows on
    another stream than the one that it started on, with calls still running."""
    from bit_hadamard_rotated_b200 import fp4 as binding
    w = weight(1024, 8192, "nv", 33, True)
    big = rows(3000, 8192, torch.bfloat16, 34).cuda()
    sizes = (20, 33, 100, 700, 1500, 3000)
    want = [hq_fp4_linear(w, big[:n]) for n in sizes]
    layer = Fp4Linear(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for i, n in enumerate(sizes):
        here = torch.cuda.current_stream() if i % 2 == 0 else s
        other = s if i % 2 == 0 else torch.cuda.current_stream()
        for _ in range(8):
            got.append((i, layer(big[:n], stream=here)))
        other.wait_stream(here)
        # what would take the workspace's memory if it were free for the stream that it came from
        with torch.cuda.stream(other):
            junk = [torch.full((layer._ws.numel(),), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        need = int(binding.lib().hq_fp4_linear_workspace_size(w._ref, n))
        assert layer._ws.numel() == need and layer._outgrown == []
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
    layer.check_status()


def test_workspaces_of_captured_graphs_only_are_kept():
    w = weight(1024, 8192, "nv", 35, True)
    layer = Fp4Linear(w)
    x = rows(900, 8192, torch.bfloat16, 36).cuda()
    layer(x[:3])
    y = layer(x[:40])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x[:40], out=y)
    held = layer._ws
    for n in (100, 400, 900):
        layer(x[:n])
    assert len(layer._outgrown) == 1 and layer._outgrown[0] is held
    y.zero_()
    g.replay()
    assert torch.equal(y, hq_fp4_linear(w, x[:40]))


def test_growing_keeps_the_status():
    """A device error recorded before the workspace grew is still reported."""
    w = weight(512, 8192, "nv", 37, True)
    layer = Fp4Linear(w)
    x = rows(300, 8192, torch.bfloat16, 38).cuda()
    layer(x[:3])
    layer._ws[:4].view(torch.int32).fill_(1)
    layer(x)
    with pytest.raises(HqError):
        layer.check_status()
    layer.check_status()
    assert torch.equal(layer(x), hq_fp4_linear(w, x))


def test_two_host_threads():
    """Layers of different widths (the fused launch's shared memory goes by K) and sorts of different numbers of
    experts, called by two threads at once on their own streams."""
    from concurrent.futures import ThreadPoolExecutor

    from bit_hadamard_rotated_b200 import hq_moe_sort
    torch.cuda.synchronize()

    def work(K, E):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            w = weight(128, K, "nv", K, False)
            x = rows(1, K, torch.bfloat16, K).cuda()
            layer = Fp4Linear(w)
            ids = torch.arange(64, dtype=torch.int32, device="cuda").remainder(E).view(8, 8)
            want, pos = layer(x).clone(), hq_moe_sort(ids, E).pos.clone()
            good = torch.ones((), dtype=torch.bool, device="cuda")
            for _ in range(1500):
                y, p = layer(x), hq_moe_sort(ids, E).pos
            good &= (y == want).all() & (p == pos).all()
            return bool(good)

    with ThreadPoolExecutor(2) as ex:
        assert all(f.result() for f in [ex.submit(work, 256, 900), ex.submit(work, 8192, 16384)])


def test_shared_memory_limits_of_two_host_threads():
    """The C entry called in tight loops by four threads, with much and with little shared memory for one kernel."""
    from concurrent.futures import ThreadPoolExecutor

    from bit_hadamard_rotated_b200._lib import lib
    L = lib()

    def work(E):
        ids = torch.zeros(4, dtype=torch.int32, device="cuda")
        out = torch.empty(4 + 2 * E + 1, dtype=torch.int32, device="cuda")
        ws = torch.empty(L.hq_moe_sort_workspace_size(4, 1, E), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        p = out.data_ptr()
        a = (ids.data_ptr(), 4, 1, E, 1, p, p + 16, p + 16 + 4 * (E + 1), ws.data_ptr(), ws.numel(), s.cuda_stream)
        bad = sum(L.hq_moe_sort(*a) != 0 for _ in range(3000))
        s.synchronize()
        return bad, out[:4].tolist() == [0, 1, 2, 3]

    with ThreadPoolExecutor(4) as ex:
        assert list(ex.map(work, (900, 16384, 1000, 16000))) == [(0, True)] * 4
