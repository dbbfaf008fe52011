"""GPU parity of the packed expert layer (hq_fp4_experts).

Both products are those of hq_fp4_matmul (checked on their own) on the same
packed rows, so g and u are taken from it in fp32 and the rest is followed in
64 bits.  What the layer may add:
  - h = g / (1 + exp(-g)) u: the fast exponential is within 2 + 1.173 |g| ulps
    and the fast division within 2, plus three products: relative
    (8 + 1.2 |g|) 2^-23;
  - h that close to a border between two codes, or a block's largest h to one
    between two scales, may be packed either way: every packing of the interval
    is allowed, D_i the largest difference of value i;
  - d: sum_i |w_i| D_i, K = inter fp32 additions as in hq_fp4_matmul, one
    rounding to y's type; y: k products and sums in fp32 and one rounding.
"""
import numpy as np
import pytest
import torch

from bit_hadamard_rotated_b200 import (Fp4Experts, Fp4Matrix, HqError, hq_fp4_matmul, hq_fp4_quantize,
                                       hq_fp4_tensor_scale, hq_launch_count)
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_hadamard_rotated_b200 import build
    build.build()


def bits(t):
    return t.cpu().numpy()


def rnd(shape, seed, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale).float()


def pack_experts(E, rows, K, fmt, seed):
    """One stacked matrix with a tensor scale per expert ("nv")."""
    w = rnd((E * rows, K), seed, K**-0.5).cuda()
    if fmt == "mx":
        return hq_fp4_quantize(w, "mx")
    parts = []
    for e in range(E):
        p = w[e * rows:(e + 1) * rows]
        parts.append(hq_fp4_quantize(p, "nv", tensor_scale=hq_fp4_tensor_scale(p)))
    return Fp4Matrix(torch.cat([p.codes for p in parts]), torch.cat([p.scales for p in parts]), "nv",
                     torch.stack([p.tensor_scale for p in parts]))


def expert(m, e, rows):
    ts = None if m.tensor_scale is None else m.tensor_scale[e:e + 1]
    return Fp4Matrix(m.codes[e * rows:(e + 1) * rows].contiguous(),
                     m.scales[e * rows // 128:(e + 1) * rows // 128].contiguous(), m.fmt, ts)


def dense(m):
    return fp4.values(bits(m.codes), bits(m.scales), m.fmt, None if m.tensor_scale is None else bits(m.tensor_scale))


def values_at(h, fmt, scale_from, ts):
    """h packed with the block scales of `scale_from`."""
    n = fp4.BLOCK[fmt]
    t = np.float64(1 if ts is None else np.float32(ts))
    amax = np.abs(scale_from).reshape(h.shape[0], -1, n).max(2)
    if fmt == "nv":
        eff = fp4.e4m3_decode(fp4.e4m3_encode((amax / np.float64(np.float32(6 * t))).astype(np.float32).astype(np.float64)))
        eff = (eff * t).astype(np.float32).astype(np.float64)
    else:
        _, e = np.frexp(amax)
        eff = np.exp2(np.where(amax > 0, np.maximum(e - 3, -127), -127).astype(np.float64))
    b = h.reshape(h.shape[0], -1, n)
    with np.errstate(all="ignore"):
        q = np.where(eff[..., None] > 0, b / eff[..., None], 0.0)
    c = fp4.e2m1_encode(q.astype(np.float32).astype(np.float64))
    return (np.where(c >= 8, -1.0, 1.0) * fp4.GRID[c & 7] * eff[..., None]).reshape(h.shape)


def check_layer(layer, gate, up, down, E, x, ids, w, y, x_scale=None, h_scale=None):
    T, k = ids.shape
    H, I, fmt = gate.K, down.K, gate.fmt
    dt = y.dtype
    eps = torch.finfo(dt).eps
    small = 2.0**-25 if dt == torch.float16 else 2.0**-149
    want, tol, mags = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    xs = None if x_scale is None else x_scale.item()
    hs = None if h_scale is None else h_scale.item()
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        a = hq_fp4_quantize(x[torch.from_numpy(t).cuda()], fmt, tensor_scale=x_scale)
        g, u = (bits(hq_fp4_matmul(expert(m, e, I), a)).astype(np.float64) for m in (gate, up))
        h = g / (1 + np.exp(-g)) * u
        d = (8 + 1.2 * np.abs(g)) * 2.0**-23 * np.abs(h)
        hi, lo = np.abs(h) + d, np.maximum(np.abs(h) - d, 0)
        v = values_at(h, fmt, h, hs)
        D = np.zeros_like(h)
        for scale_from in (lo, hi):
            for end in (h - d, h + d):
                D = np.maximum(D, np.abs(values_at(end, fmt, scale_from, hs) - v))
        W = dense(expert(down, e, H))
        out, base = v @ W.T, np.abs(v) @ np.abs(W).T
        err = D @ np.abs(W).T + ((I + 64) * 2.0**-23 + 3 * 2.0**-24) * base
        err += eps / 2 * (np.abs(out) + err) + small
        wt = w[t, j].astype(np.float64)[:, None]
        np.add.at(want, t, wt * out)
        np.add.at(tol, t, np.abs(wt) * err)
        np.add.at(mags, t, np.abs(wt) * (np.abs(out) + err))
    tol += (2 * k + 1) * 2.0**-24 * mags
    tol += eps / 2 * (np.abs(want) + tol) + small
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= tol), float(np.max(err / tol))
    layer.check_status()
    return xs


def make(E, H, I, fmt, seed=0):
    return [pack_experts(E, r, K, fmt, seed + i) for i, (r, K) in enumerate([(I, H), (I, H), (H, I)])]


def route(T, k, E, seed, masked=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]).astype(np.int32)
    if masked:
        ids[rng.random(T) < masked] = -1
        ids[0, 0] = E
    return ids, rng.random((T, k)).astype(np.float32)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("T,k,E,H,I,masked", [
    (1, 1, 1, 128, 128, 0), (1, 8, 16, 256, 128, 0), (5, 2, 3, 384, 256, 0.3), (32, 8, 24, 512, 384, 0),
    (200, 3, 4, 256, 640, 0.2), (700, 2, 3, 640, 128, 0), (130, 1, 1, 2048, 512, 0), (129, 4, 300, 128, 128, 0),
])
def test_layer_parity(fmt, T, k, E, H, I, masked):
    m = make(E, H, I, fmt, T + E)
    layer = Fp4Experts(*m, E)
    x = rnd((T, H), 5).bfloat16().cuda()
    ids, w = route(T, k, E, T, masked)
    y = layer(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    assert y.dtype == torch.bfloat16
    check_layer(layer, *m, E, x, ids, w, y)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_layer_types_and_scales(dtype):
    E, H, I, T, k = 6, 256, 256, 40, 3
    m = make(E, H, I, "nv", 7)
    xs, hs = (torch.tensor(v, device="cuda") for v in (0.01, 0.003))
    layer = Fp4Experts(*m, E, x_scale=xs, h_scale=hs)
    x = rnd((T, H), 1).to(dtype).cuda()
    ids, w = route(T, k, E, 3)
    y = layer(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    check_layer(layer, *m, E, x, ids, w, y, xs, hs)


def test_masked_tokens_get_zeros_and_repeats_are_equal():
    E, H, I = 5, 256, 128
    m = make(E, H, I, "nv")
    layer = Fp4Experts(*m, E)
    x = rnd((50, H), 1).cuda()
    ids, w = route(50, 4, E, 2)
    ids[10:20] = -1
    a = [torch.from_numpy(v).cuda() for v in (ids, w)]
    y = layer(x, *a)
    assert bool((y[10:20] == 0).all()) and bool((y[:10] != 0).any(1).all())
    # other batches in between, then the same again
    layer(x[:3], a[0][:3], a[1][:3])
    big = x.repeat(4, 1)
    layer(big, a[0].repeat(4, 1), a[1].repeat(4, 1))
    assert torch.equal(layer(x, *a), y)
    ids[:] = -1
    assert bool((layer(x, torch.from_numpy(ids).cuda(), a[1]) == 0).all())


@pytest.mark.parametrize("T,k,E", [(900, 2, 1024), (23000, 4, 1000), (1, 1, 1024), (2000, 1, 700)])
def test_many_experts_few_of_them_busy(T, k, E):
    """More experts than threads, runs of empty ones at both ends and between, one with many tiles."""
    H = I = 128
    m = make(E, H, I, "nv", T)
    layer = Fp4Experts(*m, E)
    x = rnd((T, H), 6).bfloat16().cuda()
    rng = np.random.default_rng(T)
    ids = rng.choice([3, 360, 361, E - 2], (T, k), p=[0.1, 0.6, 0.2, 0.1]).astype(np.int32)
    some = rng.random((T, k)) < 0.2
    ids[some] = rng.integers(40, E - 40, some.sum()) // 3 * 3
    w = rng.random((T, k)).astype(np.float32)
    y = layer(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    check_layer(layer, *m, E, x, ids, w, y)


def test_one_expert_twice_in_a_token_and_all_tokens_to_one():
    E, H, I, T = 4, 128, 256, 33
    m = make(E, H, I, "mx")
    layer = Fp4Experts(*m, E)
    x = rnd((T, H), 1).half().cuda()
    ids = np.full((T, 3), 2, dtype=np.int32)
    w = np.random.default_rng(0).random((T, 3)).astype(np.float32)
    y = layer(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda())
    check_layer(layer, *m, E, x, ids, w, y)


def test_captured_and_replayed():
    E, H, I, T = 8, 256, 128, 16
    m = make(E, H, I, "nv")
    layer = Fp4Experts(*m, E)
    x = rnd((T, H), 1).bfloat16().cuda()
    ids, w = (torch.from_numpy(v).cuda() for v in route(T, 4, E, 1))
    y = torch.empty_like(x)
    layer(x, ids, w, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(x, ids, w, out=y)
    fresh = Fp4Experts(*m, E)
    for s in range(3):
        x.copy_(rnd((T, H), 10 + s))
        ids.copy_(torch.from_numpy(route(T, 4, E, 20 + s, 0.2 * s)[0]))
        g.replay()
        assert torch.equal(y, fresh(x, ids, w))


def test_refusals():
    m = make(2, 256, 128, "nv")
    with pytest.raises(ValueError):
        Fp4Experts(m[0], m[1], m[0], 2)
    with pytest.raises(ValueError):
        Fp4Experts(*m, 3)
    layer = Fp4Experts(*m, 2)
    x, ids, w = torch.zeros((4, 256), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError):
        layer(x, ids.long(), w)
    with pytest.raises(ValueError):
        layer(x, ids[:3], w)
    with pytest.raises(ValueError):
        layer(x[:, :128], ids, w)
    with pytest.raises(HqError):
        layer(x, torch.zeros((4, 33), dtype=torch.int32, device="cuda"), torch.zeros((4, 33), device="cuda"))
    n0 = hq_launch_count()
    assert layer(x[:0], ids[:0], w[:0]).shape == (0, 256) and hq_launch_count() == n0


def test_outputs_are_rounded_once():
    """A 16-bit y is the fp32 y rounded: each expert's output joins the weighted sum in fp32."""
    E, H, I, T, k = 12, 512, 256, 90, 6
    for fmt in ("nv", "mx"):
        m = make(E, H, I, fmt, 21)
        x = rnd((T, H), 22).bfloat16().cuda()
        ids, w = (torch.from_numpy(v).cuda() for v in route(T, k, E, 23, 0.1))
        want = Fp4Experts(*m, E, out_dtype=torch.float32)(x, ids, w)
        for dt in (torch.bfloat16, torch.float16):
            assert torch.equal(Fp4Experts(*m, E, out_dtype=dt)(x, ids, w), want.to(dt))


def test_expert_outputs_beyond_fp16_whose_sum_is_within():
    """Two experts of opposite down weights: each output passes 65504, the weighted sum does not."""
    E, H, I, T = 2, 256, 128, 9
    g, u = (rnd((I, H), s, H**-0.5) for s in (1, 2))
    d = rnd((H, I), 3, 4e5 * I**-0.5)
    def put(a, b):
        parts = [hq_fp4_quantize(v.cuda(), "mx") for v in (a, b)]
        return Fp4Matrix(torch.cat([p.codes for p in parts]), torch.cat([p.scales for p in parts]), "mx")
    m = [put(g, g), put(u, u), put(d, -d)]
    x = rnd((T, H), 4).half().cuda()
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda")
    one = Fp4Experts(*m, E, out_dtype=torch.float32)(x, ids[:, :1].contiguous(), torch.ones(T, 1, device="cuda"))
    assert one.abs().max().item() > 65504
    w = torch.tensor([[0.5, 0.499]] * T, device="cuda")
    y = Fp4Experts(*m, E)(x, ids, w)
    assert y.dtype == torch.float16 and bool(torch.isfinite(y).all())
    want = one.double() * (w[:, :1].double() - w[:, 1:].double())
    # two products of d and one sum in fp32 (2^-24 each of 0.5 |d| at most), one rounding to fp16
    tol = 3 * 2.0**-24 * one.double().abs() + 2.0**-11 * want.abs() + 2.0**-25
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("at", [-60.0, -20.0, 0.0, 12.0])
def test_h_to_its_last_place(fmt, at):
    """h = g / (1 + exp(-g)) u where the exponential is far from 1, read back through identity down matrices and fp32
    outputs: y is 6 times the packed h.  Single-precision exp is within 1 ulp (2^-23), the sum, the quotient and the
    product within half an ulp each: every packing of h (1 +- 2.6 2^-23) is allowed and no other."""
    E, H, I, T = 2, 128, 128, 6000
    rng = np.random.default_rng(int(at) + 100)
    g, u = (hq_fp4_quantize(torch.from_numpy(v).float().cuda(), fmt) for v in
            (at / H * (1 + 0.15 * rng.standard_normal((E * I, H))) + (0.05 if at == 0 else 0) * rng.standard_normal((E * I, H)),
             rng.standard_normal((E * I, H)) * H**-0.5))
    eye = hq_fp4_quantize(6 * torch.eye(128).repeat(E, 1).cuda(), fmt)
    assert np.array_equal(dense(eye), np.tile(6 * np.eye(128), (E, 1)))
    hs = None
    if fmt == "nv":
        hs = torch.tensor(abs(at / (1 + np.exp(-at)) if at else 0.5) / 1000, dtype=torch.float32, device="cuda")
    x = torch.from_numpy(1 + 0.1 * rng.standard_normal((T, H))).float().cuda()
    ids = torch.from_numpy(rng.integers(0, E, (T, 1)).astype(np.int32)).cuda()
    y = bits(Fp4Experts(g, u, eye, E, h_scale=hs, out_dtype=torch.float32)(x, ids, torch.ones(T, 1, device="cuda"))).astype(np.float64)
    t = 1.0 if hs is None else hs.item()
    some = 0
    for e in range(E):
        r = np.flatnonzero(ids.cpu().numpy()[:, 0] == e)
        a = hq_fp4_quantize(x[torch.from_numpy(r).cuda()], fmt)
        gv, uv = (bits(hq_fp4_matmul(expert(m, e, I), a)).astype(np.float64) for m in (g, u))
        h = gv / (1 + np.exp(-gv)) * uv
        d = 2.6 * 2.0**-23 * np.abs(h)
        hi, lo = np.abs(h) + d, np.maximum(np.abs(h) - d, 0)
        # fp32 products of a code's value, its scale and the tensor scale: 2^-24 once more
        ok = np.zeros(h.shape, dtype=bool)
        for scale_from in (lo, hi):
            for end in (h - d, h + d):
                v = values_at(end, fmt, scale_from, t if fmt == "nv" else None)
                ok |= np.abs(y[r] - 6 * v) <= 3 * 2.0**-24 * np.abs(6 * v)
        some += int(np.count_nonzero(y[r]))
        assert ok.all(), np.argwhere(~ok)[:5]
    assert some > T * I / 4


@pytest.mark.parametrize("ex,eg,eu,eh", [(-75, 46, -75, -133), (66, 66, 66, None)])
def test_tensor_scales_whose_product_leaves_fp32(ex, eg, eu, eh):
    """Tensor scales 2^ex of x and 2^eg, 2^eu of gate and up whose products are subnormal (u about 2^-122, h about as
    large, h's own scale 2^eh) or infinite (g a large negative number, whose silu is 0); rows of zeros stay zeros."""
    E, H, I, T = 2, 128, 128, 20
    size = 2.0**-9 if ex > 0 else 512.0
    rng = np.random.default_rng(5)
    g, u = (rng.integers(-4, 5, (E * I, H)) * 2.0**e * size for e in (eg, eu))
    dn, x = rng.integers(-4, 5, (E * H, I)) * 1.0, rng.integers(-4, 5, (T, H)) * 2.0**ex * size
    if ex > 0:
        g[:, 8:], u[:, 8:], x[:, 8:] = 0, 0, 0
        g, x = -np.abs(g), np.abs(x)
    x[3] = 0
    m = []
    for v, e in ((g, eg), (u, eu), (dn, 0)):
        t = torch.full((), 2.0**e, device="cuda")
        q = hq_fp4_quantize(torch.from_numpy(v).float().cuda(), "nv", tensor_scale=t)
        m.append(Fp4Matrix(q.codes, q.scales, "nv", t.repeat(E)))
    xs, hs = (None if e is None else torch.full((1,), 2.0**e, device="cuda") for e in (ex, eh))
    ids, w = torch.from_numpy(rng.integers(0, E, (T, 1)).astype(np.int32)).cuda(), torch.ones(T, 1, device="cuda")
    layer = Fp4Experts(*m, E, x_scale=xs, h_scale=hs, out_dtype=torch.float32)
    x = torch.from_numpy(x).float().cuda()
    y = layer(x, ids, w)
    check_layer(layer, *m, E, x, ids.cpu().numpy(), w.cpu().numpy(), y, xs, hs)
    assert bool((y[3] == 0).all()) and (bool((y == 0).all()) if eh is None else y.abs().max().item() > 2.0**-126)


def test_one_token_of_an_odd_pitch():
    """A single row of a wider buffer whose pitch is no multiple of 16 bytes."""
    E, H, I = 3, 256, 128
    m = make(E, H, I, "nv", 9)
    big = rnd((3, H + 1), 10).bfloat16().cuda()
    ids, w = (torch.from_numpy(v).cuda() for v in route(1, 2, E, 11))
    for x in (big[:1, :H], big[1:2, :H], big[:1, 1:]):
        assert torch.equal(Fp4Experts(*m, E)(x, ids, w), Fp4Experts(*m, E)(x.repeat(2, 1)[:1], ids, w))
