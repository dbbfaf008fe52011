"""GPU parity of the routing steps (hq_moe_sort and the row movers) against the
64-bit oracle.  Positions are integers and must be equal; gathered rows are
copies; sums run over at most k = 32 terms in fp32 (each addition and product
half an ulp: (2 k + 1) 2^-24 of the sum of magnitudes) and are rounded once;
dw sums H products (in lanes and a tree: at most H + 5 roundings).
"""
import numpy as np
import pytest
import torch

from bit_hadamard_rotated_b200 import (HqError, hq_moe_combine, hq_moe_combine_grad, hq_moe_gather,
                                       hq_moe_gather_grad, hq_moe_sort)
from oracle import fp4

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_hadamard_rotated_b200 import build
    build.build()


def routing(T, k, E, seed, masked=0.0, skew=False):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]) if T else np.zeros((0, k), dtype=np.int64)
    if skew and T:
        ids[:, 0] = 0
    if masked and T:
        ids[rng.random(T) < masked] = -1
        ids.reshape(-1)[rng.integers(0, T * k, max(1, T * k // 50))] = E + 3
    return ids.astype(np.int32)


CASES = [  # T, k, E, align, masked
    (1, 1, 1, 1, 0), (1, 8, 256, 1, 0), (32, 8, 256, 1, 0), (32, 8, 256, 128, 0.3), (1000, 4, 60, 16, 0.2), (1024, 8, 8, 1, 0),
    (1025, 8, 7, 3, 0), (5003, 8, 256, 128, 0.125), (40000, 8, 300, 1, 0.5), (3000, 2, 16384, 1, 0), (9000, 1, 1025, 64, 0),
    (5, 32, 40, 1, 0), (0, 4, 9, 8, 0), (700, 3, 5, 1, 1.0), (70000, 1, 2, 1, 0),
]


@pytest.mark.parametrize("T,k,E,align,masked", CASES)
def test_sort(T, k, E, align, masked):
    ids = routing(T, k, E, T + k + E, masked, skew=T == 1000)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), E, align=align)
    pos, off, cnt = fp4.sort(ids, E, align)
    assert np.array_equal(plan.pos.cpu().numpy(), pos)
    assert np.array_equal(plan.offsets.cpu().numpy(), off)
    assert np.array_equal(plan.counts.cpu().numpy(), cnt)
    assert off[-1] <= plan.n_rows or off[-1] - plan.n_rows < align
    assert pos.max(initial=-1) < max(plan.n_rows, 1)


def test_sort_same_expert_twice_in_a_token():
    ids = np.array([[3, 3, 1], [1, 3, 1]], dtype=np.int32)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), 4)
    assert plan.pos.cpu().tolist() == [[3, 4, 0], [1, 5, 2]]


def rnd(shape, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).to(dtype)


def near(got, want, sums, dtype, terms):
    """|got - want| within `terms` roundings of the sum of magnitudes and one of the result."""
    s = terms * 2.0**-24 * sums
    tol = s + torch.finfo(dtype).eps / 2 * (np.abs(want) + s) + (2.0**-25 if dtype == torch.float16 else 2.0**-149)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,align,masked", [
    (1, 1, 3, 8, 1, 0), (1, 8, 16, 2048, 1, 0), (32, 8, 256, 2048, 128, 0.3), (61, 5, 9, 999, 1, 0.2), (7, 32, 40, 33, 4, 0.5),
    (300, 4, 60, 4096, 1, 0), (40, 2, 4, 1, 1, 0), (20, 3, 6, 9000, 1, 0.2), (12, 3, 6, 64, 1, 1.0),
])
def test_rows_there_and_back(dtype, T, k, E, H, align, masked):
    ids = routing(T, k, E, T + H, masked)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), E, align=align)
    pos, _, _ = fp4.sort(ids, E, align)
    has, n = pos >= 0, plan.n_rows
    x, dy, z, dxs = (rnd((r, H), dtype, i) for i, r in enumerate((T, T, n, n)))
    w = rnd((T, k), torch.float32, 9)
    z[np.setdiff1d(np.arange(n), pos[has])] = float("nan")  # rows without a pair are never read
    dxs[np.setdiff1d(np.arange(n), pos[has])] = float("nan")
    out = torch.full((n, H), 5.0, dtype=dtype, device="cuda")
    xs = hq_moe_gather(x.cuda(), plan, out=out).cpu()
    want = torch.full((n, H), 5.0, dtype=dtype)
    t_of, j_of = np.nonzero(has)
    want[pos[has]] = x[t_of]
    assert torch.equal(xs, want)
    xd, dyd, wd = x.double().numpy(), dy.double().numpy(), w.double().numpy()
    zd = np.where(has[..., None], z.double().numpy()[pos], 0)
    y = hq_moe_combine(z.cuda(), plan, w.cuda())
    near(y, (wd[..., None] * zd).sum(1), np.abs(wd[..., None] * zd).sum(1), dtype, 2 * k + 1)
    y32 = hq_moe_combine(z.cuda(), plan, w.cuda(), out_dtype=torch.float32)
    near(y32, (wd[..., None] * zd).sum(1), np.abs(wd[..., None] * zd).sum(1), torch.float32, 2 * k + 1)
    gd = np.where(has[..., None], dxs.double().numpy()[pos], 0)
    near(hq_moe_gather_grad(dxs.cuda(), plan), gd.sum(1), np.abs(gd).sum(1), dtype, k)
    out = torch.full((n, H), 5.0, dtype=dtype, device="cuda")
    dz, dw = hq_moe_combine_grad(dy.cuda(), z.cuda(), plan, w.cuda(), out=out)
    wdz = np.full((n, H), 5.0)
    wdz[pos[has]] = wd[has][:, None] * dyd[t_of]
    near(dz, wdz, np.abs(wdz), dtype, 1)
    near(dw, (dyd[:, None] * zd).sum(2), np.abs(dyd[:, None] * zd).sum(2), torch.float32, H + 5)


def test_gradients_against_differences():
    """hq_moe_gather_grad and hq_moe_combine_grad are the gradients of gather
    and combine: both are linear (or bilinear), so a difference over any step
    is exact up to roundings."""
    T, k, E, H = 6, 3, 5, 16
    ids = routing(T, k, E, 1, 0.2)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), E)
    n = plan.n_rows
    x, z, w, dy, g = (rnd(s, torch.float32, i).cuda() for i, s in enumerate([(T, H), (n, H), (T, k), (T, H), (n, H)]))

    def f_gather(v):
        return (hq_moe_gather(v, plan, out=torch.zeros(n, H, device="cuda")).double() * g.double()).sum().item()

    def f_combine(rows, weights):
        return (hq_moe_combine(rows, plan, weights).double() * dy.double()).sum().item()

    g0 = g.clone()
    dx = hq_moe_gather_grad(g0, plan)
    dz, dw = hq_moe_combine_grad(dy, z, plan, w, out=torch.zeros(n, H, device="cuda"))
    for d, f, at in ((dx, f_gather, x), (dz, lambda v: f_combine(v, w), z), (dw, lambda v: f_combine(z, v), w)):
        for i in np.random.default_rng(3).integers(0, at.numel(), 12):
            e = torch.zeros_like(at).view(-1)
            e[i] = 1.0
            e = e.view_as(at)
            diff = (f(at + e) - f(at - e)) / 2
            # values of at + e are rounded to fp32 and summed over at most T k H terms of magnitude about 1
            assert abs(diff - d.view(-1)[i].item()) <= 1e-4


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return hq_moe_gather(x, plan, out=torch.zeros((plan.n_rows, x.shape[1]), dtype=x.dtype, device=x.device))

    @staticmethod
    def backward(ctx, g):
        return hq_moe_gather_grad(g.contiguous(), ctx.plan), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, plan):
        ctx.plan = plan
        ctx.save_for_backward(rows, w)
        return hq_moe_combine(rows, plan, w)

    @staticmethod
    def backward(ctx, g):
        rows, w = ctx.saved_tensors
        drows, dw = hq_moe_combine_grad(g.contiguous(), rows, ctx.plan, w, out=torch.zeros_like(rows))
        return drows, dw, None


def test_expert_layer_trains_through_them():
    """Sort, gather, each expert's own product, combine, as a training program joins them: outputs and all gradients
    against the same layer written per token in 64 bits.  fp32 products of K terms: K 2^-24 of the sum of magnitudes
    at most, here bounded through the largest values."""
    T, k, E, H, F = 37, 3, 6, 24, 16
    ids = routing(T, k, E, 5, 0.2)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), E, align=4)
    x, w, W = rnd((T, H), torch.float32, 1), rnd((T, k), torch.float32, 2), rnd((E, H, F), torch.float32, 3)
    dy = rnd((T, F), torch.float32, 4)
    a = [v.cuda().requires_grad_() for v in (x, w, W)]
    off, cnt = plan.offsets.tolist(), plan.counts.tolist()
    xs = _Gather.apply(a[0], plan)
    parts = [torch.zeros(0, F, device="cuda")]
    for e in range(E):
        rows_ = xs[off[e]:off[e + 1]]
        parts.append(torch.tanh(rows_ @ a[2][e]) if off[e + 1] > off[e] else rows_.new_zeros(0, F))
    z = torch.cat(parts)
    z = torch.cat([z, z.new_zeros(plan.n_rows - z.shape[0], F)])
    y = _Combine.apply(z, a[1], plan)
    y.backward(dy.cuda())
    b = [v.double().requires_grad_() for v in (x, w, W)]
    want = torch.zeros(T, F, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                want[t] = want[t] + b[1][t, j] * torch.tanh(b[0][t] @ b[2][ids[t, j]])
    want.backward(dy.double())
    assert torch.allclose(y.detach().cpu().double(), want.detach(), rtol=0, atol=k * (H + 8) * 2.0**-22)
    for got, ref in zip(a, b):
        assert torch.allclose(got.grad.cpu().double(), ref.grad, rtol=0, atol=float(ref.grad.abs().max()) * (T * k + H) * 2.0**-22)


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    plan = hq_moe_sort(ids, 3)
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        hq_moe_sort(ids.long(), 3)
    with pytest.raises(HqError):
        hq_moe_sort(ids, 0)
    with pytest.raises(HqError):
        hq_moe_sort(ids, 3, align=0)
    with pytest.raises(HqError):
        hq_moe_sort(torch.zeros((4, 33), dtype=torch.int32, device="cuda"), 3)
    with pytest.raises(ValueError):
        hq_moe_gather(x[:3], plan)
    with pytest.raises(ValueError):
        hq_moe_gather(x.double(), plan)
    with pytest.raises(ValueError):
        hq_moe_combine(x, plan, torch.zeros((4, 3), device="cuda"))
    with pytest.raises(HqError):
        hq_moe_combine(x.half(), plan, torch.zeros((4, 2), device="cuda"), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hq_moe_combine_grad(x, x.half(), plan, torch.zeros((4, 2), device="cuda"))


def test_rows_outside_the_buffer_are_skipped():
    """A buffer smaller than the plan's rows: what does not fit is neither written nor read."""
    ids = routing(20, 4, 6, 3)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), 6)
    x = rnd((20, 24), torch.float32, 1).cuda()
    guard = torch.full((60, 24), 3.0, device="cuda")
    out = hq_moe_gather(x, plan, out=guard[:40])
    assert bool((guard[40:] == 3).all())
    full = hq_moe_gather(x, plan)
    assert torch.equal(out, full[:40])


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^32, forward and back."""
    T, H, E = 300000, 15001, 3
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-64:] = torch.randn(64, H, device="cuda").bfloat16()
    ids = torch.full((T, 1), 1, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), 0.5, device="cuda")
    plan = hq_moe_sort(ids, E)
    assert torch.equal(plan.pos[:, 0], torch.arange(T, dtype=torch.int32, device="cuda"))
    xs = hq_moe_gather(x, plan)
    assert torch.equal(xs[-64:], x[-64:]) and bool((xs[-200:-64] == 0).all())
    y = hq_moe_combine(xs, plan, w)
    assert torch.equal(y[-64:], (x[-64:].float() * 0.5).bfloat16())
    dz, dw = hq_moe_combine_grad(x, xs, plan, w, out=y)
    assert torch.equal(dz[-64:], (x[-64:].float() * 0.5).bfloat16())
    want = (x[-64:].double() ** 2).sum(1)
    assert bool(((dw[-64:, 0].double() - want).abs() <= (H / 32 + 5) * 2.0**-24 * want).all())


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, None), (torch.bfloat16, None), (torch.bfloat16, torch.float32),
                                             (torch.float32, torch.float16)])
@pytest.mark.parametrize("given", [False, True])
def test_autograd_records_gather_and_combine(dtype, out_dtype, given):
    """Gather, scale, combine under autograd, on the current stream and on a given one: the gradients of x, of the rows'
    factor and of the weights against the formulas in 64 bits."""
    T, k, E, H = 45, 4, 7, 72
    ids = routing(T, k, E, 8, 0.2)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), E, align=8)
    pos, _, _ = fp4.sort(ids, E, 8)
    has = pos >= 0
    x, w = rnd((T, H), dtype, 1).cuda().requires_grad_(), rnd((T, k), torch.float32, 2).cuda().requires_grad_()
    f = rnd((plan.n_rows, H), dtype, 3).cuda().requires_grad_()
    s = torch.cuda.Stream() if given else None
    if given:
        s.wait_stream(torch.cuda.current_stream())
    xs = hq_moe_gather(x, plan, stream=s)
    if given:
        torch.cuda.current_stream().wait_stream(s)
    z = xs * f
    if given:
        s.wait_stream(torch.cuda.current_stream())
    y = hq_moe_combine(z, plan, w, out_dtype=out_dtype, stream=s)
    if given:
        torch.cuda.current_stream().wait_stream(s)
    assert y.dtype == (out_dtype or dtype) and y.requires_grad
    dy = rnd((T, H), y.dtype, 4).cuda()
    y.backward(dy)
    torch.cuda.synchronize()
    free = np.setdiff1d(np.arange(plan.n_rows), pos[has])
    assert bool((xs.detach()[free] == 0).all()) and bool((f.grad[free] == 0).all())
    zd, dyd, wd = z.detach().double().cpu().numpy(), dy.double().cpu().numpy(), w.detach().double().cpu().numpy()
    xd, fd = x.detach().double().cpu().numpy(), f.detach().double().cpu().numpy()
    zp = np.where(has[..., None], zd[pos], 0)
    near(y.detach(), (wd[..., None] * zp).sum(1), np.abs(wd[..., None] * zp).sum(1), y.dtype, 2 * k + 1)
    near(w.grad, (dyd[:, None] * zp).sum(2), np.abs(dyd[:, None] * zp).sum(2), torch.float32, H + 5)
    # dz is rounded to the rows' type, then times f and x in that type, then (x) summed over the slots
    step = torch.finfo(dtype).eps / 2
    t_of, j_of = np.nonzero(has)
    dz = wd[has][:, None] * dyd[t_of]
    df = dz * xd[t_of]
    err = np.abs(f.grad.double().cpu().numpy()[pos[has]] - df)
    assert np.all(err <= 3 * step * np.abs(df) + 2.0**-126)
    dxs = np.zeros((T, k, H))
    dxs[has] = dz * fd[pos[has]]
    sums = np.abs(dxs).sum(1)
    err = np.abs(x.grad.double().cpu().numpy() - dxs.sum(1))
    assert np.all(err <= 3 * step * sums + k * 2.0**-24 * sums + step * np.abs(dxs.sum(1)) + 2.0**-126)


def test_autograd_stays_out_of_it_where_nothing_is_recorded():
    ids = routing(20, 2, 5, 9)
    plan = hq_moe_sort(torch.from_numpy(ids).cuda(), 5)
    x = torch.randn(20, 16, device="cuda").requires_grad_()
    w = torch.rand(20, 2, device="cuda")
    with torch.no_grad():
        rows_ = hq_moe_gather(x, plan)
        assert not rows_.requires_grad and not hq_moe_combine(rows_, plan, w.clone().requires_grad_()).requires_grad
    assert not hq_moe_combine(rows_, plan, w).requires_grad
    assert hq_moe_combine(rows_, plan, w.clone().requires_grad_()).requires_grad
    with pytest.raises(ValueError):
        hq_moe_gather(x, plan, out=torch.empty(plan.n_rows, 16, device="cuda"))
    with pytest.raises(ValueError):
        hq_moe_combine(rows_, plan, w.clone().requires_grad_(), out=torch.empty(20, 16, device="cuda"))
    y = hq_moe_combine(hq_moe_gather(x, plan), plan, w)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)  # once only: no second derivatives
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_plans_hold_every_routing():
    """No segment ends past n_rows, which is reached where every expert has one pair."""
    for T, k, E, align in ((16, 8, 128, 128), (3, 4, 40, 128), (33, 1, 32, 32), (7, 1, 7, 4096), (64, 2, 64, 2)):
        ids = np.arange(T * k).reshape(T, k) % E
        plan = hq_moe_sort(torch.from_numpy(ids.astype(np.int32)).cuda(), E, align=align)
        end = int(plan.offsets[-1])
        assert end <= plan.n_rows
        pairs = np.bincount(ids.reshape(-1), minlength=E)
        assert end == int((-(-pairs // align) * align).sum())
        assert int(plan.pos.max()) < plan.n_rows
    full = hq_moe_sort(torch.arange(128, dtype=torch.int32, device="cuda").view(16, 8), 128, align=128)
    assert int(full.offsets[-1]) == full.n_rows == 128 * 128


def test_a_recorded_step_is_captured_and_replayed():
    """Forward and backward in one graph (warmed up on a side stream, whose autograd graph is gone before the capture),
    replayed with other values and another routing of the same sizes."""
    T, k, E, H = 30, 3, 6, 40
    x, w, f = (rnd(s, torch.float32, i).cuda().requires_grad_() for i, s in enumerate([(T, H), (T, k), (T * k, H)]))
    ids = torch.from_numpy(routing(T, k, E, 1, 0.2)).cuda()
    dy = rnd((T, H), torch.float32, 5).cuda()

    def step():
        plan = hq_moe_sort(ids, E)
        y = hq_moe_combine(hq_moe_gather(x, plan) * f, plan, w)
        return (y.detach(), *torch.autograd.grad(y, (x, w, f), dy))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in range(3):
        with torch.no_grad():
            x.copy_(rnd((T, H), torch.float32, 10 + seed))
            w.copy_(rnd((T, k), torch.float32, 20 + seed))
        ids.copy_(torch.from_numpy(routing(T, k, E, 30 + seed, 0.3 * seed)))
        g.replay()
        have = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(have, step()))
