"""The residual norm and its gradient on the GPU, against their formulas in float64.

Tolerances: an output is off by its rounding, U = finfo(type).eps / 2 of its value, and by what float32 sums lose
before.  A row's sum of squares goes through at most 32 additions in a thread and 13 joins, and a handful of products
and one division and root follow: under 128 roundings of 2^-24, so 2^-17 of what they act on.
"""
import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, E4M3, INT8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8
U = torch.finfo(BF16).eps / 2
F = 2.0 ** -17
LEAST = 2.0 ** -133  # bf16's smallest step, below its normal range

# sizes at the borders of the thread layouts (1024 channels a row and multiples beyond), the smallest and the largest
SIZES = [(1, 8), (3, 16), (5, 1016), (7, 1024), (129, 1032), (2, 4096), (33, 4104), (9, 5120), (4, 8192), (3, 8200),
         (2, 16384), (700, 24)]


@pytest.fixture(scope="module")
def tr():
    from speculative_decoding_drafter_gb300 import training

    return training


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def make(N, C, seed=0):
    g = gen(seed + 1000 * N + C)
    x, r = randn(g, N, C).to(BF16), (randn(g, N, C) * (0.2 + 3 * torch.rand(C, device="cuda", generator=g))).to(BF16)
    return x, r, (1 + 0.3 * randn(g, C)).to(BF16)


def norm64(z, gamma, eps):
    n = (z.square().mean(1, keepdim=True) + eps).sqrt()
    return torch.where(n > 0, z / n, torch.zeros_like(z)) * gamma.double()


def close(got, want, bound):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("N,C", SIZES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(tr, N, C, residual):
    x, r, gamma = make(N, C)
    out = tr.dflash2_residual_norm(x, gamma, residual=r if residual else None, eps=1e-5)
    z = x.double() + (r.double() if residual else 0)
    want = norm64(z, gamma, 1e-5)
    close(out["y"], want, want.abs() * (U + F) + LEAST)
    assert ("sum" in out) == residual
    if residual:
        close(out["sum"], z, z.abs() * (U + 2.0 ** -24) + LEAST)


@pytest.mark.parametrize("N,C", SIZES)
@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_codes(tr, N, C, dtype):
    x, r, gamma = make(N, C, 1)
    out = tr.dflash2_residual_norm(x, gamma, residual=r, codes=dtype, y=False)
    assert set(out) == {"sum", "codes", "scale"}
    want = norm64(x.double() + r.double(), gamma, 1e-6)
    top = 448.0 if dtype == E4M3 else 127.0
    scale = want.abs().amax(1) / top
    close(out["scale"], scale, scale * F)
    held = out["codes"].to(torch.float32).double() * out["scale"].double()[:, None]
    if dtype == E4M3:  # half a step: 2^-4 of a code, 2^-10 below the smallest normal
        bound = torch.maximum(want.abs() * 2.0 ** -4, scale[:, None] * 2.0 ** -10)
    else:
        bound = 0.5 * scale[:, None].expand_as(want)
    close(held, want, bound + (want.abs() + scale[:, None] * top) * F)


def test_all_outputs_at_once_and_in_place(tr):
    x, r, gamma = make(37, 520, 2)
    apart = tr.dflash2_residual_norm(x, gamma, residual=r, codes=INT8)
    a, b = x.clone(), r.clone()
    out = tr.dflash2_residual_norm(a, gamma, residual=b, sum=b, y=a, codes=INT8)
    assert out["sum"] is b and out["y"] is a
    for name in ("sum", "y", "codes", "scale"):
        assert torch.equal(apart[name], out[name])
    only = tr.dflash2_residual_norm(x, gamma, residual=r, y=False)
    assert set(only) == {"sum"} and torch.equal(only["sum"], apart["sum"])


@pytest.mark.parametrize("size", [1e-40, 1e-30, 1e-22, 1e-12, 1e12, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_squares_beyond_float32(tr, size, eps):
    """Rows whose squares float32 does not hold, among ordinary ones."""
    g = gen(5)
    for C in (64, 2048, 8192):
        x = (torch.rand(4, C, device="cuda", generator=g) * 2 - 1)
        x[1] *= size
        x[3] = 0
        x, gamma = x.to(BF16), torch.ones(C, dtype=BF16, device="cuda")
        z = x.double()
        want = norm64(z, gamma, eps)
        close(tr.dflash2_residual_norm(x, gamma, eps=eps)["y"], want, want.abs() * (U + F) + LEAST)
        dy = randn(g, 4, C).to(BF16)
        got = tr.dflash2_residual_norm_grad(x, gamma, dy, eps=eps)["dx"]
        n = (z.square().mean(1, keepdim=True) + eps).sqrt()
        some = (n > 0) & (dy.double().abs().amax(1, keepdim=True) / n < 1e38)
        zh = torch.where(n > 0, z / n, torch.zeros_like(z))
        u = dy.double()
        dx = torch.where(n > 0, (u - zh * (u * zh).mean(1, keepdim=True)) / n, torch.zeros_like(u))
        slack = torch.where(n > 0, (u.abs() + zh.abs() * (u * zh).abs().mean(1, keepdim=True)) / n, torch.zeros_like(u))
        keep = some[:, 0] | (n[:, 0] == 0)
        close(got[keep], dx[keep], dx[keep].abs() * U + slack[keep] * F + LEAST)


def test_rows_that_are_not_finite_stay_alone(tr):
    x, r, gamma = make(6, 256, 3)
    want = tr.dflash2_residual_norm(x, gamma, residual=r, codes=E4M3)
    x[2, 7], r[4, 9] = math.nan, math.inf
    out = tr.dflash2_residual_norm(x, gamma, residual=r, codes=E4M3)
    others = [0, 1, 3, 5]
    for name in ("sum", "y", "codes", "scale"):
        a, b = out[name].view(torch.uint8)[others], want[name].view(torch.uint8)[others]
        if name != "scale":
            assert torch.equal(a, b)
    assert torch.equal(out["scale"][others], want["scale"][others])
    assert out["y"][2].isnan().all() and out["y"][4, 9].isnan()
    assert out["scale"][[2, 4]].isnan().all()


def grad64(z, gamma, dy, d_sum, eps):
    n = (z.square().mean(1, keepdim=True) + eps).sqrt()
    zh, u = z / n, dy * gamma
    dx = (u - zh * (u * zh).mean(1, keepdim=True)) / n + d_sum
    slack = (u.abs() + zh.abs() * (u * zh).abs().mean(1, keepdim=True)) / n + d_sum.abs()
    return dx, (dy * zh).sum(0), slack, (dy * zh).abs().sum(0)


@pytest.mark.parametrize("N,C", SIZES + [(5000, 520), (3001, 4096)])
@pytest.mark.parametrize("stream_grad", [True, False])
def test_gradient(tr, N, C, stream_grad):
    z, d, gamma = make(N, C, 4)
    dy = (randn(gen(N + C), N, C) * 0.01).to(BF16)
    d = (d * 0.01).to(BF16)
    out = tr.dflash2_residual_norm_grad(z, gamma, dy, d_sum=d if stream_grad else None, eps=1e-6)
    ds = d.double() if stream_grad else torch.zeros_like(d, dtype=torch.float64)
    dx, dg, slack, sums = grad64(z.double(), gamma.double(), dy.double(), ds, 1e-6)
    close(out["dx"], dx, dx.abs() * U + slack * F + LEAST)
    # a channel's sum: at most 20 rows a CTA here, 608 / 8 joins a thread and 8 more, on top of a row's own error
    close(out["dgamma"], dg, sums * 2.0 ** -16 + 1e-45)


def test_gradient_against_differences(tr):
    N, C, eps = 5, 72, 1e-6
    x, r, gamma = make(N, C, 6)
    z = tr.dflash2_residual_norm(x, gamma, residual=r)["sum"]
    dy = randn(gen(8), N, C).to(BF16)
    out = tr.dflash2_residual_norm_grad(z, gamma, dy)
    f = lambda zz, gg: float((norm64(zz, gg, eps) * dy.double()).sum())  # noqa: E731
    for seed in range(4):
        v, w = randn(gen(20 + seed), N, C).double(), randn(gen(40 + seed), C).double()
        h = 1e-5
        along = (f(z.double() + h * v, gamma) - f(z.double() - h * v, gamma)) / (2 * h)
        # each element of dx is off by U of it; the differences by about h^2
        bound = (out["dx"].double() * v).abs().sum() * (U + F) + 1e-6
        assert abs(along - (out["dx"].double() * v).sum()) <= bound
        g64 = gamma.double()
        along = (f(z.double(), g64 + h * w) - f(z.double(), g64 - h * w)) / (2 * h)
        assert abs(along - (out["dgamma"].double() * w).sum()) <= (out["dgamma"].double() * w).abs().sum() * F + 1e-4


def test_gradient_outputs(tr):
    z, d, gamma = make(50, 264, 7)
    dy = randn(gen(9), 50, 264).to(BF16)
    want = tr.dflash2_residual_norm_grad(z, gamma, dy, d_sum=d)
    assert set(tr.dflash2_residual_norm_grad(z, gamma, dy, d_sum=d, dgamma=False)) == {"dx"}
    for name in ("dy", "d_sum"):
        a = {"dy": dy.clone(), "d_sum": d.clone()}
        out = tr.dflash2_residual_norm_grad(z, gamma, a["dy"], d_sum=a["d_sum"], dx=a[name])
        assert torch.equal(out["dx"], want["dx"]) and torch.equal(out["dgamma"], want["dgamma"])


def test_no_rows(tr):
    x, gamma = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    assert tr.dflash2_residual_norm(x, gamma)["y"].shape == (0, 64)
    out = tr.dflash2_residual_norm_grad(x, gamma, x, dgamma=torch.full((64,), 7.0, device="cuda"))
    assert (out["dgamma"] == 0).all()


def test_captured_replayed_and_on_other_streams(tr):
    x, r, gamma = make(300, 1032, 10)
    dy = randn(gen(11), 300, 1032).to(BF16)
    eager = tr.dflash2_residual_norm(x, gamma, residual=r)
    back = tr.dflash2_residual_norm_grad(eager["sum"], gamma, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    forward = tr.ResidualNormPlan(x, gamma, residual=r, stream=s)
    backward = tr.ResidualNormGradPlan(forward.outputs["sum"], gamma, dy, stream=s)
    with torch.cuda.stream(s):
        forward(), backward()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            forward(), backward()
    torch.cuda.synchronize()
    for new in (x, -x):
        x.copy_(new.clone())
        for t in (*forward.outputs.values(), *backward.outputs.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        a = tr.dflash2_residual_norm(x, gamma, residual=r)
        b = tr.dflash2_residual_norm_grad(a["sum"], gamma, dy)
        for name, t in {**a, **b}.items():
            assert torch.equal({**forward.outputs, **backward.outputs}[name], t)
    x.neg_()
    assert torch.equal(tr.dflash2_residual_norm(x, gamma, residual=r)["y"], eager["y"])
    assert torch.equal(tr.dflash2_residual_norm_grad(eager["sum"], gamma, dy)["dgamma"], back["dgamma"])


def test_refused(tr):
    x, r, gamma = make(4, 64)
    with pytest.raises(ValueError, match="overlaps"):
        tr.dflash2_residual_norm(x, gamma, residual=r, sum=x, y=x)
    with pytest.raises(ValueError, match="overlaps"):
        tr.dflash2_residual_norm_grad(x, gamma, r, dx=x)
    with pytest.raises(ValueError, match="at least one"):
        tr.dflash2_residual_norm(x, gamma, y=False)
    with pytest.raises(ValueError, match="contiguous"):
        tr.dflash2_residual_norm(x.t().contiguous().t(), gamma)
    with pytest.raises(TypeError):
        tr.dflash2_residual_norm(x.float(), gamma)
    with pytest.raises(TypeError, match="codes"):
        tr.dflash2_residual_norm(x, gamma, codes=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        tr.dflash2_residual_norm(x, gamma[:32])
    with pytest.raises(ValueError, match="hold"):
        tr.dflash2_residual_norm_grad(x, gamma, r, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_two_threads(tr):
    """Plans of different sizes called from two host threads at once, each on its own stream."""
    failed = []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            x, r, gamma = make(200 + seed, 512 * (1 + seed), seed)
            want = tr.dflash2_residual_norm(x, gamma, residual=r)["y"]
            torch.cuda.synchronize()
            plan = tr.ResidualNormPlan(x, gamma, residual=r, stream=s)
            for _ in range(20):
                plan()
            s.synchronize()
            if not torch.equal(plan.outputs["y"], want):
                failed.append(seed)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed


@pytest.mark.parametrize("C", [64, 1024, 2048, 16384])
@pytest.mark.parametrize("N", [1, 2, 5])
def test_dgamma_anywhere_in_a_flat_buffer(tr, N, C):
    """A view of a buffer of many gradients, at any element; what lies around it stays."""
    z, _, gamma = make(N, C, 12)
    dy = randn(gen(13), N, C).to(BF16)
    want = tr.dflash2_residual_norm_grad(z, gamma, dy)
    for at in (1, 2, 3, 4):
        flat = torch.full((C + 8,), 7.0, device="cuda")
        got = tr.dflash2_residual_norm_grad(z, gamma, dy, dgamma=flat[at:at + C])
        assert torch.equal(got["dgamma"], want["dgamma"]) and torch.equal(got["dx"], want["dx"])
        assert (flat[:at] == 7).all() and (flat[at + C:] == 7).all()


def check_gradient(tr, z, gamma, dy, d, eps):
    out = tr.dflash2_residual_norm_grad(z, gamma, dy, d_sum=d, eps=eps)
    ds = torch.zeros_like(z, dtype=torch.float64) if d is None else d.double()
    dx, dg, slack, sums = grad64(z.double(), gamma.double(), dy.double(), ds, eps)
    close(out["dx"], dx, dx.abs() * U + slack * F + LEAST)
    close(out["dgamma"], dg, sums * 2.0 ** -16 + 1e-45)


@pytest.mark.parametrize("size", [1e-40, 1e-38, 1e-30, 1e-20, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("C", [64, 1024, 2048, 8192])
def test_gradient_of_rows_whose_squares_leave_float32(tr, size, C):
    """dx and dgamma, with eps = 0: 1 / n of a row below the normal range is more than float32 holds, z / n is not."""
    g = gen(C)
    z = torch.rand(5, C, device="cuda", generator=g) * 2 - 1
    z[1:4] *= size
    z[2, ::3] = 0
    z, gamma = z.to(BF16), (1 + 0.3 * randn(g, C)).to(BF16)
    dy, d = (randn(g, 5, C) * 1e-4).to(BF16), randn(g, 5, C).to(BF16)
    check_gradient(tr, z, gamma, dy, None, 0.0)
    dy[3] = 0  # nothing came back to this row
    check_gradient(tr, z, gamma, dy, d, 0.0)
    out = tr.dflash2_residual_norm_grad(z, gamma, dy, d_sum=d, eps=0.0)
    assert torch.equal(out["dx"][3], d[3])


@pytest.mark.parametrize("size,back", [(1e-11, 1e-35), (1e-4, 1e-33), (1e5, 1e30), (1e15, 1e28)])
@pytest.mark.parametrize("C", [64, 2048, 8192])
def test_gradient_whose_products_leave_float32(tr, size, back, C):
    """Rows whose squares float32 holds, and not their products with the gradient."""
    g = gen(C + 1)
    z, dy = (randn(g, 3, C) * size).to(BF16), (randn(g, 3, C) * back).to(BF16)
    dy[1] = z[1] * (back / size)  # along the row: the formula takes most of it away
    check_gradient(tr, z, (1 + 0.3 * randn(g, C)).to(BF16), dy, None, 0.0)
