"""The norm of many gradients together and their clipping on the GPU, against float64.

Tolerances: the norm comes from float32 sums of up to a few thousand squares a thread, joined in double: each
square and addition rounds by 2^-24; 2^-13 of the sum is what 2^11 additions lose at most, half of that the root.
A clipped element is x times a float32 factor (norm's error), rounded to its type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NORM = 2.0 ** -14


@pytest.fixture(scope="module")
def tr():
    from speculative_decoding_drafter_gb300 import training

    return training


def randn(seed, n, dtype, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, device="cuda", generator=g) * size).to(dtype)


def norm64(tensors, kind):
    if kind == "max":
        return max((float(t.double().abs().max()) for t in tensors if t.numel()), default=0.0)
    return math.sqrt(sum(float(t.double().square().sum()) for t in tensors))


def check(tr, tensors, max_norm, kind="l2", out=None, slack=NORM):
    before = [t.clone() for t in tensors]
    norm = norm64(tensors, kind)
    got = tr.dflash2_grad_clip(tensors, max_norm=max_norm, kind=kind, out=out)
    assert abs(float(got["norm"]) - norm) <= norm * slack + 1e-45
    factor = max_norm / norm if norm > max_norm else 1.0
    for t, o, b in zip(tensors, got["tensors"], before):
        if out is not None:
            assert torch.equal(t, b)
        want = b.double() * factor
        info = torch.finfo(t.dtype)
        if factor == 1.0:
            assert torch.equal(o, b)
        else:
            assert ((o.double() - want).abs() <= want.abs() * (info.eps / 2 + slack) + info.smallest_normal * info.eps).all()


SETS = {
    "one": [(1, F32)],
    "one 16-bit": [(1, BF16)],
    "few": [(5, F32), (0, BF16), (17, F16), (1000, BF16)],
    "ragged": [(8191, BF16), (8192, BF16), (8193, BF16), (4097, F32), (1, F16), (70001, F16), (300000, F32)],
    "many": [((i * 7919) % 997, (BF16, F32, F16)[i % 3]) for i in range(1500)],
    "sixty-four": [(100 + i, F32) for i in range(64)],
    "sixty-five": [(100 + i, F32) for i in range(65)],
    "large": [(30000007, BF16), (12345, F32)],
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("apart", [False, True])
def test_clip(tr, name, kind, apart):
    tensors = [randn(i, n, dtype, 0.1 + i % 3) for i, (n, dtype) in enumerate(SETS[name])]
    norm = norm64(tensors, kind)
    for limit in (norm * 2, norm * 0.37):
        check(tr, tensors, limit, kind, out=[torch.full_like(t, 3.0) for t in tensors] if apart else None)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_any_alignment(tr, dtype):
    """Views that start anywhere, in place and into outputs that start elsewhere; what lies around them stays."""
    for shift in range(0, 9):
        whole = randn(shift, 40000, dtype)
        held = torch.full((40040,), 5.0, dtype=dtype, device="cuda")
        for to in (0, 1, shift, 7):
            view, out = whole[shift:20001 + shift], held[to:20001 + to]
            held.fill_(5.0)
            check(tr, [view], 1.0, out=[out])
            assert (held[:to] == 5).all() and (held[20001 + to:] == 5).all()
        around = whole.clone()
        check(tr, [whole[shift:20001 + shift]], 1.0)
        assert torch.equal(whole[:shift], around[:shift]) and torch.equal(whole[20001 + shift:], around[20001 + shift:])
        for n in (1, 2, 3, 5, 8):  # within a vector or two
            around = whole.clone()
            check(tr, [whole[shift:shift + n]], 0.25)
            assert torch.equal(whole[:shift], around[:shift]) and torch.equal(whole[shift + n:], around[shift + n:])


def test_other_orders(tr):
    a = randn(1, 600 * 700, BF16).view(600, 700).t()
    check(tr, [a, randn(2, 24, F32).view(2, 3, 4).permute(2, 0, 1)], 1.0)
    check(tr, [a[:, :300]], 1.0)  # whole rows of the matrix below
    with pytest.raises(ValueError, match="gaps"):
        tr.dflash2_grad_clip([a[:300]])


@pytest.mark.parametrize("size", [1e-42, 1e-38, 1e-30, 1e-20, 1e15, 1e19, 1e30])
def test_squares_beyond_float32(tr, size):
    t = [randn(1, 5000, F32, size), randn(2, 70000, BF16, size), torch.zeros(100, device="cuda")]
    check(tr, t, norm64(t, "l2") / 2)
    ordinary = randn(3, 1000, F32)
    check(tr, [ordinary, *t], norm64([ordinary, *t], "l2") / 2)


def test_zeros(tr):
    t = [torch.zeros(10000, device="cuda"), torch.zeros(3, dtype=BF16, device="cuda")]
    check(tr, t, 1.0)
    check(tr, t, 0.0)
    t = [randn(1, 100, F32)]
    check(tr, t, 0.0)
    assert (t[0] == 0).all()


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_leaves_the_gradients(tr, kind, bad):
    t = [randn(1, 50000, BF16), randn(2, 300, F32), randn(3, 500, F16)]
    for which in range(3):
        for apart in (False, True):
            mine = [x.clone() for x in t]
            mine[which][7] = bad
            before = [x.clone() for x in mine]
            out = tr.dflash2_grad_clip(mine, max_norm=1.0, kind=kind,
                                       out=[torch.zeros_like(x) for x in mine] if apart else None)
            assert math.isnan(out["norm"]) if math.isnan(bad) else float(out["norm"]) == math.inf
            for a, b in zip(out["tensors"], before):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_alone(tr):
    t = [randn(i, 1000 + i, (BF16, F32)[i % 2]) for i in range(10)]
    before = [x.clone() for x in t]
    out = tr.dflash2_grad_clip(t)
    assert set(out) == {"norm"} and abs(float(out["norm"]) / norm64(t, "l2") - 1) <= NORM
    assert all(torch.equal(a, b) for a, b in zip(t, before))
    assert float(tr.dflash2_grad_clip([])["norm"]) == 0 and float(tr.dflash2_grad_clip([], max_norm=1.0)["norm"]) == 0
    assert float(tr.dflash2_grad_clip([torch.empty(0, device="cuda")], max_norm=1.0)["norm"]) == 0


def test_same_bits_captured_and_on_other_streams(tr):
    t = [randn(i, 10000 * (i + 1) + i, (BF16, F32, F16)[i % 3]) for i in range(9)]
    want = tr.dflash2_grad_clip(t, max_norm=1.0, out=[torch.empty_like(x) for x in t])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan = tr.GradClipPlan(t, max_norm=1.0, out=[torch.empty_like(x) for x in t], stream=s)
    with torch.cuda.stream(s):
        plan()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan()
    torch.cuda.synchronize()
    for _ in range(5):
        for o in plan.outputs["tensors"]:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.outputs["norm"], want["norm"])
        assert all(torch.equal(a, b) for a, b in zip(plan.outputs["tensors"], want["tensors"]))


def test_refused(tr):
    t = randn(1, 100, F32)
    with pytest.raises(ValueError, match="overlap"):
        tr.dflash2_grad_clip([t, t], max_norm=1.0)
    with pytest.raises(ValueError, match="overlap"):
        tr.dflash2_grad_clip([t[:60], t[50:]])
    with pytest.raises(ValueError, match="overlap"):
        tr.dflash2_grad_clip([t[:60]], max_norm=1.0, out=[t[20:80]])
    with pytest.raises(ValueError, match="max_norm"):
        tr.dflash2_grad_clip([t], max_norm=math.inf)
    with pytest.raises(ValueError, match="max_norm"):
        tr.dflash2_grad_clip([t], out=[torch.empty_like(t)])
    with pytest.raises(ValueError, match="kind"):
        tr.dflash2_grad_clip([t], kind="l1")
    with pytest.raises(TypeError, match="one of"):
        tr.dflash2_grad_clip([t.double()])
    with pytest.raises(ValueError, match="type, shape"):
        tr.dflash2_grad_clip([t], max_norm=1.0, out=[torch.empty(99, device="cuda")])


def test_what_is_bound_stays_bound(tr):
    t = [randn(i, 5000, F32) for i in range(3)]
    plan = tr.GradClipPlan(t, max_norm=1.0)
    want = tr.dflash2_grad_clip([x.clone() for x in t], max_norm=1.0)
    kept = plan.outputs["tensors"]
    t.clear()
    torch.cuda.synchronize()
    got = plan()
    assert got["norm"].shape == () and torch.equal(got["norm"], want["norm"])
    assert all(torch.equal(a, b) for a, b in zip(kept, want["tensors"]))
    x = randn(9, 100, F32)
    with pytest.raises(ValueError, match="overlap"):
        tr.dflash2_grad_clip([x], norm=x[3:4])
    assert tr.dflash2_grad_clip([x], norm=torch.zeros(1, device="cuda"))["norm"].shape == (1,)


@pytest.mark.parametrize("size", [1e-2, 1e20, 1e36])
@pytest.mark.parametrize("limit", [1.0, 1e-3, 1e-9, 1e-20, 1e-36])
def test_factors_below_float32(tr, size, limit):
    """max_norm / norm may be less than float32 holds, what it makes of an element is not."""
    for apart in (False, True):
        t = [randn(1, 5001, F32, size), randn(2, 7000, BF16, size), randn(3, 3, F32, size)]
        check(tr, t, limit, out=[torch.empty_like(x) for x in t] if apart else None)
        t = [randn(1, 5001, F32, size), randn(2, 7000, BF16, size)]
        check(tr, t, limit, "max", out=[torch.empty_like(x) for x in t] if apart else None)
