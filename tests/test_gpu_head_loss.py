"""The LM head's cross entropy and its gradient on the GPU, against their formulas in float64.

Tolerances.  A logit is a float32 sum of H exact products in steps of 16: under (H / 8 + 32) roundings of 2^-23 of the sum of
the products' magnitudes.  lse adds the rounding of exp2 (2^-22), of sums of positive terms (under 2^8 roundings, 2^-16) and its own.
dz is rounded to bf16 once (U = 2^-8 of each at most; up to 128 rows to two bf16, U^2) and carries its logit's error; a product adds its own sum's roundings and,
for bf16 outputs, U of the result.  Those bounds hold for every element.  Roundings to bf16 are as often up as down, so that in the
2-norm a result is off by about U / 2 / sqrt(3) twice over: below U.
"""
import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = torch.finfo(BF16).eps / 2

# borders of tiles (256 rows, 256 columns, 128 of K), of the packed rows (64) and of what is odd
SIZES = [(1, 8, 1), (1, 8, 5), (2, 16, 256), (3, 64, 257), (5, 72, 300), (127, 128, 511), (128, 128, 512), (129, 136, 1000),
         (256, 256, 256), (257, 64, 513), (300, 1024, 4096), (1000, 520, 3001), (17, 2048, 20011), (40, 4096, 9000),
         (513, 264, 77)]
# two pieces of the vocabulary, one with several blocks of the loss's rows, the others with d_hidden in parts, the last two
# with dz in two
LARGE = [(20000, 64, 14001), (2048, 72, 140001), (128, 8, 1100001), (127, 64, 1100001)]


@pytest.fixture(scope="module")
def tr():
    from speculative_decoding_drafter_gb300 import training

    return training


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def make(N, H, V, seed=0, ignored=True):
    g = torch.Generator(device="cuda").manual_seed(seed + N + 1000 * H + 7 * V)
    W = (randn(g, V, H) * (2.0 / math.sqrt(H))).to(BF16)
    labels = torch.randint(0, V, (N,), device="cuda", generator=g)
    hidden = (randn(g, N, H) + torch.rand(N, 1, device="cuda", generator=g) * 2 * W[labels].float()).to(BF16)
    labels = labels.to(torch.int32)
    labels[-1] = V - 1  # the last column
    if ignored and N > 2:
        labels[1], labels[N // 2] = -1, V
        labels[2::9] = -100
    grad = torch.rand(N, device="cuda", generator=g) / N
    return hidden, W, labels, grad


def logit_error(hidden, W):
    """Largest error of each row's logits."""
    H = hidden.shape[1]
    return (hidden.double().abs() @ W.double().abs().T).amax(1) * ((H / 8 + 32) * 2.0 ** -23)


def reference(hidden, W, labels):
    z = hidden.double() @ W.double().T
    lse = z.logsumexp(1)
    seen = (labels >= 0) & (labels < W.shape[0])
    rows = torch.arange(len(labels), device="cuda")
    at = labels.long().clamp(0, W.shape[0] - 1)
    return z, lse, torch.where(seen, lse - z[rows, at], torch.zeros_like(lse)), seen


def check_loss(out, hidden, W, labels):
    _, lse, loss, seen = reference(hidden, W, labels)
    bound = logit_error(hidden, W) + 2.0 ** -16 + lse.abs() * 2.0 ** -22
    assert ((out["lse"].double() - lse).abs() <= bound).all()
    assert ((out["loss"].double() - loss).abs() <= 2 * bound)[seen].all()
    assert (out["loss"][~seen] == 0).all()


def check_grad(out, hidden, W, labels, lse, grad):
    z = hidden.double() @ W.double().T
    seen = (labels >= 0) & (labels < W.shape[0])
    p = torch.exp(z - lse.double()[:, None])
    d = p.clone()
    rows = seen.nonzero()[:, 0]
    d[rows, labels[rows].long()] -= 1
    weight = torch.where(seen, grad.double(), torch.zeros_like(grad, dtype=torch.float64))[:, None]
    d, p = d * weight, p * weight.abs()
    # off by its rounding, and by its logit's and exp2's errors
    own = U if len(labels) > 128 else U * U
    slack = d.abs() * own + p * (logit_error(hidden, W)[:, None] * 1.01 + 2.0 ** -18)
    h = torch.where(seen[:, None], hidden, torch.zeros_like(hidden)).double()
    for name, a, b in (("d_hidden", d, W.double()), ("d_W", d.T, h)):
        if name not in out:
            continue
        want = a @ b
        got = out[name].double()
        s = slack if name == "d_hidden" else slack.T
        bound = s @ b.abs() + (a.abs() @ b.abs()) * ((a.shape[1] / 8 + 64) * 2.0 ** -23) + 2.0 ** -130
        if out[name].dtype == BF16:
            bound = bound + want.abs() * U
        bad = ~((got - want).abs() <= bound)
        assert not bad.any(), (name, int(bad.sum()), got[bad][:4], want[bad][:4], bad.nonzero()[:4])
        # (a result's own rounding alone is 0.6 U at most in the 2-norm, and U / 2 / sqrt(3) on average)
        assert (got - want).norm() <= (U if len(labels) > 128 else 0.6 * U) * want.norm() + 1e-30, name
        if name == "d_hidden":
            assert (out[name][~seen] == 0).all()


@pytest.mark.parametrize("N,H,V", SIZES)
def test_loss(tr, N, H, V):
    hidden, W, labels, _ = make(N, H, V)
    check_loss(tr.dflash2_lm_head_loss(hidden, W, labels), hidden, W, labels)


@pytest.mark.parametrize("N,H,V", SIZES)
def test_gradient(tr, N, H, V):
    hidden, W, labels, grad = make(N, H, V, 1)
    lse = reference(hidden, W, labels)[1].float()
    check_grad(tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad), hidden, W, labels, lse, grad)


@pytest.mark.parametrize("N,H,V", LARGE)
def test_pieces(tr, N, H, V):
    hidden, W, labels, grad = make(N, H, V, 2)
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    check_loss(out, hidden, W, labels)
    check_grad(tr.dflash2_lm_head_loss_grad(hidden, W, labels, out["lse"], grad), hidden, W, labels, out["lse"], grad)


@pytest.mark.parametrize("N", [3, 60, 200, 300])
def test_one_of_the_two_and_float32(tr, N):
    hidden, W, labels, grad = make(N, 200, 700, 3)
    lse = tr.dflash2_lm_head_loss(hidden, W, labels)["lse"]
    both = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad)
    only = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad, d_W=False)
    assert set(only) == {"d_hidden"} and torch.equal(only["d_hidden"], both["d_hidden"])
    only = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad, d_hidden=False)
    assert set(only) == {"d_W"} and torch.equal(only["d_W"], both["d_W"])
    wide = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad, d_W=torch.full((700, 200), 9.0, device="cuda"))
    assert torch.equal(wide["d_W"].to(BF16), both["d_W"])
    check_grad(wide, hidden, W, labels, lse, grad)


def test_ignored_rows_may_hold_anything(tr):
    hidden, W, labels, grad = make(70, 136, 600, 4)
    want = tr.dflash2_lm_head_loss(hidden, W, labels)
    back = tr.dflash2_lm_head_loss_grad(hidden, W, labels, want["lse"], grad)
    seen = (labels >= 0) & (labels < 600)
    hidden[~seen] = math.nan
    grad[~seen] = math.inf
    lse = torch.where(seen, want["lse"], torch.full_like(want["lse"], -math.inf))
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    assert torch.equal(out["loss"], want["loss"]) and torch.equal(out["lse"][seen], want["lse"][seen])
    got = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad)
    for name in back:
        assert torch.equal(got[name], back[name])
    labels.fill_(-1)
    got = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad)
    assert (got["d_hidden"] == 0).all() and (got["d_W"] == 0).all()
    assert (tr.dflash2_lm_head_loss(hidden, W, labels)["loss"] == 0).all()


def test_rows_that_are_not_finite(tr):
    hidden, W, labels, _ = make(300, 64, 400, 5, ignored=False)
    want = tr.dflash2_lm_head_loss(hidden, W, labels)
    hidden[7, 3], hidden[260, 1] = math.nan, math.inf
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    other = torch.ones(300, dtype=torch.bool, device="cuda")
    other[[7, 260]] = False
    assert torch.equal(out["loss"][other], want["loss"][other])
    assert not out["loss"][~other].isfinite().any()


def test_extreme_logits(tr):
    """A token far above all others, and one far below: no exponential overflows, and what is nothing is nothing."""
    H, V = 64, 1000
    W = torch.zeros(V, H, dtype=BF16, device="cuda")
    W[:, 0] = torch.linspace(-1, 1, V, device="cuda").to(BF16)
    W[500, 1] = 1
    hidden = torch.zeros(4, H, dtype=BF16, device="cuda")
    hidden[0, 0], hidden[1, 0], hidden[2, 1], hidden[3, 1] = 1e4, -1e4, 3e4, -3e4
    labels = torch.tensor([0, 0, 500, 500], dtype=torch.int32, device="cuda")
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    check_loss(out, hidden, W, labels)
    grad = torch.ones(4, device="cuda")
    got = tr.dflash2_lm_head_loss_grad(hidden, W, labels, out["lse"], grad)
    assert all(t.isfinite().all() for t in got.values())
    # a vocabulary whose rows are all alike
    hidden, W, labels, _ = make(9, 64, 3000, 6)
    W[:] = W[0].clone()
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    seen = (labels >= 0) & (labels < 3000)
    assert ((out["loss"][seen] - math.log(3000)).abs() <= 2.0 ** -15).all()


def test_gradient_against_differences(tr):
    N, H, V = 6, 40, 90
    hidden, W, labels, grad = make(N, H, V, 7)
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    back = tr.dflash2_lm_head_loss_grad(hidden, W, labels, out["lse"], grad)
    g = torch.Generator(device="cuda").manual_seed(9)

    def total(h, w):
        z = h @ w.T
        seen = (labels >= 0) & (labels < V)
        rows = seen.nonzero()[:, 0]
        return float(((z.logsumexp(1)[rows] - z[rows, labels[rows].long()]) * grad.double()[rows]).sum())

    h64, w64, step = hidden.double(), W.double(), 1e-5
    for _ in range(4):
        v, w = randn(g, N, H).double(), randn(g, V, H).double()
        for name, along, arg in (("d_hidden", (v, 0), v), ("d_W", (0, w), w)):
            diff = (total(h64 + step * along[0], w64 + step * along[1]) -
                    total(h64 - step * along[0], w64 - step * along[1])) / (2 * step)
            # every term is off by its own rounding and its operands'
            assert abs(diff - float((back[name].double() * arg).sum())) <= \
                4 * U * float((back[name].double() * arg).abs().sum()) + 1e-6


def test_no_rows(tr):
    hidden, W = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(300, 64, dtype=BF16, device="cuda")
    none, ids = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert tr.dflash2_lm_head_loss(hidden, W, ids)["loss"].shape == (0,)
    for dtype in (BF16, F32):
        out = tr.dflash2_lm_head_loss_grad(hidden, W, ids, none, none, d_W=torch.full((300, 64), 2.0, device="cuda").to(dtype))
        assert (out["d_W"] == 0).all()


def test_captured_replayed_shared_workspace_and_streams(tr):
    from speculative_decoding_drafter_gb300 import dflash2 as df

    hidden, W, labels, grad = make(150, 320, 2000, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = tr.LossWorkspace(150, 320, 2000)
        forward = tr.LossPlan(hidden, W, labels, workspace=ws)
        backward = tr.LossGradPlan(hidden, W, labels, forward.outputs["lse"], grad, workspace=ws)
        forward(), backward()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            forward(), backward()
    torch.cuda.synchronize()
    for sign in (-1, -1):
        hidden.mul_(sign)
        for t in (*forward.outputs.values(), *backward.outputs.values()):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        a = tr.dflash2_lm_head_loss(hidden, W, labels)
        b = tr.dflash2_lm_head_loss_grad(hidden, W, labels, a["lse"], grad)
        for name, t in {**a, **b}.items():
            assert torch.equal({**forward.outputs, **backward.outputs}[name], t)
        check_loss(a, hidden, W, labels)
    df.dflash2_check_device_status(ws)


def test_same_bits_beside_other_work(tr):
    """Results do not depend on which tiles are first: alone, and beside copies that keep the memory busy."""
    hidden, W, labels, grad = make(700, 1024, 6000, 9)
    want = tr.dflash2_lm_head_loss(hidden, W, labels)
    back = tr.dflash2_lm_head_loss_grad(hidden, W, labels, want["lse"], grad)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    for _ in range(10):
        with torch.cuda.stream(s):
            for _ in range(8):
                y.copy_(x)
        a = tr.dflash2_lm_head_loss(hidden, W, labels)
        b = tr.dflash2_lm_head_loss_grad(hidden, W, labels, want["lse"], grad)
        for name, t in {**want, **back}.items():
            assert torch.equal({**a, **b}[name], t)
    torch.cuda.synchronize()


def test_two_threads(tr):
    failed = []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            hidden, W, labels, grad = make(100 + 200 * seed, 256, 900 + seed, seed)
            a = tr.dflash2_lm_head_loss(hidden, W, labels)
            b = tr.dflash2_lm_head_loss_grad(hidden, W, labels, a["lse"], grad)
            torch.cuda.synchronize()
            forward = tr.LossPlan(hidden, W, labels, stream=s)
            backward = tr.LossGradPlan(hidden, W, labels, a["lse"], grad, stream=s)
            for _ in range(10):
                forward(), backward()
            s.synchronize()
            if not all(torch.equal({**forward.outputs, **backward.outputs}[n], t) for n, t in {**a, **b}.items()):
                failed.append(seed)
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed


def test_refused(tr):
    hidden, W, labels, grad = make(4, 64, 100)
    with pytest.raises(ValueError, match="shape"):
        tr.dflash2_lm_head_loss(hidden[:, :56].contiguous(), W, labels)
    with pytest.raises(TypeError, match="labels"):
        tr.dflash2_lm_head_loss(hidden, W, labels.long())
    with pytest.raises(ValueError, match="sizes"):
        tr.dflash2_lm_head_loss(hidden[:, :60].contiguous(), W[:, :60].contiguous(), labels)
    with pytest.raises(ValueError, match="left out"):
        tr.dflash2_lm_head_loss_grad(hidden, W, labels, grad, grad, d_hidden=False, d_W=False)
    with pytest.raises(ValueError, match="overlaps"):
        tr.dflash2_lm_head_loss_grad(hidden, W, labels, grad, grad, d_W=W)
    with pytest.raises(ValueError, match="overlaps"):
        tr.dflash2_lm_head_loss(hidden, W, labels, loss=grad, lse=grad)
    with pytest.raises(TypeError, match="d_W"):
        tr.dflash2_lm_head_loss_grad(hidden, W, labels, grad, grad, d_W=W.half())
    with pytest.raises(ValueError, match="workspace"):
        tr.dflash2_lm_head_loss_grad(hidden, W, labels, grad, grad, workspace=tr.LossWorkspace(1, 64, 100, grad=False))


@pytest.mark.parametrize("H", [64, 72])
@pytest.mark.parametrize("N,kept", [(1, 0), (40, 7), (65, 64), (128, 0), (128, 1), (128, 128), (129, 100), (256, 3), (300, 0),
                                    (300, 1), (300, 128), (300, 129), (300, 256), (300, 257), (70000, 3000)])
def test_rows_left_by_the_labels(tr, N, kept, H):
    """As many rows as stages and tiles end at, spread over all; what a workspace held before does not matter."""
    hidden, W, labels, grad = make(N, H, 520, kept, ignored=False)
    order = torch.randperm(N, generator=torch.Generator().manual_seed(kept))[:N - kept].cuda()
    labels[order] = -1
    hidden[order] = math.nan
    lse = tr.dflash2_lm_head_loss(hidden, W, labels)["lse"]
    ws = tr.LossWorkspace(N, H, 520)
    ws.view[256:] = 255  # NaN in every type
    out = tr.dflash2_lm_head_loss_grad(hidden, W, labels, lse, grad, workspace=ws)
    hidden[order] = 0
    check_grad(out, hidden, W, labels, torch.where(lse.isnan(), torch.zeros_like(lse), lse), grad)


def test_rows_in_several_blocks(tr):
    """A vocabulary so large that the loss takes 256 rows at a time."""
    N, H, V = 600, 16, 5000001
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.empty(V, H, dtype=BF16, device="cuda").normal_(0, 0.5, generator=g)
    hidden = randn(g, N, H).to(BF16)
    labels = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    labels[::7] = -1
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    lse, loss = [], []
    for r in range(0, N, 100):
        _, a, b, _ = reference(hidden[r:r + 100], W, labels[r:r + 100])
        lse.append(a), loss.append(b)
    lse, loss = torch.cat(lse), torch.cat(loss)
    # (the sums of exponentials of 39,064 tiles' halves: their joins add 2^-22 each at most, in 10 levels and turns of 128)
    bound = 2.0 ** -12 * (1 + lse.abs())
    assert ((out["lse"].double() - lse).abs() <= bound).all() and ((out["loss"].double() - loss).abs() <= 2 * bound).all()


# few rows before a large W, which the kernels read from copies: one copy for each of many pairs and fewer, widths that are a
# multiple of 128, of 64 and of neither
@pytest.mark.parametrize("N,H,V", [(1, 64, 600001), (1, 2048, 20011), (3, 4160, 9001), (15, 1000, 40009), (100, 136, 260001),
                                   (128, 192, 200003)])
def test_few_rows_of_a_large_head(tr, N, H, V):
    hidden, W, labels, grad = make(N, H, V)
    f = tr.dflash2_lm_head_loss(hidden, W, labels)
    check_loss(f, hidden, W, labels)
    seen = (labels >= 0) & (labels < V)
    anything = torch.where(seen[:, None], hidden, torch.full_like(hidden, math.nan))
    out = tr.dflash2_lm_head_loss_grad(anything, W, labels, f["lse"], grad)
    check_grad(out, hidden, W, labels, f["lse"], grad)
    again = tr.dflash2_lm_head_loss_grad(anything, W, labels, f["lse"], grad)
    assert torch.equal(out["d_hidden"], again["d_hidden"]) and torch.equal(out["d_W"], again["d_W"])
    if N > 3:  # a row that is not finite leaves the others as they are
        bad = hidden.clone()
        bad[3, ::2] = math.inf
        b = tr.dflash2_lm_head_loss(bad, W, labels)
        rest = torch.arange(N, device="cuda") != 3
        assert torch.equal(b["lse"][rest], f["lse"][rest]) and torch.equal(b["loss"][rest], f["loss"][rest])


@pytest.mark.parametrize("N,H", [(16, 4096), (16, 16384), (128, 4160), (200, 4096), (300, 16384)])
def test_confident_rows(tr, N, H):
    """Rows that are nearly fitted: 1 - p of the label from 1e-3 to 1e-5, which is what is left of their gradient.

    The logits of both passes are the same sums, so what they are off by moves every probability by its own share, as
    other logits would (rel below), and leaves in 1 - p only what lse and exp2 lose: lse's rounding (2^-20 below 32), under
    40 roundings of 2^-24 of the sum around its largest term, exp2 twice (2^-22), log2(e) as float32 (2^-26 of 32): 2^-17."""
    V = 2048
    g = torch.Generator(device="cuda").manual_seed(N + H)
    W = (randn(g, V, H) / math.sqrt(H)).to(BF16)
    labels = torch.randint(0, V, (N,), device="cuda", generator=g)
    top = torch.linspace(math.log(1e3 * V), math.log(1e5 * V), N, device="cuda")[:, None]
    own = W[labels].float()
    hidden = (randn(g, N, H) + top * own / own.square().sum(1, keepdim=True)).to(BF16)
    labels = labels.int()
    z, lse, _, _ = reference(hidden, W, labels)
    assert lse.max() < 32
    f = tr.dflash2_lm_head_loss(hidden, W, labels)
    got = tr.dflash2_lm_head_loss_grad(hidden, W, labels, f["lse"], torch.ones(N, device="cuda"), d_W=False)["d_hidden"]
    rows = torch.arange(N, device="cuda")
    d = torch.exp(z - lse[:, None])
    d[rows, labels.long()] = 0
    d[rows, labels.long()] = -d.sum(1)  # p - 1 of the label
    want = d @ W.double()
    rel = torch.expm1(2 * logit_error(hidden, W)) + 2.0 ** -16
    size = W.double().norm(dim=1)
    parts = (d.abs() * size).sum(1)
    rounded = (U if N > 128 else U * U) + (V / 8 + 64) * 2.0 ** -23
    bound = parts * (rel + rounded) + 2.0 ** -17 * size[labels.long()] + U * want.norm(dim=1)
    off = (got.double() - want).norm(dim=1)
    assert (off <= bound).all(), (off / bound).max()


def test_logits_are_summed_in_groups(tr):
    """Products that are all positive, so that what an accumulator cuts off adds up: at most 2^-23 of what it holds, at each of
    its steps of 16 products.  A group of 768 takes 48 steps and holds half of its sum on average: it loses 24 times 2^-23 of
    the sum at most, and the additions of the six sums are rounded, 2^-24 each: below 2^-18 of a logit.  One accumulator for
    all 4096 loses 128 times 2^-23 at most, and half of that on average (lse was off by twice the bound)."""
    N, H, V = 20, 4096, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    W = ((0.5 + torch.rand(V, H, device="cuda", generator=g)) / 256).to(BF16)
    hidden = (0.5 + torch.rand(N, H, device="cuda", generator=g)).to(BF16)
    labels = torch.arange(N, device="cuda", dtype=torch.int32) % V
    out = tr.dflash2_lm_head_loss(hidden, W, labels)
    z, lse, _, _ = reference(hidden, W, labels)
    # (exp2 and the sum of eight: 2^-22 and 16 roundings of 2^-24; lse's own)
    bound = z.abs().amax(1) * 2.0 ** -18 + 2.0 ** -20 + lse.abs() * 2.0 ** -23
    assert ((out["lse"].double() - lse).abs() <= bound).all(), ((out["lse"].double() - lse).abs() / bound).max()
