"""Rotary positions, the paged cache and attention over it, on the GPU against float64 plain forms."""
import math

import pytest
import torch

from attention_rules import BF16, EPS16, Batch, attend, attend_bound, quantise, rotate, rotate32, rotate_bound

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module")
def at():
    from speculative_decoding_drafter_gb300 import attention

    return attention


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def make_table(max_pos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], 1).float().cuda().contiguous()


# ------------------------------------------------------------------------------------------- rotation


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,heads,dim,rot", [(1, 1, 64, 64), (3, 5, 128, 128), (17, 40, 128, 96), (5, 7, 80, 40),
                                             (9, 3, 8, 2), (4, 2, 256, 256), (6, 33, 200, 50), (2000, 11, 128, 64)])
def test_rope(at, N, heads, dim, rot, interleaved):
    g = gen(N + dim + rot)
    x = randn(g, N, heads, dim).to(BF16)
    pos = torch.randint(0, 5000, (N,), device="cuda", generator=g, dtype=torch.int32)
    table = make_table(5000, rot)
    for inverse in (False, True):
        want = rotate(x, table, pos, interleaved, inverse)
        got = at.dflash2_rope(x, pos, table, interleaved=interleaved, inverse=inverse)
        assert ((got.double() - want).abs() <= rotate_bound(x, want)).all()
        assert torch.equal(got[..., rot:], x[..., rot:])
        inplace = x.clone()
        at.dflash2_rope(inplace, pos, table, interleaved=interleaved, inverse=inverse, out=inplace)
        assert torch.equal(inplace, got)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_takes_views_and_table_offsets(at, interleaved):
    """Views of a fused projection, a table that is not 16-byte aligned, outputs laid out heads first."""
    g = gen(5)
    qkv = randn(g, 13, 10, 64).to(BF16)
    pos = torch.arange(13, device="cuda", dtype=torch.int32)
    flat = torch.empty(100 * 64 + 1, device="cuda")
    table = flat[1:].view(100, 2, 32)
    table.copy_(make_table(100, 64))
    x = qkv[:, 3:8]
    out = torch.zeros(5, 13, 64, dtype=BF16, device="cuda").transpose(0, 1)
    at.dflash2_rope(x, pos, table, interleaved=interleaved, out=out)
    assert torch.equal(out, at.dflash2_rope(x.contiguous(), pos, make_table(100, 64), interleaved=interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(at, interleaved):
    """<rope(x + e), w> - <rope(x), w> = <e, inverse(w)>: the map is linear, so a difference of any size is the
    derivative; and turning back gives x."""
    g = gen(8)
    N, heads, dim = 6, 4, 128
    pos = torch.randint(0, 900, (N,), device="cuda", generator=g, dtype=torch.int32)
    table = make_table(900, 96)
    x, e, w = (randn(g, N, heads, dim).to(BF16) for _ in range(3))
    xe = (x.float() + e.float()).to(BF16)
    f = lambda t, inv=False: at.dflash2_rope(t, pos, table, interleaved=interleaved, inverse=inv)  # noqa: E731
    left = ((f(xe).double() - f(x).double()) * w.double()).sum()
    right = ((xe.double() - x.double()) * f(w, True).double()).sum()
    # each of the 3 N heads dim rounded products is off by at most 2^-8 of itself
    size = ((f(xe).double().abs() + f(x).double().abs()) * w.double().abs()).sum() + \
        ((xe.double() - x.double()).abs() * f(w, True).double().abs()).sum()
    assert (left - right).abs() <= EPS16 * size
    back = f(f(x), True).double()
    assert ((back - x.double()).abs() <= 3 * EPS16 * x.double().abs().amax(-1, keepdim=True)).all()


def frequencies(kind, rot, theta, factor, original_len, low, high):
    out = []
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if kind == "linear":
            f /= factor
        elif kind == "base":
            f = (theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        elif kind == "ramp":
            at_turns = lambda r: rot * math.log(original_len / (r * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
            a, b = max(math.floor(at_turns(high)), 0), min(math.ceil(at_turns(low)), rot - 1)
            w = min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
            f = f * (1 - w) + f / factor * w
        elif kind == "band":
            wavelength = 2 * math.pi / f
            if wavelength > original_len / low:
                f /= factor
            elif wavelength >= original_len / high:
                w = (original_len / wavelength - low) / (high - low)
                f = (1 - w) * f / factor + w * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("kind,factor,low,high,mult", [("plain", 1.0, 1.0, 32.0, 1.0), ("linear", 4.0, 1.0, 32.0, 1.0),
                                                       ("base", 8.0, 1.0, 32.0, 1.0), ("ramp", 16.0, 1.0, 32.0, 1.277),
                                                       ("band", 8.0, 1.0, 4.0, 1.0)])
@pytest.mark.parametrize("rot", [6, 64, 128])
def test_rope_table(at, kind, factor, low, high, mult, rot):
    P = 70001
    got = at.dflash2_rope_table(P, rot, theta=500000.0, kind=kind, factor=factor, original_len=8192.0, low=low,
                                high=high, multiplier=mult).cpu().double()
    a = torch.arange(P, dtype=torch.float64)[:, None] * frequencies(kind, rot, 500000.0, factor, 8192.0, low, high)
    want = torch.stack([a.cos(), a.sin()], 1) * mult
    # one rounding to float32 (half a unit in the last place: 2^-25 up to 1, 2^-24 up to 2), and an angle that is off
    # by a few 2^-53 of itself on each side
    assert (got - want).abs().max() <= (2.0 ** -25 if mult <= 1 else 2.0 ** -24) + mult * P * 2.0 ** -49


# ---------------------------------------------------------------------------------------------- cache

BATCHES = [([1], [1], 8), ([40, 7, 100], [3, 7, 1], 16), ([33, 0, 65], [33, 0, 2], 24), ([5], [9], 8),
           ([300, 17, 128, 64, 1], [200, 17, 64, 1, 1], 64)]


@pytest.mark.parametrize("dtype", [BF16, E4M3, INT8])
@pytest.mark.parametrize("lens,news,ps", BATCHES)
@pytest.mark.parametrize("qh,kvh,dim,rot,interleaved", [(8, 2, 128, 128, False), (5, 5, 80, 40, True), (3, 1, 48, 22, False)])
def test_append_and_read(at, dtype, lens, news, ps, qh, kvh, dim, rot, interleaved):
    g = gen(sum(lens) + dim)
    b = Batch(lens, news, ps, seed=3)
    tokens = b.on_gpu(at)
    qkv = randn(g, b.N, qh + 2 * kvh, dim).to(BF16)
    q, k, v = qkv.split([qh, kvh, kvh], 1)
    if b.N > 2:
        k[1, 0] = 0                 # a row of zeros
        v[0, 0] *= 2.0 ** -120      # a row below what 8 bits hold
        v[2, kvh - 1, 5] = math.inf
    table = make_table(400, rot)
    cache = at.PagedCache.allocate(b.pages, ps, kvh, dim, dtype)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x11)
    places = b.places()
    pos = torch.tensor([p[1] for p in places], device="cuda").clamp(min=0)
    out = at.dflash2_cache_append(cache, tokens, k, v, q=q, table=table, interleaved=interleaved)
    want_q = rotate(q, table, pos, interleaved)
    assert ((out["q"].double() - want_q).abs() <= rotate_bound(q, want_q)).all()
    k32 = rotate32(k.cpu(), table.cpu(), pos.cpu(), interleaved)
    read = at.dflash2_cache_read(cache, tokens)
    touched = torch.zeros(b.pages, ps, dtype=torch.bool)
    for name, x32 in (("k", k32), ("v", v.cpu().float())):
        held = getattr(cache, name).view(torch.uint8 if dtype != BF16 else BF16).cpu()
        if dtype != BF16:
            codes, scales = quantise(x32, dtype)
            codes, got_scales = codes.view(torch.uint8), getattr(cache, name + "_scale").cpu()
        for n, (_, p, page, slot) in enumerate(places):
            if p < 0:
                assert not read[name][n].any()
                continue
            touched[page, slot] = True
            if dtype == BF16:
                assert torch.equal(held[page, :, slot], x32[n].to(BF16))
                assert torch.equal(read[name][n].cpu(), x32[n].to(BF16))
                continue
            # the same float32 operations on both sides: the same bits
            ok = torch.isfinite(scales[n])
            assert torch.equal(held[page, :, slot][ok], codes[n][ok])
            assert torch.equal(got_scales[page, :, slot][ok], scales[n][ok])
            value = codes[n].view(dtype).float() * scales[n][:, None]
            assert torch.equal(read[name][n].cpu()[ok], value.to(BF16)[ok])
            assert torch.isnan(read[name][n].cpu()[~ok]).all()
            step = 2.0 ** -4 if dtype == E4M3 else 0.5 / 127  # half a step of the codes
            big = x32[n][ok].abs().amax(-1, keepdim=True)
            err = (value[ok] - x32[n][ok]).abs()
            assert (err <= (step * x32[n][ok].abs() + 2.0 ** -10 / 448 * big if dtype == E4M3 else step * big) * 1.0001
                    + 1e-30).all()
    # nothing else was written
    for t in (cache.k, cache.v):
        rest = t.view(torch.uint8).cpu().permute(0, 2, 1, 3)[~touched]
        assert (rest == 0x11).all()


def test_append_without_rotation_or_queries(at):
    g = gen(1)
    b = Batch([20, 31], [20, 5], 16)
    cache = at.PagedCache.allocate(b.pages, 16, 3, 64)
    k, v = randn(g, b.N, 3, 64).to(BF16), randn(g, b.N, 3, 64).to(BF16)
    out = at.dflash2_cache_append(cache, b.on_gpu(at), k, v)
    assert set(out) == {"k_cache", "v_cache"}
    read = at.dflash2_cache_read(cache, b.on_gpu(at))
    assert torch.equal(read["k"], k) and torch.equal(read["v"], v)
    only = torch.zeros_like(v)
    assert set(at.dflash2_cache_read(cache, b.on_gpu(at), v_out=only)) == {"v"}
    assert torch.equal(only, v)


def test_page_ids_out_of_range_are_not_followed(at):
    g = gen(2)
    b = Batch([40], [40], 16)
    b.table[0, 1] = -1
    b.table[0, 2] = b.pages
    cache = at.PagedCache.allocate(b.pages, 16, 2, 64)
    k = randn(g, 40, 2, 64).to(BF16)
    at.dflash2_cache_append(cache, b.on_gpu(at), k, k)
    read = at.dflash2_cache_read(cache, b.on_gpu(at))["k"]
    assert torch.equal(read[:16], k[:16]) and not read[16:].any()


# ------------------------------------------------------------------------------------------ attention


def filled(at, b, kvh, dim, dtype, seed, spread=1.0):
    """A cache with random rows, NaN bytes wherever no position below a length lives, and its float64 rows."""
    g = gen(seed)
    cache = at.PagedCache.allocate(b.pages, b.page_size, kvh, dim, dtype)
    whole = Batch(b.lens, b.lens, b.page_size)
    whole.table, whole.pages = b.table, b.pages
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0xFF)  # NaN as bf16 and as e4m3
    if cache.k_scale is not None:
        cache.k_scale.fill_(math.nan)
        cache.v_scale.fill_(math.nan)
    k = (randn(g, whole.N, kvh, dim) * spread).to(BF16)
    v = (randn(g, whole.N, kvh, dim) * torch.rand(whole.N, kvh, 1, device="cuda", generator=g) * 3).to(BF16)
    rows = {"k": [], "v": []}
    if whole.N:
        at.dflash2_cache_append(cache, whole.on_gpu(at), k, v)
    for name in rows:
        codes, scale = getattr(cache, name), getattr(cache, name + "_scale")
        for s, n in enumerate(b.lens):
            p = torch.arange(n, device="cuda")
            pages, slots = b.table.cuda()[s][p // b.page_size].long(), p % b.page_size
            if dtype == BF16:
                rows[name].append(codes[pages, :, slots].double())
            else:
                r = codes.view(torch.uint8)[pages, :, slots].view(dtype).double()
                rows[name].append(r * scale[pages, :, slots].double()[..., None])
    return cache, rows["k"], rows["v"]


def check(at, lens, news, ps, qh, kvh, dim, dtype, causal, window, seed=0, scale=None, spread=1.0):
    b = Batch(lens, news, ps, seed=seed, poison=True)
    cache, k, v = filled(at, b, kvh, dim, dtype, seed, spread)
    q = randn(gen(seed + 1), b.N, qh, dim).to(BF16)
    sc = dim ** -0.5 if scale is None else scale
    want, mag, lse = attend(q, k, v, b.lens, b.news, sc, causal, window)
    got = at.dflash2_paged_attention(q, cache, b.on_gpu(at), causal=causal, window=window, scale=scale)
    err = (got["out"].double() - want).abs()
    bad = ~(err <= attend_bound(want, mag))
    assert not bad.any(), (int(bad.sum()), bad.numel(), float(err[bad].max()), bad.nonzero()[:5].tolist())
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(got["lse"]), empty) and (got["lse"][empty] < 0).all()
    assert not got["out"][empty].any()
    # float32 scores of size up to 2^4 summed over dim terms, and a sum of positive terms
    assert ((got["lse"].double() - lse)[~empty].abs() <= 2.0 ** -14 * (1 + lse[~empty].abs())).all()
    return b, cache, q, got


TYPES = pytest.mark.parametrize("dtype", [BF16, E4M3, INT8])


@TYPES
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,news,ps", [
    ([1], [1], 8), ([2], [1], 16), ([127], [1], 16), ([128], [1], 64), ([129], [1], 128), ([777], [1], 16),
    ([300, 1, 64, 1000], [8, 1, 8, 8], 24), ([50, 0, 3, 130], [16, 0, 3, 16], 40),
    ([5, 260], [9, 4], 8), ([0, 70], [4, 70], 32),
    ([400], [150], 64), ([333, 129], [333, 1], 256), ([700, 90, 515], [515, 90, 2], 8)])
def test_attention_lengths_and_pages(at, dtype, causal, lens, news, ps):
    check(at, lens, news, ps, 8, 2, 128, dtype, causal, 0, seed=len(lens))


@TYPES
@pytest.mark.parametrize("qh,kvh,dim", [(1, 1, 64), (7, 1, 64), (6, 2, 96), (20, 4, 80), (16, 1, 128), (64, 1, 16),
                                        (3, 3, 48), (10, 2, 112), (33, 3, 128)])
def test_attention_heads(at, dtype, qh, kvh, dim):
    check(at, [530, 31], [40, 5], 32, qh, kvh, dim, dtype, True, 0, seed=dim)


@TYPES
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 2, 64, 129, 1000])
def test_attention_windows(at, dtype, causal, window):
    check(at, [700, 16, 260], [33, 16, 200], 16, 4, 2, 64, dtype, causal, window, seed=window)


@TYPES
def test_attention_pages_given_back_below_the_window(at, dtype):
    """The page-table entries and the values of positions that no row sees are never used."""
    b = Batch([900], [4], 32, poison=True)
    cache, k, v = filled(at, b, 2, 128, dtype, 4)
    q = randn(gen(9), 4, 8, 128).to(BF16)
    first = at.dflash2_paged_attention(q, cache, b.on_gpu(at), window=100)
    gone = b.table[0, :(900 - 4 - 100 + 1) // 32].clone()
    cache.k.view(torch.uint8)[gone.cuda().long()] = 0xFF
    cache.v.view(torch.uint8)[gone.cuda().long()] = 0xFF
    b.table[0, :len(gone)] = -7
    again = at.dflash2_paged_attention(q, cache, b.on_gpu(at), window=100)
    assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])
    want, mag, _ = attend(q, k, v, b.lens, b.news, 128 ** -0.5, True, 100)
    assert ((again["out"].double() - want).abs() <= attend_bound(want, mag)).all()


@TYPES
def test_attention_large_and_negative_scales(at, dtype):
    """Scores of hundreds: one key takes all the weight, and sums of far smaller ones must not spill."""
    for scale, spread in ((-0.05, 1.0), (0.0, 1.0), (0.02, 4.0)):
        check(at, [600, 45], [17, 3], 16, 4, 1, 64, dtype, True, 0, seed=3, scale=scale, spread=spread)


@TYPES
def test_attention_rising_scores(at, dtype):
    """Keys whose scores grow along the sequence, so the running maximum moves in every tile."""
    n, dim = 1200, 64
    b = Batch([n], [5], 40)
    cache = at.PagedCache.allocate(b.pages, 40, 1, dim, dtype)
    g = gen(6)
    q = torch.ones(5, 2, dim, device="cuda").to(BF16)
    k = (torch.linspace(-12, 12, n, device="cuda")[:, None, None] / 8 + 0.02 * randn(g, n, 1, dim)).to(BF16)
    v = (randn(g, n, 1, dim) * torch.logspace(-3, 3, n, device="cuda")[:, None, None]).to(BF16)
    whole = Batch([n], [n], 40)
    whole.table, whole.pages = b.table, b.pages
    at.dflash2_cache_append(cache, whole.on_gpu(at), k, v)
    if dtype != BF16:
        p = torch.arange(n, device="cuda")
        pages, slots = b.table.cuda()[0][p // 40].long(), p % 40
        rows = [getattr(cache, c).view(torch.uint8)[pages, :, slots].view(dtype).double() *
                getattr(cache, c + "_scale")[pages, :, slots].double()[..., None] for c in ("k", "v")]
    else:
        rows = [k.double(), v.double()]
    want, mag, lse = attend(q, [rows[0]], [rows[1]], [n], [5], 0.125, True, 0)
    got = at.dflash2_paged_attention(q, cache, b.on_gpu(at), scale=0.125)
    assert ((got["out"].double() - want).abs() <= attend_bound(want, mag)).all()
    assert ((got["lse"].double() - lse).abs() <= 2.0 ** -14 * (1 + lse.abs())).all()


@TYPES
def test_attention_values_far_from_one(at, dtype):
    """Values of 2^-60 and 2^60 and rows of zeros among them: nothing rests on their size."""
    n, dim = 300, 128
    b = Batch([n], [3], 16)
    cache = at.PagedCache.allocate(b.pages, 16, 2, dim, dtype)
    g = gen(7)
    size = torch.tensor([2.0 ** -60, 2.0 ** 60], device="cuda")[None, :, None]
    k, v = randn(g, n, 2, dim).to(BF16), (randn(g, n, 2, dim) * size).to(BF16)
    v[10:20] = 0
    whole = Batch([n], [n], 16)
    whole.table, whole.pages = b.table, b.pages
    at.dflash2_cache_append(cache, whole.on_gpu(at), k, v)
    read = at.dflash2_cache_read(cache, whole.on_gpu(at))
    q = (randn(g, 3, 4, dim) * torch.tensor([1.0, 2.0 ** -40, 0.0], device="cuda")[:, None, None]).to(BF16)
    if dtype == BF16:
        rows = [k.double(), v.double()]
    else:
        p = torch.arange(n, device="cuda")
        pages, slots = b.table.cuda()[0][p // 16].long(), p % 16
        rows = [getattr(cache, c).view(torch.uint8)[pages, :, slots].view(dtype).double() *
                getattr(cache, c + "_scale")[pages, :, slots].double()[..., None] for c in ("k", "v")]
    want, mag, _ = attend(q, [rows[0]], [rows[1]], [n], [3], dim ** -0.5, True, 0)
    got = at.dflash2_paged_attention(q, cache, b.on_gpu(at))
    assert ((got["out"].double() - want).abs() <= attend_bound(want, mag)).all()
    assert read["v"].dtype == BF16


def test_attention_takes_views_and_streams(at):
    """Queries inside a fused projection, outputs laid out heads first, a side stream, a plan called twice: the
    same bits; and the workspace's status word stays clear."""
    from speculative_decoding_drafter_gb300 import dflash2 as df

    b, cache, q, ref = check(at, [900, 33, 260], [16, 16, 16], 64, 8, 2, 128, BF16, True, 0)
    fused = torch.zeros(b.N, 12, 128, dtype=BF16, device="cuda")
    fused[:, 2:10] = q
    out = torch.zeros(8, b.N, 128, dtype=BF16, device="cuda").transpose(0, 1)
    ws = at.AttentionWorkspace(cache, b.on_gpu(at), 8)
    at.dflash2_paged_attention(fused[:, 2:10], cache, b.on_gpu(at), out=out, workspace=ws)
    assert torch.equal(out, ref["out"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = at.dflash2_paged_attention(q, cache, b.on_gpu(at), stream=stream)
        side.synchronize()
        assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])
    plan = at.PagedAttentionPlan(q, cache, b.on_gpu(at), workspace=ws)
    plan()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        got = plan()
    side.synchronize()
    assert torch.equal(got["out"], ref["out"])
    df.dflash2_check_device_status(ws)


def test_attention_in_a_graph_follows_the_lengths(at):
    """One captured step, replayed after the bound lengths, tables and rows changed in place."""
    b = Batch([500, 90], [4, 4], 32, seed=1)
    cache, k, v = filled(at, b, 2, 64, BF16, 2)
    tokens = b.on_gpu(at)
    q = randn(gen(3), b.N, 4, 64).to(BF16)
    plan = at.PagedAttentionPlan(q, cache, tokens)
    plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for lens in ([500, 90], [131, 90], [4, 61]):
        tokens.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(randn(gen(sum(lens)), b.N, 4, 64))
        graph.replay()
        want, mag, _ = attend(q, [x[:n] for x, n in zip(k, lens)], [x[:n] for x, n in zip(v, lens)], lens, b.news, 0.125,
                              True, 0)
        assert ((plan.outputs["out"].double() - want).abs() <= attend_bound(want, mag)).all()


def test_attention_repeats_its_bits(at):
    b, cache, q, ref = check(at, [5000, 300], [16, 16], 64, 16, 2, 128, E4M3, True, 0)
    for _ in range(3):
        got = at.dflash2_paged_attention(q, cache, b.on_gpu(at))
        assert torch.equal(got["out"], ref["out"]) and torch.equal(got["lse"], ref["lse"])


@TYPES
@pytest.mark.parametrize("new", [2, 40])
def test_attention_long(at, dtype, new):
    """So many key tiles for each SM that every ring wraps many times over, and no wait gives up."""
    from speculative_decoding_drafter_gb300 import dflash2 as df

    n, kvh, dim = 163000, 8, 64
    b = Batch([n], [new], 64, poison=True)
    cache, k, v = filled(at, b, kvh, dim, dtype, 5)
    q = randn(gen(6), new, 16, dim).to(BF16)
    ws = at.AttentionWorkspace(cache, b.on_gpu(at), 16)
    want, mag, lse = attend(q, k, v, b.lens, b.news, dim ** -0.5, True, 0)
    got = at.dflash2_paged_attention(q, cache, b.on_gpu(at), workspace=ws)
    df.dflash2_check_device_status(ws)
    first = {name: t.clone() for name, t in got.items()}
    for _ in range(3):  # SMs take what is left in another order each time
        again = at.dflash2_paged_attention(q, cache, b.on_gpu(at), workspace=ws)
        assert torch.equal(again["out"], first["out"]) and torch.equal(again["lse"], first["lse"])
    assert ((got["out"].double() - want).abs() <= attend_bound(want, mag)).all()
    assert ((got["lse"].double() - lse).abs() <= 2.0 ** -14 * (1 + lse.abs())).all()


@TYPES
@pytest.mark.parametrize("new", [1, 16, 40])
def test_attention_beside_memory_traffic(at, dtype, new):
    """Tiles that arrive late, one by one and at random: the products of every tile are in the result all the same."""
    lens = [8192 - 157 * ((11 * i) % 32) for i in range(32)]
    b = Batch(lens, [new] * 32, 64)
    cache, k, v = filled(at, b, 4, 128, dtype, 8)
    q = randn(gen(9), 32 * new, 16, 128).to(BF16)
    want, mag, lse = attend(q, k, v, b.lens, b.news, 128 ** -0.5, True, 0)
    batch = b.on_gpu(at)
    ws = at.AttentionWorkspace(cache, batch, 16)
    noise, side = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    runs = []
    for _ in range(100):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(4):
                noise.add_(1)
        runs.append(at.dflash2_paged_attention(q, cache, batch, workspace=ws))
        torch.cuda.current_stream().wait_stream(side)
    assert ((runs[0]["out"].double() - want).abs() <= attend_bound(want, mag)).all()
    assert ((runs[0]["lse"].double() - lse).abs() <= 2.0 ** -14 * (1 + lse.abs())).all()
    assert all(torch.equal(r["out"], runs[0]["out"]) and torch.equal(r["lse"], runs[0]["lse"]) for r in runs[1:])


def test_attention_many_sequences(at):
    """More sequences than lanes, SMs and probes of one lookup step, several of them empty."""
    lens = [(37 * i) % 211 for i in range(600)]
    check(at, lens, [min(n, 1 + i % 3) for i, n in enumerate(lens)], 16, 4, 2, 64, BF16, True, 0)


def test_offsets_past_32_bits(at):
    """A cache of more than 2^32 bytes (and 2^31 elements): the last pages are written, read and attended to."""
    ps, kvh, dim = 1024, 8, 128
    pages = 2100  # 2100 * 8 * 1024 * 128 = 2.2e9 elements, 4.4 GB each
    cache = at.PagedCache(torch.empty(pages, kvh, ps, dim, dtype=BF16, device="cuda"),
                          torch.empty(pages, kvh, ps, dim, dtype=BF16, device="cuda"))
    b = Batch([1500], [1500], ps)
    b.table[0, :2] = torch.tensor([pages - 1, pages - 2], dtype=torch.int32)
    b.pages = pages
    g = gen(4)
    k, v = randn(g, 1500, kvh, dim).to(BF16), randn(g, 1500, kvh, dim).to(BF16)
    at.dflash2_cache_append(cache, b.on_gpu(at), k, v)
    assert torch.equal(cache.k[pages - 1, :, :].transpose(0, 1), k[:1024])
    read = at.dflash2_cache_read(cache, b.on_gpu(at))
    assert torch.equal(read["k"], k) and torch.equal(read["v"], v)
    b.news, b.start, b.N = [3], torch.tensor([0, 3], dtype=torch.int32), 3
    q = randn(g, 3, 16, dim).to(BF16)
    want, mag, _ = attend(q, [k.double()], [v.double()], [1500], [3], dim ** -0.5, True, 0)
    got = at.dflash2_paged_attention(q, cache, b.on_gpu(at))
    assert ((got["out"].double() - want).abs() <= attend_bound(want, mag)).all()


def test_no_tokens(at):
    cache = at.PagedCache.allocate(2, 16, 2, 64)
    b = Batch([5], [0], 16)
    empty = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    at.dflash2_cache_append(cache, b.on_gpu(at), empty, empty)
    assert at.dflash2_cache_read(cache, b.on_gpu(at))["k"].shape == (0, 2, 64)
    assert at.dflash2_paged_attention(empty, cache, b.on_gpu(at))["out"].shape == (0, 2, 64)
    assert at.dflash2_rope(empty, torch.empty(0, dtype=torch.int32, device="cuda"), make_table(4, 8)).shape == (0, 2, 64)


# ---------------------------------------------------------------------------------------- all together


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
def test_draft_steps(at, kind):
    """The example's layer: every step's attention equals the plain form over what the cache holds."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    B, T = 3, 8
    step = example.DraftStep(B, T, cache_type=kind, max_len=64)
    ids = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    anchor = torch.tensor([5, 9, 77], dtype=torch.int32, device="cuda")
    for n in range(3):
        ids = step(ids, anchor)
        anchor = ids[:, -1].contiguous()
        held = T * (n + 1)
        whole = at.TokenBatch(torch.arange(B + 1, dtype=torch.int32, device="cuda") * held, step.kv_len,
                              step.tokens.page_table, tokens=B * held, max_new=held)
        if kind == "bf16":
            back = at.dflash2_cache_read(step.cache, whole)
            k, v = (list(back[x].double().view(B, held, step.kv_heads, step.dim)) for x in ("k", "v"))
        else:
            p = torch.arange(held, device="cuda")
            pages, slots = step.tokens.page_table[:, p // 16].long(), p % 16
            k, v = ([getattr(step.cache, x).view(torch.uint8)[pages[b], :, slots].view(example.TYPES[kind]).double() *
                     getattr(step.cache, x + "_scale")[pages[b], :, slots].double()[..., None] for b in range(B)]
                    for x in ("k", "v"))
        q = step.qkv[:, :step.q_heads]
        want, mag, _ = attend(q, k, v, [held] * B, [T] * B, step.dim ** -0.5, False, 0)
        assert ((step.out.double() - want).abs() <= attend_bound(want, mag)).all()
        assert ids.shape == (B, T) and (ids >= 0).all() and (ids < 8192).all()
