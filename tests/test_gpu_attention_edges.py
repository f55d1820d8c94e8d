"""Attention over the paged cache where numbers, sizes or callers are at an edge, on the GPU against float64."""
import math
import threading

import pytest
import torch

from attention_rules import BF16, EPS16, EPS_F16, Batch, attend, attend_bound, tile_bound, tile_values
from test_gpu_attention import check

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
TYPES = pytest.mark.parametrize("dtype", [BF16, E4M3, INT8])
EIGHT_BITS = pytest.mark.parametrize("dtype", [E4M3, INT8])


@pytest.fixture(scope="module")
def at():
    from speculative_decoding_drafter_gb300 import attention

    return attention


def randn(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def one_sequence(at, k, v, dtype, page_size=64, copies=1, new=1):
    """A cache that holds k and v [n, heads, dim], as `copies` sequences over the same pages; its batch of `new` tokens
    each, and the rows as held, in float64."""
    n, heads, dim = k.shape
    b = Batch([n], [n], page_size, spare=0)
    cache = at.PagedCache.allocate(b.pages, page_size, heads, dim, dtype)
    at.dflash2_cache_append(cache, b.on_gpu(at), k.to(BF16), v.to(BF16))
    p = torch.arange(n, device="cuda")
    pages, slots = b.table.cuda()[0][p // page_size].long(), p % page_size
    rows = []
    for name in ("k", "v"):
        if dtype == BF16:
            rows.append(getattr(cache, name)[pages, :, slots].double())
        else:
            r = getattr(cache, name).view(torch.uint8)[pages, :, slots].view(dtype).double()
            rows.append(r * getattr(cache, name + "_scale")[pages, :, slots].double()[..., None])
    batch = at.TokenBatch(torch.arange(copies + 1, dtype=torch.int32, device="cuda") * new,
                          torch.full((copies,), n, dtype=torch.int32, device="cuda"),
                          b.table.expand(copies, -1).contiguous().cuda(), tokens=copies * new, max_new=new)
    return cache, batch, rows[0], rows[1]


def lse_close(got, want):
    """float32 scores of size up to 2^4 summed over dim terms, and a sum of positive terms."""
    return ((got.double() - want).abs() <= 2.0 ** -14 * (1 + want.abs())).all()


def unit_scale(dim):
    """The scale at which a key of c's scores c powers of two with a query of ones."""
    return 1.0 / (dim * math.log2(math.e))


# ------------------------------------------------------------------------------------------ callers


def test_calls_of_several_sizes_from_two_threads(at):
    """What a call needs of the device does not depend on what another thread called before."""
    k, v = randn(1, 100, 2, 128), randn(2, 100, 2, 128)
    failed = []

    def call(copies):
        try:
            cache, batch, _, _ = one_sequence(at, k, v, BF16, copies=copies)
            at.dflash2_paged_attention(randn(3, copies, 4, 128).to(BF16), cache, batch)
        except Exception as e:  # noqa: BLE001
            failed.append((copies, repr(e)))

    call(32)
    other = threading.Thread(target=call, args=(1,))
    other.start()
    other.join()
    call(32)
    torch.cuda.synchronize()
    assert not failed


def test_what_a_plan_binds_stays_bound(at):
    """Emptying the dict that a call returned, or taking the names off a cache, a batch and a workspace, leaves the
    next call's buffers alive and its results the same."""
    k, v = randn(1, 300, 2, 128), randn(2, 300, 2, 128)
    cache, batch, _, _ = one_sequence(at, k, v, E4M3, new=5)
    q = randn(3, 5, 4, 128).to(BF16)
    plan = at.PagedAttentionPlan(q, cache, batch)
    first = plan()
    want = {name: t.clone() for name, t in first.items()}
    first.clear()
    plan.outputs.clear()
    plan.workspace = None
    cache.k = cache.v = cache.k_scale = cache.v_scale = None
    batch.token_start = batch.kv_len = batch.page_table = None
    fill = [torch.full((1 << 16,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(64)]  # takes what was let go
    again = plan()
    assert set(again) == set(want) and all(torch.equal(again[name], want[name]) for name in want)
    assert all((f == 0xFF).all() for f in fill)


def test_counts_that_32_bits_do_not_hold(at):
    """A window past every position is no limit, not what is left of it in 32 bits; other counts are refused."""
    k, v = randn(1, 300, 2, 64), randn(2, 300, 2, 64)
    cache, batch, _, _ = one_sequence(at, k, v, BF16, new=5)
    q = randn(3, 5, 4, 64).to(BF16)
    want = at.dflash2_paged_attention(q, cache, batch)
    for window in (2 ** 31 - 1, 2 ** 32 + 1, 10 ** 12):
        got = at.dflash2_paged_attention(q, cache, batch, window=window)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    for kw in (dict(tokens=5, max_new=2 ** 32 + 1), dict(tokens=2 ** 32 + 5)):
        with pytest.raises(ValueError, match="must fit 32 bits"):
            at.TokenBatch(batch.token_start, batch.kv_len, batch.page_table, **kw)


@pytest.mark.parametrize("new", [0, 1, 3])
def test_a_batch_shorter_than_its_block_length(at, new):
    """max_new bound once to a loop's block length, and a last batch with fewer tokens in all."""
    k, v = randn(1, 300, 2, 64), randn(2, 300, 2, 64)
    cache, batch, kk, vv = one_sequence(at, k, v, E4M3, new=new)
    short = at.TokenBatch(batch.token_start, batch.kv_len, batch.page_table, tokens=new, max_new=16)
    q = randn(3, new, 4, 64).to(BF16)
    got = at.dflash2_paged_attention(q, cache, short)
    want, mag, lse = attend(q, [kk], [vv], [300], [new], 64 ** -0.5, True, 0)
    assert ((got["out"].double() - want).abs() <= attend_bound(want, mag)).all() and lse_close(got["lse"], lse)
    read, both = at.dflash2_cache_read(cache, short), at.dflash2_cache_read(cache, batch)
    assert torch.equal(read["k"], both["k"]) and torch.equal(read["v"], both["v"])
    at.dflash2_cache_append(cache, short, both["k"], both["v"])


@TYPES
@pytest.mark.parametrize("new", [5, 70])
def test_a_sequence_with_more_tokens_than_said(at, dtype, new):
    """Every row is there, also where its item is worked on by several SMs."""
    k, v = randn(1, 5000, 2, 64), randn(2, 5000, 2, 64)
    cache, batch, kk, vv = one_sequence(at, k, v, dtype, copies=3, new=new)
    wrong = at.TokenBatch(batch.token_start, batch.kv_len, batch.page_table, tokens=3 * new, max_new=1)
    q = randn(3, new, 4, 64).to(BF16).repeat(3, 1, 1)
    out, lse_out = torch.full_like(q, math.nan), torch.full((3 * new, 4), math.nan, device="cuda")
    got = at.dflash2_paged_attention(q, cache, wrong, out=out, lse=lse_out)
    want, mag, lse = attend(q[:new], [kk], [vv], [5000], [new], 64 ** -0.5, True, 0)
    assert ((got["out"].double() - want.repeat(3, 1, 1)).abs() <= attend_bound(want, mag).repeat(3, 1, 1)).all()
    assert lse_close(got["lse"], lse.repeat(3, 1))


# ------------------------------------------------------------------------------------------ numbers


@EIGHT_BITS
@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("size", [2.0 ** -90, 1.0, 2.0 ** 110])
def test_sum_over_many_rows_of_zeros(at, dtype, new, size):
    """Thousands of value rows of zeros before the first that is not, their scores just under what moves the running
    maximum: the sum of the exponentials leaves float32's range if it is held in units of an unknown scale."""
    dim, heads, copies = 64, 8, 19  # an item for each of 152 SMs, so that each is one run of tiles
    c = torch.cat([torch.zeros(128), torch.full((33000 + 300,), 7.875)]).cuda()
    k = c[:, None, None].expand(-1, heads, dim)
    v = randn(5, len(c), heads, dim) * size
    v[:128 + 33000] = 0
    cache, batch, kk, vv = one_sequence(at, k, v, dtype, copies=copies, new=new)
    q = torch.ones(copies * new, heads, dim, dtype=BF16, device="cuda")
    got = at.dflash2_paged_attention(q, cache, batch, scale=unit_scale(dim))
    want, mag, lse = attend(q[:new], [kk], [vv], [len(c)], [new], unit_scale(dim), True, 0)
    assert ((got["out"].double() - want.repeat(copies, 1, 1)).abs() <= attend_bound(want, mag).repeat(copies, 1, 1)).all()
    assert lse_close(got["lse"], lse.repeat(copies, 1))


@EIGHT_BITS
@pytest.mark.parametrize("apart", [24.0, 26.0, 28.5])
@pytest.mark.parametrize("new", [1, 40])
def test_many_small_probabilities_beside_a_large_one(at, dtype, apart, new):
    """Keys 2^-24 and less below one dominant key still add up."""
    dim, n, copies = 64, 3000, 76  # an item for each of 152 SMs, so that each is one run of tiles
    k = torch.zeros(n, 2, dim, device="cuda")
    k[0] = apart
    v = torch.zeros(n, 2, dim, device="cuda")
    v[0, :, 0] = 1
    v[1:, :, 1:] = 1
    cache, batch, kk, vv = one_sequence(at, k, v, dtype, copies=copies, new=new)
    q = torch.ones(copies * new, 8, dim, dtype=BF16, device="cuda")
    got = at.dflash2_paged_attention(q, cache, batch, causal=False, scale=unit_scale(dim))
    want, mag, lse = attend(q[:new], [kk], [vv], [n], [new], unit_scale(dim), False, 0)
    # beside its relative rounding each probability has f16's absolute one, half of 2^-24 where the largest is 2^7
    bound = EPS16 * want.abs() + (EPS_F16 + 2.0 ** -13) * mag + n * 2.0 ** -32
    assert ((got["out"].double() - want.repeat(copies, 1, 1)).abs() <= bound.repeat(copies, 1, 1)).all()
    assert lse_close(got["lse"], lse.repeat(copies, 1))


@TYPES
@pytest.mark.parametrize("new", [2, 20, 100])
@pytest.mark.parametrize("copies", [1, 80])  # items in pieces, and whole ones
def test_lse_where_a_value_is_not_finite(at, dtype, new, copies):
    """lse is a function of queries and keys: a value row that is not finite reaches out and not lse."""
    dim, n = 64, 700
    k, v = randn(1, n, 2, dim), randn(2, n, 2, dim)
    at_value = n - 1 - new // 2
    v[at_value, 0, 3] = math.inf
    cache, batch, kk, _ = one_sequence(at, k, v, dtype, copies=copies, new=new)
    q = randn(3, new, 8, dim).to(BF16).repeat(copies, 1, 1)
    got = at.dflash2_paged_attention(q, cache, batch)
    clean = torch.zeros_like(kk)
    _, _, lse = attend(q[:new], [kk], [clean], [n], [new], dim ** -0.5, True, 0)
    assert lse_close(got["lse"], lse.repeat(copies, 1))
    sees = (n - new + torch.arange(new, device="cuda") >= at_value).repeat(copies)
    assert not torch.isfinite(got["out"][sees][:, :4]).all(-1).any()
    assert torch.isfinite(got["out"][:, 4:]).all()  # another cache head's rows


@TYPES
@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
@pytest.mark.parametrize("new", [3, 100])
def test_values_of_very_different_size_side_by_side(at, dtype, order, new):
    """Value rows 2^100 apart, and rows of zeros: each key counts in the sum of the exponentials whatever its value."""
    dim, n = 64, 2500
    power = torch.linspace(-50, 50, n, device="cuda").round()
    power = {"mixed": power[torch.randperm(n, generator=torch.Generator().manual_seed(1)).cuda()], "rising": power,
             "falling": power.flip(0)}[order]
    k = randn(1, n, 2, dim)
    v = randn(2, n, 2, dim) * torch.exp2(power)[:, None, None]
    v[::7] = 0
    cache, batch, kk, vv = one_sequence(at, k, v, dtype, copies=76, new=new)
    q = randn(3, new, 8, dim).to(BF16)
    got = at.dflash2_paged_attention(q.repeat(76, 1, 1), cache, batch)
    want, mag, lse = attend(q, [kk], [vv], [n], [new], dim ** -0.5, True, 0)
    assert ((got["out"].double() - want.repeat(76, 1, 1)).abs() <= attend_bound(want, mag).repeat(76, 1, 1)).all()
    assert lse_close(got["lse"], lse.repeat(76, 1))


# ------------------------------------------------------------------------------------------ every tile


@TYPES
@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("lens,new", [([163000], 2), ([163000], 40), ([9000 - 211 * i for i in range(40)], 1),
                                      ([9000 - 211 * i for i in range(40)], 40), ([50000, 20, 7], 100)])
def test_every_tile_is_in_the_result(at, dtype, spread, lens, new):
    """Channels that count tiles: one tile's products lost, or taken twice, is an error of 1 / 20 and more."""
    heads, dim, n = 2, 64, max(lens)
    k = randn(1, n, heads, dim)
    cache, batch, kk, vv = one_sequence(at, k, tile_values(n, heads, dim), dtype, copies=len(lens), new=new)
    batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    q = (spread * randn(2, len(lens) * new, 4, dim)).to(BF16)
    got = at.dflash2_paged_attention(q, cache, batch, causal=False)
    group = 4 // heads
    for b, length in enumerate(lens):
        rows = slice(b * new, (b + 1) * new)  # positions below zero are padding, which sees the keys there are
        want, _, lse = attend(q[rows], [kk[:length]], [vv[:length]], [length], [new], dim ** -0.5, False, 0)
        s = torch.einsum("thd,jhd->thj", q[rows].double(), kk[:length].repeat_interleave(group, 1)) * dim ** -0.5
        p = torch.exp(s - lse[..., None])
        squares = torch.einsum("thj,jhd->thd", p * p, vv[:length].repeat_interleave(group, 1))
        bound = tile_bound(want, squares, EPS16 if dtype == BF16 else EPS_F16)
        assert ((got["out"][rows].double() - want).abs() <= bound).all()
        assert lse_close(got["lse"][rows], lse)


@TYPES
@pytest.mark.parametrize("most,dim", [(3, 64), (3, 128), (45, 64), (45, 128)])
def test_as_many_sequences_as_there_may_be(at, dtype, most, dim):
    """2048 sequences, many of them empty or without new tokens, in one row tile and in two."""
    lens = [(37 * i) % 211 for i in range(2048)]
    lens[-40:] = [0] * 40
    news = [min(n, i % 4) for i, n in enumerate(lens)]
    for i in range(3, 2000, 250):
        news[i] = min(lens[i], most)
    check(at, lens, news, 16, 4, 1, dim, dtype, True, 0, seed=dim + most)


# ------------------------------------------------------------------------------------------ waits

def test_a_row_tile_that_stays_idle_for_long(at):
    """Items of one row tile among those of two, over 2^30 positions (of one page, over and over): the warps of the
    second row tile then have nothing to do for longer than a wait inside a pipeline may take."""
    from speculative_decoding_drafter_gb300 import dflash2 as df

    ps, heads, dim, new, copies = 1024, 1, 16, 65, 24
    cache = at.PagedCache.allocate(1, ps, heads, dim, BF16)
    batch = at.TokenBatch(torch.arange(copies + 1, dtype=torch.int32, device="cuda") * new,
                          torch.full((copies,), 1 << 30, dtype=torch.int32, device="cuda"),
                          torch.zeros(copies, (1 << 30) // ps, dtype=torch.int32, device="cuda"),
                          tokens=copies * new, max_new=new)
    q = randn(1, copies * new, 4, dim).to(BF16)
    ws = at.AttentionWorkspace(cache, batch, 4)
    got = at.dflash2_paged_attention(q, cache, batch, causal=False, workspace=ws)
    df.dflash2_check_device_status(ws)
    assert ((got["lse"].double() - 30 * math.log(2)).abs() <= 2.0 ** -10 * 30).all()
