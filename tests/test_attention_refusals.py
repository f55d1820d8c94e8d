"""The attention-side entry points refuse bad arguments on the host, before any CUDA call (no GPU needed; the
pointer values below are never dereferenced), and the binding refuses host tensors."""
import ctypes
import re

import pytest
import torch

from speculative_decoding_drafter_gb300 import build as build_mod

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BASE = 0x200000


@pytest.fixture(scope="module")
def df():
    build_mod.build()
    from speculative_decoding_drafter_gb300 import dflash2

    dflash2.library()
    return dflash2


def ref(x):
    return None if x is None else ctypes.byref(x)


def cache(df, pages=4, page_size=16, heads=2, dim=64, type=0, k=BASE, v=BASE, ks=BASE, vs=BASE):
    return df.CacheArgs(pages, page_size, heads, dim, type, k, v, ks, vs)


def tokens(df, B=2, N=5, max_new=3, max_pages=4, start=BASE, kv_len=BASE, table=BASE):
    return df.TokenArgs(B, N, max_new, max_pages, start, kv_len, table)


def rows(df, heads=2, ts=128, hs=64, data=BASE):
    return df.HeadRows(data, heads, ts, hs)


def rope(df, table=BASE, max_pos=100, rot=64, inter=0):
    return df.RopeArgs(table, max_pos, rot, inter)


BAD_CACHES = [(dict(pages=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=12), UNSUPPORTED),
              (dict(page_size=2048), UNSUPPORTED), (dict(dim=72), UNSUPPORTED), (dict(dim=256), UNSUPPORTED),
              (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(k=None), INVALID), (dict(v=BASE + 8), INVALID),
              (dict(type=1, ks=None), INVALID), (dict(type=2, vs=BASE + 4), INVALID), (dict(heads=2000), UNSUPPORTED)]
BAD_TOKENS = [(dict(B=0), INVALID), (dict(B=2049), UNSUPPORTED), (dict(N=-1), INVALID), (dict(max_new=0), INVALID),
              (dict(max_new=6), INVALID), (dict(start=None), INVALID), (dict(kv_len=BASE + 2), INVALID),
              (dict(table=None), INVALID), (dict(max_pages=1 << 28), UNSUPPORTED)]


def append(df, c=None, t=None, r=None, q="same", qo="same", k=None, v=None):
    h = rows(df)
    return df.library().dflash2_cache_append(
        ref(c or cache(df)), ref(t or tokens(df)), ref(r), ref(None if q is None else h if q == "same" else q),
        ref(None if qo is None else h if qo == "same" else qo), ref(k or h), ref(v or h), None)


def attend(df, c=None, t=None, scale=0.1, window=0, q=None, out=None, lse=None, ws=0x100000, n=1 << 40, opts=True):
    o = df.AttentionArgs(scale, 1, window)
    return df.library().dflash2_paged_attention(ref(c or cache(df)), ref(t or tokens(df)), ref(o if opts else None),
                                                ref(q or rows(df)), ref(out or rows(df)), lse, ws, n, None)


def read(df, c=None, t=None, k="rows", v="rows"):
    h = rows(df)
    return df.library().dflash2_cache_read(ref(c or cache(df)), ref(t or tokens(df)), ref(h if k == "rows" else k),
                                           ref(h if v == "rows" else v), None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches(df, bad, status):
    for call in (append, attend, read):
        assert call(df, c=cache(df, **bad)) == status


@pytest.mark.parametrize("bad,status", BAD_TOKENS)
def test_bad_tokens(df, bad, status):
    for call in (append, attend, read):
        assert call(df, t=tokens(df, **bad)) == status


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=BASE + 8), dict(heads=3), dict(ts=-128), dict(ts=132),
                                 dict(hs=4)])
def test_bad_rows(df, bad):
    h = rows(df, **bad)
    assert append(df, k=h) == INVALID and append(df, v=h) == INVALID
    assert read(df, k=h) == INVALID and read(df, v=h) == INVALID
    if "heads" not in bad:
        assert append(df, q=h) == INVALID and append(df, qo=h) == INVALID
        assert attend(df, q=h) == INVALID and attend(df, out=h) == INVALID


def test_outputs_that_overlap_themselves(df):
    for h in (rows(df, ts=64, hs=64), rows(df, ts=0, hs=64), rows(df, ts=128, hs=0), rows(df, ts=120, hs=64)):
        assert attend(df, out=h) == INVALID
        assert read(df, k=h) == INVALID
        assert append(df, qo=h) == INVALID
    # in place the two sides have the same strides
    assert append(df, q=rows(df), qo=rows(df, ts=256)) == INVALID


def test_append_rope_and_queries(df):
    for r in (rope(df, table=None), rope(df, table=BASE + 2), rope(df, max_pos=0), rope(df, rot=0), rope(df, rot=63),
              rope(df, rot=66)):
        assert append(df, r=r) == INVALID
    assert append(df, q=None) == INVALID and append(df, qo=None) == INVALID
    assert read(df, k=None, v=None) == INVALID
    lib = df.library()
    assert lib.dflash2_cache_append(None, ref(tokens(df)), None, None, None, ref(rows(df)), ref(rows(df)), None) == INVALID
    assert lib.dflash2_cache_append(ref(cache(df)), None, None, None, None, ref(rows(df)), ref(rows(df)), None) == INVALID
    assert lib.dflash2_cache_append(ref(cache(df)), ref(tokens(df)), None, None, None, None, ref(rows(df)), None) == INVALID


def test_attention_options_and_workspace(df):
    assert attend(df, scale=float("nan")) == INVALID and attend(df, scale=float("inf")) == INVALID
    assert attend(df, window=-1) == INVALID and attend(df, opts=False) == INVALID
    assert attend(df, lse=BASE + 2) == INVALID
    assert attend(df, q=rows(df, heads=3, ts=192)) == INVALID           # not a multiple of the cache's heads
    many = rows(df, heads=130, ts=130 * 64)
    assert attend(df, q=many, out=many) == UNSUPPORTED                   # 65 query heads a cache head
    assert attend(df, ws=None) == WORKSPACE and attend(df, ws=0x100010) == WORKSPACE and attend(df, n=4096) == WORKSPACE
    need = df.library().dflash2_paged_attention_workspace_bytes
    n = need(ref(cache(df)), ref(tokens(df)), 2)
    assert n > 256 and n % 256 == 0
    assert attend(df, n=n - 1) == WORKSPACE
    assert need(ref(cache(df, dim=72)), ref(tokens(df)), 2) == 0
    assert need(ref(cache(df)), ref(tokens(df, B=0)), 2) == 0
    assert need(ref(cache(df)), ref(tokens(df)), 3) == 0
    assert need(None, ref(tokens(df)), 2) == 0 and need(ref(cache(df)), None, 2) == 0


def test_no_tokens_is_no_work(df):
    t = tokens(df, N=0, max_new=0)
    assert append(df, t=t) == OK and attend(df, t=t) == OK and read(df, t=t) == OK


def test_rope_refusals(df):
    lib = df.library()

    def call(r=None, N=4, dim=64, x=None, pos=BASE, y=None):
        return lib.dflash2_rope(ref(r or rope(df)), N, dim, ref(x or rows(df)), pos, 0, ref(y or rows(df)), None)

    assert call(N=-1) == INVALID and call(dim=0) == INVALID and call(pos=None) == INVALID and call(pos=BASE + 1) == INVALID
    assert call(dim=60) == UNSUPPORTED and call(dim=264) == UNSUPPORTED
    assert call(r=rope(df, rot=66)) == INVALID and call(r=rope(df, rot=7)) == INVALID and call(r=rope(df, table=None)) == INVALID
    assert call(x=rows(df, data=BASE + 4)) == INVALID and call(y=rows(df, heads=1)) == INVALID
    assert call(y=rows(df, ts=256)) == INVALID  # in place with other strides
    assert call(y=rows(df, data=BASE + 4096, ts=64)) == INVALID  # tokens overlap
    assert call(N=1 << 30, x=rows(df, heads=4, ts=256), y=rows(df, heads=4, ts=256)) == UNSUPPORTED
    assert lib.dflash2_rope(None, 4, 64, ref(rows(df)), BASE, 0, ref(rows(df)), None) == INVALID
    assert call(N=0, pos=None) == OK


def test_rope_table_refusals(df):
    def call(max_pos=16, rot=8, table=BASE, **kw):
        s = df.RopeScaling(**{**dict(kind=0, theta=1e4, factor=1.0, original_len=64.0, low=1.0, high=4.0, multiplier=1.0), **kw})
        return df.library().dflash2_rope_table(ctypes.byref(s), max_pos, rot, table, None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(max_pos=0), dict(rot=7), dict(rot=0), dict(table=None), dict(table=BASE + 2), dict(kind=5), dict(kind=-1),
                dict(theta=1.0), dict(theta=nan), dict(theta=inf), dict(multiplier=0.0), dict(multiplier=nan),
                dict(kind=1, factor=0.0), dict(kind=1, factor=inf), dict(kind=2, rot=2), dict(kind=3, original_len=0.0),
                dict(kind=3, low=0.0), dict(kind=4, low=4.0), dict(kind=4, high=inf), dict(kind=4, original_len=nan)):
        assert call(**bad) == INVALID, bad
    assert call(rot=258) == UNSUPPORTED
    assert df.library().dflash2_rope_table(None, 16, 8, BASE, None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes(df):
    from speculative_decoding_drafter_gb300 import attention as at

    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        at.dflash2_rope(x, torch.zeros(4, dtype=torch.int32), torch.zeros(8, 2, 32))
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        at.PagedCache(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        at.TokenBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                      torch.zeros(1, 4, dtype=torch.int32), tokens=1)
    with pytest.raises(ValueError, match="kind must be one of"):
        at.dflash2_rope_table(16, 8, kind="other")


def test_every_new_entry_point_is_listed(df):
    names = {n for n in df.EXPORTED_SYMBOLS if re.search("rope|cache|attention", n)}
    assert names == {"dflash2_rope_table", "dflash2_rope", "dflash2_cache_append", "dflash2_cache_read",
                     "dflash2_paged_attention_workspace_bytes", "dflash2_paged_attention"}
