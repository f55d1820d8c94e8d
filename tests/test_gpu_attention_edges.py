"""Attention over the paged cache where numbers, sizes or callers are at an edge, on the GPU against float64."""
import math

import pytest
import torch

from attention_rules import BF16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def at():
    from speculative_decoding_drafter_gb300 import attention

    return attention


def randn(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


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
