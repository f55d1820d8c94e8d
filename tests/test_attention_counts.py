"""The binding of the attention-side operators refuses counts that the C ABI's 32 bits do not hold (no GPU needed)."""
from types import SimpleNamespace

import pytest

from speculative_decoding_drafter_gb300 import build as build_mod


@pytest.fixture(scope="module")
def at():
    build_mod.build()
    from speculative_decoding_drafter_gb300 import attention

    return attention


@pytest.mark.parametrize("max_pos,rot", [(2 ** 32 + 8, 8), (16, 2 ** 32 + 8), (-2 ** 32 + 8, 8)])
def test_rope_table(at, max_pos, rot):
    with pytest.raises(ValueError, match="must fit 32 bits"):
        at.dflash2_rope_table(max_pos, rot)


def test_workspace_bytes(at):
    from speculative_decoding_drafter_gb300 import dflash2 as df

    cache = SimpleNamespace(args=df.CacheArgs(4, 16, 2, 64, 0, None, None, None, None))
    batch = SimpleNamespace(args=df.TokenArgs(2, 5, 3, 4, None, None, None))
    assert at.dflash2_paged_attention_workspace_bytes(cache, batch, 4) > 0
    with pytest.raises(ValueError, match="must fit 32 bits"):
        at.dflash2_paged_attention_workspace_bytes(cache, batch, 2 ** 32 + 4)
