"""The bounds that attention is held to see what they are there for: mistakes planted in the plain form (no GPU needed)."""
import pytest
import torch

from attention_rules import EPS16, EPS_F16, attend, tile_bound, tile_values


@pytest.mark.parametrize("eps", [EPS16, EPS_F16])
@pytest.mark.parametrize("n,spread", [(163000, 0.0), (163000, 1.0), (9000, 1.0)])
def test_a_lost_or_repeated_tile_is_seen(n, spread, eps):
    g = torch.Generator().manual_seed(n)
    q, k = spread * torch.randn(2, 1, 64, generator=g).double(), torch.randn(n, 1, 64, generator=g).double()
    v = tile_values(n, 1, 64, device="cpu").double()
    want, _, lse = attend(q, [k], [v], [n], [2], 0.125, False, 0)
    p = torch.exp(torch.einsum("thd,jhd->thj", q, k) * 0.125 - lse[..., None])
    bound = tile_bound(want, torch.einsum("thj,jhd->thd", p * p, v), eps)
    for tile in (0, 5, n // 128 // 2, n // 128 - 1):
        for times in (0, 2):
            other = v.clone()
            other[tile * 128:(tile + 1) * 128] *= times
            got, _, _ = attend(q, [k], [other], [n], [2], 0.125, False, 0)
            assert ((got - want).abs() > bound).any(-1).all()
