"""How the LM-head loss's products are cut into tiles and dealt out to the pairs of CTAs: the code that the kernels run, compiled
for the host and followed (no GPU needed)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_drafter_gb300", "csrc")
TILE, STAGE = 256, 128
HIDDEN, WEIGHTS = 1, 2


@pytest.fixture(scope="module")
def work(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("work") / "head_work")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, os.path.join(ROOT, "tests", "c", "head_work.cpp"), "-o", exe], check=True)

    def run(N, H, V, pairs=76, kept=None, hidden=1, weights=1):
        args = [N, H, V, pairs, N if kept is None else kept, hidden, weights]
        res = subprocess.run([exe, *map(str, args)], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr
        loss, pieces, plan = [], [], None
        for line in res.stdout.splitlines():
            kind, *x = line.split()
            x = tuple(map(int, x))
            if kind == "loss":
                loss.append(x)
            elif kind == "plan":
                plan = dict(zip(("piece", "splits", "pitch", "parts"), x))
            elif kind == "piece":
                pieces.append(dict(zip(("v0", "width", "row_tiles", "splits", "hidden_tiles", "weight_tiles"), x), score=[], grad=[]))
            else:
                pieces[-1][kind].append(x)
        return loss, plan, pieces

    return run


def tiles(n):
    return -(-n // TILE)


# rows around a tile, one piece and several, heads of one tile to many, more pairs than tiles and fewer
SIZES = [(1, 8, 1), (8, 256, 4096), (128, 72, 300), (129, 136, 1000), (257, 64, 513), (64, 5120, 30000), (2048, 1024, 20000),
         (1000, 520, 3001), (16, 4096, 32000), (1 << 20, 264, 1000), (40000, 64, 20001), (300, 16384, 4000)]


@pytest.mark.parametrize("N,H,V", SIZES)
@pytest.mark.parametrize("pairs", [1, 7, 76])
def test_every_tile_is_dealt_out_once(work, N, H, V, pairs):
    for kept in sorted({N, 0, min(N, 3), N - N // 8}):
        for hidden, weights in ((1, 1), (1, 0), (0, 1)):
            loss, plan, pieces = work(N, H, V, pairs, kept, hidden, weights)
            stages = -(-H // STAGE)
            want = sorted((m * TILE, n * TILE, stages) for m in range(tiles(N)) for n in range(tiles(V)))
            assert sorted((m0, n0, s) for _, _, m0, n0, _, s, _ in loss) == want
            rows, parts = max(1, tiles(kept)), plan["parts"]
            assert parts == (2 if N <= 128 else 1) and N * parts * plan["piece"] <= max(1 << 28, N * parts * TILE)
            assert plan["pitch"] % 64 == 0 and 0 <= plan["pitch"] - H < 64
            at = 0
            for p in pieces:
                assert p["v0"] == at and p["width"] % TILE == 0
                at += p["width"]
                want = sorted((m * TILE, n * TILE, stages) for m in range(rows) for n in range(p["width"] // TILE))
                assert sorted((m0, n0, s) for _, _, m0, n0, _, s, _ in p["score"]) == want
                ks = p["width"] // STAGE
                ranges = {}
                for _, product, m0, n0, k0, s, split in p["grad"]:
                    if product == HIDDEN:
                        assert s >= 1 and 0 <= split < p["splits"]
                        ranges.setdefault((m0, n0), []).append((split, k0, s))
                assert len(ranges) == (rows * tiles(H) if hidden else 0)
                for r in ranges.values():  # the parts of a tile follow one another over the whole piece
                    end = 0
                    for n, (split, k0, s) in enumerate(sorted(r)):
                        assert split == n and k0 == end
                        end += s
                    assert end == ks and len(r) == p["splits"]
                want = sorted((m * TILE, n * TILE, max(1, -(-kept * parts // STAGE)))
                              for m in range(p["width"] // TILE) for n in range(tiles(H))) if weights else []
                assert sorted((m0, n0, s) for _, product, m0, n0, _, s, _ in p["grad"] if product == WEIGHTS) == want
            assert at >= V > at - TILE - (0 if len(pieces) == 1 else TILE * len(pieces))
            assert all(p["splits"] <= plan["splits"] for p in pieces) and pieces[0]["splits"] == plan["splits"]


@pytest.mark.parametrize("N,H,V", [(64, 5120, 152064), (2048, 4096, 151936), (254, 2032, 18994)])
def test_the_shares_end_together(work, N, H, V):
    """In half stages, a tile's ends being one: the turns of d_W's that stand for a tile of d_hidden are rounded down, less than
    one tile of d_W's short, and the last round of those ends one apart.  With parts of d_hidden as long as one another (they
    are in these cases) no pair is further than two tiles of d_W's from the mean."""
    _, plan, pieces = work(N, H, V)
    for p in pieces:
        assert len({s for _, product, _, _, _, s, _ in p["grad"] if product == HIDDEN}) == 1
        time, one = [0] * 76, 2 * max(s for _, product, _, _, _, s, _ in p["grad"] if product == WEIGHTS) + 1
        for pair, _, _, _, _, s, _ in p["grad"]:
            time[pair] += 2 * s + 1
        assert max(time) - 2 * one <= sum(time) / len(time) <= min(time) + 2 * one, (plan, min(time), max(time))


def test_the_plan_of_few_rows(work):
    """64 rows of hidden size 5120: 20 tiles of d_hidden in 6 parts of 198 stages, on 76 pairs."""
    _, plan, (p,) = work(64, 5120, 152064)
    assert plan["splits"] == 6 and p["hidden_tiles"] == 120
    assert {s for _, product, _, _, _, s, _ in p["grad"] if product == HIDDEN} == {198}
    assert {s for _, product, _, _, _, s, _ in p["grad"] if product == WEIGHTS} == {1}
