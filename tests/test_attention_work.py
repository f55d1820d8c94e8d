"""How the attention kernel's work is cut up among the CTAs, followed on the host (no GPU needed)."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_drafter_gb300", "csrc")
TILE = 128


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("work") / "attention_work")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, os.path.join(ROOT, "tests", "c", "attention_work.cpp"), "-o", exe], check=True)

    def run(mode, shape, grid, sequences):
        args = [mode, *shape, grid, *(x for s in sequences for x in s)]
        res = subprocess.run([exe, *map(str, args)], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr
        return [tuple(map(int, line.split())) for line in res.stdout.splitlines()]

    return run


def items(shape, n, length):
    """(first token, first key tile, key tiles) of a sequence's items, for all of them at once."""
    causal, window, span, _, _ = shape
    tok0 = np.arange(0, n, span, dtype=np.int64)
    p0 = length - n + tok0
    hi = np.minimum(length, p0 + np.minimum(n - tok0, span)) if causal else np.full_like(p0, length)
    lo = np.maximum(0, p0 - window + 1) if window else np.zeros_like(p0)
    empty = hi <= lo
    first = np.where(empty, 0, lo // TILE)
    return tok0, first, np.where(empty, 1, (hi - 1) // TILE - first + 1)


CASES = [
    ((1, 0, 64, 4, 2), 152, [(200, 700), (0, 5), (64, 64), (1, 3000)]),
    ((0, 0, 32, 1, 8), 152, [(16, 1000 - 31 * i) for i in range(20)]),
    ((1, 100, 16, 1, 3), 7, [(0, 0), (0, 9), (33, 20), (1, 1), (0, 0), (70, 900), (0, 3)]),
    ((1, 0, 8, 1, 1), 152, [(1, 777)]),
    ((1, 1, 4, 4, 5), 152, [(9, 5), (40, 4000)]),
    ((0, 2000, 64, 4, 1), 3, [(130, 5000)]),
    ((1, 0, 16, 1, 2), 152, [((37 * i) % 5, (37 * i) % 211) for i in range(600)]),
]


@pytest.mark.parametrize("shape,grid,sequences", CASES)
def test_every_tile_is_walked_once_and_pieces_meet(walk, shape, grid, sequences):
    heads = shape[4]
    starts = np.concatenate([[0], np.cumsum([n for n, _ in sequences])])
    want = [(b, h, int(starts[b]), int(t0), int(first), int(tiles))
            for b, (n, length) in enumerate(sequences) for h in range(heads)
            for t0, first, tiles in zip(*items(shape, n, length))]
    got, pieces = [], {}
    for cta, b, h, start, tok0, tile, tiles, first, last, slot, end in walk("walk", shape, grid, sequences):
        if first:
            got.append([b, h, start, tok0, tile, tiles])
            begun = (cta, slot, end)
            assert slot in (2 * cta, 2 * cta + 1)
        else:  # the next CTA goes on where the one before stopped, in its first slot
            assert got[-1][:4] == [b, h, start, tok0] and got[-1][4] + got[-1][5] == tile
            assert slot == 2 * cta and cta == at + 1
            got[-1][5] += tiles
        at = cta
        if not (first and last):
            assert pieces.setdefault(slot, (b, h, tok0)) == (b, h, tok0)
        if last and not first:
            assert begun[2] == cta
    assert [tuple(x) for x in got] == want


@pytest.mark.parametrize("shape,sequences", [
    # causal prompts with 64 query heads on a cache head: 4 tokens an item
    ((1, 0, 4, 4, 1), [(1_500_000, 1_500_000)]),               # 2.2e9 units: past a signed 32-bit sum
    ((1, 0, 4, 4, 1), [(3, 70), (2_200_000, 2_200_000), (5, 5)]),  # 4.7e9 in one sequence
    # 8 cache heads of 8 query heads, a million tokens over four million keys: 7e9 over the heads
    ((1, 0, 32, 4, 8), [(1_000_000, 4_000_000)]),
    ((0, 0, 32, 4, 8), [(1_000_000, 4_000_000), (1, 9)]),
])
def test_counts_past_32_bits(walk, shape, sequences):
    grid, heads = 152, shape[4]
    units = [(items(shape, n, length)[2] + shape[3]) for n, length in sequences]
    total = heads * sum(int(x.sum()) for x in units)
    assert total > 2 ** 31
    ends = [np.concatenate([[0], np.cumsum(x)]) for x in units]
    before = 0
    got = walk("begin", shape, grid, sequences)
    assert len(got) == grid
    for c, (u, u_end, b, kvh, qt, off) in enumerate(got):
        assert (u, u_end) == (total * c // grid, total * (c + 1) // grid)
        before = heads * sum(int(e[-1]) for e in ends[:b])
        assert 0 <= kvh < heads and 0 <= off < units[b][qt]
        assert before + kvh * int(ends[b][-1]) + int(ends[b][qt]) + off == u
