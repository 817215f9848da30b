"""How a prompt is cut between tiles and pairs of SMs (wq_prompt_plan), on the
CPU: the tiles cover every token, an accumulator fits its columns, cut tiles fit
the workspace they are given, and no pair is left without work."""
import random

import pytest

import weight_only_quantized_02_b200 as wq

COUNTERS = 262912  # bytes of the workspace before the partial sums


def check(bits, M, K, N, pairs, ws):
    p = wq.wq_prompt_plan(bits, M, K, N, pairs, ws)
    n, nsub, TT, G = p["n"], p["nsub"], p["TT"], p["G"]
    assert n % 16 == 0 and 16 <= n <= 192 and nsub in (1, 2) and (bits == 8 or nsub == 1)
    assert TT * nsub * n >= M, "every token has a tile"
    assert (TT - 1) * nsub * n < M, "no tile is empty"
    KB = -(-K // 128)
    tiles = -(-(-(-N // 128)) // 2) * TT
    units = tiles * KB
    assert units < 1 << 31
    assert 1 <= G <= min(pairs, 80)
    if p["align"]:
        assert G <= tiles
    else:
        assert COUNTERS + G * 4 * nsub * n * 128 * 4 <= ws
        starts = [units * c // G for c in range(G + 1)]
        assert all(b > a for a, b in zip(starts, starts[1:])), "every pair has units"
        # a pair's range meets at most two tiles that others share, its first and its last
        for a, b in zip(starts, starts[1:]):
            shared = [t for t in (a // KB, (b - 1) // KB) if a > t * KB or b < (t + 1) * KB]
            assert len(set(shared)) <= 2
    return p


@pytest.mark.parametrize("ws", [0, COUNTERS, 10 << 20, 64 << 20])
@pytest.mark.parametrize("pairs", [1, 3, 74, 400])
def test_random_shapes(ws, pairs):
    rng = random.Random(ws + pairs)
    for _ in range(400):
        bits = rng.choice((4, 8))
        K = 128 * int(2 ** rng.uniform(0, 8)) if bits == 4 else 32 * int(2 ** rng.uniform(0, 10))
        N = 16 * int(2 ** rng.uniform(0, 14))
        check(bits, int(2 ** rng.uniform(0, 16)), K, N, pairs, ws)


def test_no_workspace_takes_whole_tiles():
    for M in (129, 364, 2048):
        assert wq.wq_prompt_plan(8, M, 15744, 528, 74, 0)["align"]
        assert wq.wq_prompt_plan(4, M, 17408, 5120, 74, COUNTERS)["align"]


def test_few_panels_are_cut():
    p = check(8, 364, 15744, 528, 74, 64 << 20)
    assert not p["align"] and p["G"] >= 37


def test_refusals():
    with pytest.raises(wq.WQError):
        wq.wq_prompt_plan(8, 0, 128, 128)
    with pytest.raises(wq.WQError):
        wq.wq_prompt_plan(8, 65537, 128, 128)
    with pytest.raises(wq.WQError):
        wq.wq_prompt_plan(4, 200, 100, 128)
    with pytest.raises(wq.WQError):
        wq.wq_prompt_plan(4, 200, 128, 128, 0)
    assert wq.lib.wq_prompt_plan(8, 200, 128, 128, 74, 0, None) == -1
