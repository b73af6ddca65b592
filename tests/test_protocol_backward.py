"""The backward kernels' barrier protocol, checked on the CPU (protocol_backward.py)."""
import random

import pytest

import protocol_backward as M

LISTS = [(1,), (2,), (1, 1, 1, 1, 1), (3, 1, 0, 2), (0, 0, 0), (0, 5, 0, 0, 1, 0), (7, 2, 1, 1, 6), (4, 4, 4), (1, 2, 3, 4, 5), (9,)]
KV = [M.Params("dkv", t, (), *r) for t in LISTS for r in ((3, 2), (2, 2), (5, 4))]               # D = 128, with a mask, D = 64
Q = [M.Params("dq", t, (), *r) for t in LISTS for r in ((3, 2), (5, 4))]
TWICE = [M.Params("dq", t, w, *r) for t in LISTS for w in (tuple(range(len(t))), (0,), (1, 3)) for r in ((3, 1), (5, 4))]
SEEDS = range(6)


def _id(p):
    return f"{p.kernel}-{'_'.join(map(str, p.tiles))}-t{''.join(map(str, p.twice))}-r{p.k_ring}{p.v_ring}"


@pytest.mark.parametrize("p", KV + Q + TWICE, ids=_id)
def test_no_deadlock_and_no_race(p):
    for seed in SEEDS:
        M.run(p, seed, bias=(seed % 3) / 2)


@pytest.mark.parametrize("kernel", ["dkv", "dq"])
@pytest.mark.parametrize("seed", range(40))
def test_any_list_of_tiles(kernel, seed):
    rng = random.Random(seed)
    tiles = tuple(rng.choice([0, 1, 1, 2, 3, 8]) for _ in range(rng.randint(1, 9)))
    twice = tuple(t for t in range(len(tiles)) if rng.random() < 0.4) if kernel == "dq" and seed % 2 else ()
    rings = rng.choice([(3, 1), (5, 4)] if twice else [(3, 2), (5, 4)])
    M.run(M.Params(kernel, tiles, twice, *rings), seed, bias=rng.random())


@pytest.mark.parametrize("p", [KV[9], KV[20], Q[7], TWICE[18], TWICE[38]], ids=_id)
def test_a_wait_that_runs_out_ends_every_role(p):
    stalled = M.Params(**{**p.__dict__, "stall": True})
    for seed in SEEDS:
        assert M.run(stalled, seed, timeouts=True).timed_out
    for seed in range(30):
        M.run(p, seed, timeouts=True, bias=(seed % 3) / 2, abort_at=random.Random(seed).randint(1, 400))


LONG = (3, 1, 2, 1, 4, 1)


@pytest.mark.parametrize("p", [
    M.Params("dkv", LONG, (), 3, 2, mistake="accumulators_not_awaited"),
    M.Params("dkv", LONG, (), 3, 2, mistake="ds_not_awaited"),
    M.Params("dkv", LONG, (), 3, 2, mistake="v_not_awaited"),
    M.Params("dkv", (9, 9), (), 3, 2, mistake="deltas_not_awaited"),
    M.Params("dq", LONG, (), 3, 2, mistake="dp_not_awaited"),
    M.Params("dq", LONG, (), 3, 2, mistake="delta_not_awaited"),
    M.Params("dq", LONG, (), 5, 4, mistake="one_tile_kept"),
], ids=lambda p: p.mistake)
def test_planted_mistakes_are_caught(p):
    right = M.Params(**{**p.__dict__, "mistake": ""})
    caught = 0
    for seed in range(60):
        M.run(right, seed, bias=(seed % 3) / 2)
        try:
            M.run(p, seed, bias=(seed % 3) / 2)
        except AssertionError:
            caught += 1
    assert caught
