"""The barrier protocol of the windowed attention variants, checked on the CPU.

They differ from the other variants in the list of key blocks a tile streams (the sinks' blocks, then the window's) and
in one block of it that the upper sub-tile passes over: the MMA issuer issues neither product of it for that sub-tile
and its softmax warpgroup does not wait for it. The issuer's and the softmax's roles are re-stated here with that rule
and run in the model of protocol_model under the same adversarial schedules, with every check it makes; an issuer and a
softmax that disagree about the block must be caught.
"""
import dataclasses

import pytest

import protocol_model as M


@dataclasses.dataclass(frozen=True)
class WindowTile(M.Tile):
    passed: int = -1               # list index of the block that the upper sub-tile passes over


def window_schedule(window, sinks, plain):
    """The causal schedule's tiles with the key blocks of a window: what tile_info computes, from the definition of the
    visible keys."""
    def schedule(p):
        out = []
        for t in plain(p):
            off = p.Sk - p.Sq
            rows = [[r for r in range(t.m0 + 128 * s, min(t.m0 + 128 * (s + 1), p.Sq))] for s in range(2)]
            sub = []
            for rs in rows:
                seen = set()
                for r in rs:
                    pos = r + off
                    for lo, hi in ((max(0, pos - window + 1), pos + 1), (0, min(sinks, pos + 1))):
                        seen.update(range(lo // 128, -(-hi // 128)) if hi > lo else ())
                sub.append(seen)
            blocks = sorted(sub[0] | sub[1])
            nb = [max((blocks.index(b) + 1 for b in s), default=0) for s in sub]
            passed = [i for i in range(nb[1]) if blocks[i] not in sub[1]]
            assert len(passed) <= 1 and not [i for i in range(nb[0]) if blocks[i] not in sub[0]]
            out.append(WindowTile(t.b, t.h, t.hk, t.m0, t.split, t.kb0, tuple(nb), max(nb), *passed))
        return out
    return schedule


def _pv(sim, ti, t, v_slot, blk, before):
    """O_t (+)= P_t V_blk; `before`: the block of the sub-tile's product before this one, or None."""
    key = M._tile_key(ti)

    def fn():
        sim.expect(f"S{t}", ("P", key, t, blk), f"P V of {key} sub-tile {t} block {blk}")
        sim.expect(f"kv{v_slot}", ("KV", 1, ti.b, ti.hk, ti.kb0 + blk), f"P V of {key} sub-tile {t} block {blk}")
        o = sim.res.get(f"O{t}", "free")
        if before is None:
            if not (o == "free" or o[0] == "read"):
                raise M.ProtocolError(f"first P V of {key} sub-tile {t} overwrites O{t} holding {o}")
        elif o != ("O", key, t, before):
            raise M.ProtocolError(f"P V of {key} sub-tile {t} block {blk}: O{t} holds {o}")
        sim.res[f"S{t}"] = "free"
        sim.res[f"O{t}"] = ("O", key, t, blk)
    return ("mma", (f"S{t}", f"kv{v_slot}"), fn)


def role_mma(sim, tiles, honours=True):
    p, S = sim.p, sim.p.slots
    st = {"use": 0}
    p_cnt = [0, 0]
    nq, k, alive, issued = 0, 0, True, False

    def acquire():
        slot = st["use"] % S
        ok = yield ("wait", f"kv_full{slot}", st["use"] // S)
        st["use"] += 1
        return slot, ok

    while alive:
        ok, ti = yield from M.ring_fetch(sim, k)
        if not ok or ti is None:
            break
        k += 1
        n, (n0, n1) = ti.n, ti.nb
        passed = ti.passed if honours else -1
        on = lambda t, j: j < (n0, n1)[t] and not (t == 1 and j == passed)          # noqa: E731
        prev = [None, None]
        if n == 0:
            continue
        q_buf = M.q_bufs_of(nq, p.q_bufs)
        ok = yield ("wait", f"q_full{q_buf[0]}", M.q_slot(nq, 0, p.q_bufs)[1])
        if ok:
            ks, ok = yield from acquire()
        if not ok:
            break
        issued = True
        if on(0, 0):
            yield M._qk(sim, ti, 0, q_buf[0], ks, 0)
            yield ("commit", "s_full0")
        ok = yield ("wait", f"q_full{q_buf[1]}", M.q_slot(nq, 1, p.q_bufs)[1])
        if not ok:
            break
        nq += 1
        if on(1, 0):
            yield M._qk(sim, ti, 1, q_buf[1], ks, 0)
            yield ("commit", "s_full1")
        yield ("commit", f"kv_empty{ks}")
        for t, nt in ((0, n0), (1, n1)):
            if nt <= 1:
                yield ("commit", f"q_empty{q_buf[t]}")
        for j in range(n):
            more = j + 1 < n
            vs, alive = yield from acquire()
            if not alive:
                break
            for t, nt in ((0, n0), (1, n1)):
                if on(t, j):
                    alive = yield ("wait", f"p_full{t}", p_cnt[t])
                    p_cnt[t] += 1
                    if not alive:
                        break
                    yield _pv(sim, ti, t, vs, j, prev[t])
                    prev[t] = j
                    if j == nt - 1:
                        yield ("commit", f"o_full{t}")
                if t == 0 and more:
                    ks, alive = yield from acquire()
                    if not alive:
                        break
                if t == 1:
                    yield ("commit", f"kv_empty{vs}")
                if more and on(t, j + 1):
                    yield M._qk(sim, ti, t, q_buf[t], ks, j + 1)
                    yield ("commit", f"s_full{t}")
                if more and t == 1:
                    yield ("commit", f"kv_empty{ks}")
                if more and j + 2 == nt:
                    yield ("commit", f"q_empty{q_buf[t]}")
            if not alive:
                break
    if issued:
        yield ("commit", "drain")
        yield ("drain", "drain", 0)


def role_softmax(sim, tiles, t):
    s_cnt = o_cnt = k = 0
    while True:
        ok, ti = yield from M.ring_fetch(sim, k, arrivals=4)
        if not ok or ti is None:
            return
        k += 1
        key, nb, prev = M._tile_key(ti), ti.nb[t], None
        if nb == 0:
            continue
        for j in range(nb):
            if t == 1 and j == ti.passed:
                continue
            landed = yield ("wait", f"s_full{t}", s_cnt)
            s_cnt += 1
            if not landed:
                return

            def fn(j=j, prev=prev):
                sim.expect(f"S{t}", ("S", key, t, j), f"softmax {t} block {j}")
                if prev is not None:
                    sim.expect(f"O{t}", ("O", key, t, prev), f"rescale of O{t} at block {j}")
                sim.res[f"S{t}"] = ("P", key, t, j)
            yield ("act", fn)
            prev = j
            yield ("arrive", f"p_full{t}")
        ok = yield ("wait", f"o_full{t}", o_cnt)
        if not ok:
            return
        o_cnt += 1

        def epi(last=prev):
            sim.expect(f"O{t}", ("O", key, t, last), f"epilogue {t}")
            sim.res[f"O{t}"] = ("read", key, t)
        yield ("act", epi)


CASES = [
    (M.Params(Sq=1200, Sk=1200), 200, 0),
    (M.Params(Sq=1200, Sk=1200), 128, 0),                       # the passed block is the first of the list
    (M.Params(D=64, Sq=1500, Sk=1500), 300, 130),               # after two blocks of sinks
    (M.Params(Sq=1500, Sk=1500), 1, 4),
    (M.Params(Sq=300, Sk=2000), 500, 4),
    (M.Params(Sq=900, Sk=300, D=64), 100, 0),                   # leading tiles without a key
    (M.Params(Sq=100, Sk=1000), 400, 3),                        # upper sub-tile without rows
    (M.Params(B=2, Hq=4, Hkv=2, Sq=1200, Sk=1200, cta=3, steal_seed=1), 260, 4),
]
IDS = lambda c: f"D{c.D}_S{c.Sq}-{c.Sk}" if isinstance(c, M.Params) else str(c)      # noqa: E731


@pytest.fixture
def windowed(monkeypatch):
    plain = M.schedule

    def use(window, sinks, mma=role_mma):
        monkeypatch.setattr(M, "schedule", window_schedule(window, sinks, plain))
        monkeypatch.setattr(M, "role_mma", mma)
        monkeypatch.setattr(M, "role_softmax", role_softmax)
    return use


@pytest.mark.parametrize("p,window,sinks", CASES, ids=IDS)
def test_windowed_protocol_has_no_deadlock_or_race(windowed, p, window, sinks):
    windowed(window, sinks)
    for seed in range(12):
        M.run(p, seed=seed, bias=(seed % 4) / 4)


@pytest.mark.parametrize("p,window,sinks", CASES[:3], ids=IDS)
def test_windowed_abort_terminates(windowed, p, window, sinks):
    windowed(window, sinks)
    for seed in range(12):
        M.run(p, seed=seed, timeouts=True, abort_at=40 + 61 * seed)


def test_an_issuer_that_does_not_pass_over_the_block_is_caught(windowed):
    p, window, sinks = CASES[0]
    windowed(window, sinks, lambda sim, tiles: role_mma(sim, tiles, honours=False))
    assert any(t.passed >= 0 for t in M.schedule(p))
    with pytest.raises(M.ProtocolError):
        for seed in range(12):
            M.run(p, seed=seed)


@pytest.mark.parametrize("p,window,sinks", CASES, ids=IDS)
def test_tile_lists_match_the_kernels_arithmetic(windowed, p, window, sinks):
    """tile_info's integer arithmetic for the block list against the lists from the definition above."""
    plain = M.schedule(p)
    windowed(window, sinks)
    for t, ref in zip(M.schedule(p), plain):
        off = p.Sk - p.Sq
        first = t.m0 + off - window + 1
        low, sink_blocks = max(0, first) // 128, -(-min(sinks, p.Sk) // 128)
        gap, passed = 0, -1
        if low >= sink_blocks:
            gap = low - sink_blocks
            if max(0, first + 128) // 128 > low:
                passed = sink_blocks
        nb = [n - gap if n else 0 for n in ref.nb]
        if nb[1] == 0:
            passed = -1                                          # (no block of the upper sub-tile is ever asked for)
        assert (tuple(nb), passed) == (t.nb, t.passed), (t, nb, passed)
