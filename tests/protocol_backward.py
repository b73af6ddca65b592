"""Executable model of the backward kernels' synchronisation (transformer_attention_02_gb300/csrc/bwd_kernel.cuh).

The loading warp, the issuing warp and the element-wise warps of bwd_dkv_kernel and bwd_dq_kernel are restated as generators over
the blocks of a CTA's tiles (any list of lengths, tiles without a pair among them) and run under an adversarial scheduler together
with the copies they start, which land in any order, and the tensor cores' in-order queue. Checked on every interleaving:

* no deadlock, and no wait whose parity a barrier has run past (protocol_model.Sim.poll);
* no copy into a buffer that a product or a warp still reads; every product finds the K, V, Q, dO, P and dS that it is for;
* S and dP are overwritten only once P and dS have been used, the accumulators once every warp has taken the tile before;
* where a wait runs out, at any moment, every role ends, its copies landed and its products run.

Four element-wise warps in two groups stand for the sixteen in four.
"""
from __future__ import annotations

import random
from dataclasses import dataclass

from protocol_model import Barrier, Proc, ProtocolError, Sim, _advance

WARPS = 4
RING = 2


@dataclass
class Params:
    kernel: str = "dkv"              # or "dq"
    tiles: tuple = (3, 1, 0, 2)      # blocks of the CTA's tiles, in order
    twice: tuple = ()                # dq: tiles that are walked twice (additive mask), by their place in `tiles`
    k_ring: int = 3                  # dq: K and V; dkv: Q and dO
    v_ring: int = 2
    stall: bool = False
    mistake: str = ""                # one that must be caught


class Place:
    def __init__(self, n, at=0, round=0):
        self.n, self.at, self.round = n, at, round

    def next(self):
        return Place(self.n, 0, self.round + 1) if self.at + 1 == self.n else Place(self.n, self.at + 1, self.round)


def bars(p: Params):
    """{barrier: arrivals}"""
    b = {"stall": 1, "drain": 1, "acc": 1, "acc_empty": WARPS}
    for i in range(RING):
        b[f"tile{i}"], b[f"tile_empty{i}"] = 1, WARPS + 1
    if p.kernel == "dkv":
        b.update({"K": 1, "V": 1, "K_empty": 1, "V_empty": 1, "P": WARPS, "dS": WARPS, "S": 1, "dP": 1})
        for i in range(p.k_ring):
            b[f"Q{i}"], b[f"Q_empty{i}"] = 1, WARPS + 1
        for i in range(p.v_ring):
            b[f"G{i}"], b[f"G_empty{i}"] = 1, 1 if p.mistake == "deltas_not_awaited" else WARPS + 1
    else:
        b.update({"Q": 1, "Q_empty": 1, "G": 1, "G_empty": WARPS + 1, "dP": 1, "dP_free": WARPS, "delta": WARPS, "parts": WARPS // 2,
                  "whole": WARPS // 2})
        for i in range(2):
            b[f"S{i}"], b[f"dS{i}"] = 1, WARPS
        for i in range(p.k_ring):
            b[f"K{i}"], b[f"K_empty{i}"] = 1, 1
        for i in range(p.v_ring):
            b[f"V{i}"], b[f"V_empty{i}"] = 1, 1
    return b


# ------------------------------------------------------------ shared pieces

def publish(sim, k, entry):
    if k >= RING and not (yield ("wait", f"tile_empty{k % RING}", k // RING - 1)):
        return False

    def write():
        sim.res[f"entry{k % RING}"] = (k, entry)
    yield ("act", write)
    yield ("arrive", f"tile{k % RING}")
    return True


def next_tile(sim, k):
    """The k-th entry, or None at the end and where a wait runs out."""
    if not (yield ("wait", f"tile{k % RING}", k // RING)):
        return None
    box = []

    def read():
        got = sim.res[f"entry{k % RING}"]
        if got[0] != k:
            raise ProtocolError(f"entry {got[0]} read as entry {k}")
        box.append(got[1])
    yield ("act", read)
    yield ("arrive", f"tile_empty{k % RING}")
    return box[0]


def load(bar, res, tag):
    yield ("expect_tx", bar, 1)
    yield ("tma", bar, 1, res, tag)


def wait2(a, b):
    return (yield ("wait", *a)) and (yield ("wait", *b))


def follow(first, waits, tail, head):
    """The rest of one product and the beginning of the next. `first`: whether the barriers are looked at before."""
    if first:
        seen = True
        for w in waits:
            seen = (yield ("probe", *w)) and seen
        if seen:
            yield from tail()
            yield from head()
            return True
    yield from tail()
    for w in waits:
        if not (yield ("wait", *w)):
            return False
    yield from head()
    return True


def over_d(sim, where, ident, half, a, b):
    """Half of S or dP into `where`, in the tensor cores' queue: both operands as expected, and what was there before used up."""
    def fn():
        for name, tag in (a, b):
            sim.expect(name, tag, f"{where} of {ident}")
        for w in range(WARPS):
            got = sim.res.get(f"{where}.{w}")
            if half == 0 and not (got is None or got[0] == "used"):
                raise ProtocolError(f"{where} of {ident} over {got}")
            sim.res[f"{where}.{w}"] = ("half" if half == 0 else "whole", ident)
    return ("mma", (a[0], b[0]), fn)


def over_rows(sim, acc, where, ident, half, b, first, last, tile, readers):
    """Half of an accumulator's product: P or dS left by every warp, the buffer as expected."""
    def fn():
        sim.expect(*b, f"{acc} of {ident}")
        for w in range(WARPS):
            sim.expect(f"{where}.{w}", ("left", ident), f"{acc} of {ident}")
        state = sim.res.get(acc)
        if half == 0 and first:
            if state is not None and state != ("taken", tile - 1, readers):
                raise ProtocolError(f"{acc} of tile {tile} over {state}")
        elif state != ("sum", tile):
            raise ProtocolError(f"{acc} of tile {tile} goes on from {state}")
        sim.res[acc] = ("done", tile) if half and last else ("sum", tile)
        if half:
            for w in range(WARPS):
                sim.res[f"{where}.{w}"] = ("used", ident)
    return ("mma", (b[0],), fn)


def take(sim, acc, tile, readers):
    """A warp has a tile's accumulator in registers."""
    got = sim.res.get(acc)
    if got == ("done", tile):
        sim.res[acc] = ("taken", tile, 1)
    elif got is not None and got[0] == "taken" and got[1] == tile and got[2] < readers:
        sim.res[acc] = ("taken", tile, got[2] + 1)
    else:
        raise ProtocolError(f"{acc} of tile {tile} taken from {got}")


def shut_down(issued):
    if issued:
        yield ("commit", "drain")
        yield ("drain", "drain", 0)


def drains(fills):
    """fills: (barriers' names, number of copies)"""
    for names, n in fills:
        for s, name in enumerate(names):
            if n > s:
                yield ("drain", name, (n - 1 - s) // len(names))


# ------------------------------------------------------------------ dK, dV

def dkv_load(sim):
    p = sim.p
    tiles = v_fills = q_fills = g_fills = 0
    q, g = Place(p.k_ring), Place(p.v_ring)
    alive = True
    for t, n in list(enumerate(p.tiles)) + [(-1, -1)]:
        if n == 0:
            continue
        if not (yield from publish(sim, tiles, None if t < 0 else (tiles, n))) or t < 0:
            break
        if tiles > 0 and not (yield ("wait", "K_empty", tiles - 1)):
            break
        yield from load("K", "K", ("K", tiles))
        tiles += 1
        for it in range(n):
            ident = (tiles - 1, it)
            if q.round > 0:
                alive = yield ("wait", f"Q_empty{q.at}", q.round - 1)
                if not alive:
                    break
            yield from load(f"Q{q.at}", f"q{q.at}", ("Q", ident))
            q_fills += 1
            q = q.next()
            if g.round > 0:
                alive = yield ("wait", f"G_empty{g.at}", g.round - 1)
                if not alive:
                    break
            yield from load(f"G{g.at}", f"g{g.at}", ("G", ident))
            g_fills += 1
            g = g.next()
            if it == 0:
                if v_fills > 0 and p.mistake != "v_not_awaited":
                    alive = yield ("wait", "V_empty", v_fills - 1)
                    if not alive:
                        break
                yield from load("V", "V", ("V", tiles - 1))
                v_fills += 1
        if not alive:
            break
    yield from drains([(["K"], tiles), (["V"], v_fills), ([f"Q{i}" for i in range(p.k_ring)], q_fills),
                       ([f"G{i}" for i in range(p.v_ring)], g_fills)])


def dkv_issue(sim):
    p = sim.p
    k = tiles = use = it = n = 0
    q, g = Place(p.k_ring), Place(p.v_ring)
    alive, issued = True, False

    def next_work():
        nonlocal k
        e = yield from next_tile(sim, k)
        k += 1
        return 0 if e is None else e[1]

    def s(half, ident, at):
        return over_d(sim, "S", ident, half, ("K", ("K", ident[0])), (f"q{at}", ("Q", ident)))

    def dp(half, ident, at):
        return over_d(sim, "dP", ident, half, ("V", ("V", ident[0])), (f"g{at}", ("G", ident)))

    if p.stall:
        alive = yield ("wait", "stall", 0)
    if alive:
        n = yield from next_work()
    if n > 0:
        alive = yield from wait2(("K", 0), (f"Q{q.at}", q.round))
        if alive:
            issued = True
            yield s(0, (0, 0), q.at)
            yield s(1, (0, 0), q.at)
            yield ("commit", "S")
            if n == 1:
                yield ("commit", "K_empty")
            alive = yield from wait2(("V", 0), (f"G{g.at}", g.round))
        if alive:
            yield dp(0, (0, 0), g.at)
    while alive and n > 0:
        last, drained, ident = it + 1 == n, it > 0 or tiles == 0, (tiles, it)
        waits = [("P", use)] + ([] if drained or p.mistake == "accumulators_not_awaited" else [("acc_empty", tiles - 1)])

        def dv(half, ident=ident, g=g, first=it == 0, last=last, tile=tiles):
            return over_rows(sim, "dV", "S", ident, half, (f"g{g.at}", ("G", ident)), first, last, tile, WARPS // 2)

        def dk(half, ident=ident, q=q, first=it == 0, last=last, tile=tiles):
            return over_rows(sim, "dK", "dP", ident, half, (f"q{q.at}", ("Q", ident)), first, last, tile, WARPS // 2)

        def dp_rest(ident=ident, g=g, last=last):
            yield dp(1, ident, g.at)
            yield ("commit", "dP")
            if last:
                yield ("commit", "V_empty")

        def one(op):
            def f():
                yield op
            return f

        def dv_rest(g=g):
            yield dv(1)
            yield ("commit", f"G_empty{g.at}")

        def dk_rest(q=q, last=last):
            yield dk(1)
            yield ("commit", f"Q_empty{q.at}")
            if last:
                yield ("commit", "acc")

        def dk_all():
            yield dk(0)
            yield from dk_rest()

        alive = yield from follow(True, waits, dp_rest, one(dv(0)))
        if not alive:
            break
        q1, g1 = q.next(), g.next()
        n1, i1 = ((yield from next_work()), 0) if last else (n, it + 1)
        ds_wait = [] if p.mistake == "ds_not_awaited" else [("dS", use)]
        if n1 == 0:
            alive = yield from follow(False, ds_wait, dv_rest, dk_all)
            break
        ident1 = (tiles + last, i1)

        def s_rest(i1=i1, n1=n1, ident1=ident1, q1=q1):
            yield s(1, ident1, q1.at)
            yield ("commit", "S")
            if i1 + 1 == n1:
                yield ("commit", "K_empty")

        alive = yield from follow(True, [(f"Q{q1.at}", q1.round)] + ([("K", tiles + 1)] if last else []), dv_rest,
                                  one(s(0, ident1, q1.at)))
        if not alive:
            break
        alive = yield from follow(True, ds_wait, s_rest, one(dk(0)))
        if not alive:
            break
        alive = yield from follow(True, [(f"G{g1.at}", g1.round)] + ([("V", tiles + 1)] if last else []), dk_rest,
                                  one(dp(0, ident1, g1.at)))
        tiles += last
        n, it, q, g = n1, i1, q1, g1
        use += 1
    yield from shut_down(issued)


def dkv_warp(sim, w):
    p = sim.p
    acc = "dK" if w >= WARPS // 2 else "dV"
    tiles = use = k = 0
    q, g = Place(p.k_ring), Place(p.v_ring)
    done = False
    alive = True

    def finish():
        nonlocal done, tiles
        if not done:
            return True
        if not (yield ("wait", "acc", tiles)):
            return False
        yield ("act", lambda t=tiles: take(sim, acc, t, WARPS // 2))
        yield ("arrive", "acc_empty")
        done = False
        tiles += 1
        return True

    while alive:
        e = yield from next_tile(sim, k)
        k += 1
        if e is None:
            break
        tile, n = e
        for it in range(n):
            ident = (tile, it)
            alive = yield ("wait", f"Q{q.at}", q.round)
            if not alive:
                break
            alive = yield ("wait", "S", use)
            if not alive:
                break

            def left_p(ident=ident, at=q.at):
                sim.expect(f"q{at}", ("Q", ident), f"statistics of {ident}")
                sim.expect(f"S.{w}", ("whole", ident), f"P of {ident}")
                sim.res[f"S.{w}"] = ("left", ident)
            yield ("act", left_p)
            yield ("arrive", "P")
            yield ("arrive", f"Q_empty{q.at}")
            if it == 0:
                alive = yield from finish()
                if not alive:
                    break
            alive = yield from wait2((f"G{g.at}", g.round), ("dP", use))
            if not alive:
                break

            def left_ds(ident=ident, at=g.at):
                sim.expect(f"g{at}", ("G", ident), f"delta of {ident}")
                sim.expect(f"dP.{w}", ("whole", ident), f"dS of {ident}")
                sim.res[f"dP.{w}"] = ("left", ident)
            yield ("act", left_ds)
            yield ("arrive", "dS")
            if p.mistake != "deltas_not_awaited":
                yield ("arrive", f"G_empty{g.at}")
            use += 1
            q, g = q.next(), g.next()
        if not alive:
            break
        done = True
    if alive:
        yield from finish()


# ---------------------------------------------------------------------- dQ

def dq_load(sim):
    p = sim.p
    tiles = g_fills = kf = vf = 0
    alive = True

    def load_k(ident):
        nonlocal kf
        s = kf % p.k_ring
        if kf >= p.k_ring and not (yield ("wait", f"K_empty{s}", kf // p.k_ring - 1)):
            return False
        yield from load(f"K{s}", f"k{s}", ("K", ident))
        kf += 1
        return True

    for t, n in list(enumerate(p.tiles)) + [(-1, -1)]:
        if n == 0:
            continue
        twice = t in p.twice
        if not (yield from publish(sim, tiles, None if t < 0 else (tiles, n, twice))) or t < 0:
            break
        if tiles > 0 and not (yield ("wait", "Q_empty", tiles - 1)):
            break
        yield from load("Q", "q", ("Q", tiles))
        tiles += 1
        if twice:
            for j in range(n):
                alive = yield from load_k((tiles - 1, j))
                if not alive:
                    break
        for j in range(n if alive else 0):
            ident = (tiles - 1, j + n if twice else j)
            alive = yield from load_k(ident)
            if not alive:
                break
            if j == 0:
                if g_fills > 0:
                    alive = yield ("wait", "G_empty", g_fills - 1)
                    if not alive:
                        break
                yield from load("G", "g", ("G", tiles - 1))
                g_fills += 1
            s = vf % p.v_ring
            if vf >= p.v_ring:
                alive = yield ("wait", f"V_empty{s}", vf // p.v_ring - 1)
                if not alive:
                    break
            yield from load(f"V{s}", f"v{s}", ("V", ident))
            vf += 1
        if not alive:
            break
    yield from drains([(["Q"], tiles), (["G"], g_fills), ([f"K{i}" for i in range(p.k_ring)], kf),
                       ([f"V{i}" for i in range(p.v_ring)], vf)])


class At:
    def __init__(self):
        self.tile = self.j = self.n = self.skip = 0

    def begin(self, blocks):
        self.j, self.n, self.skip = 0, abs(blocks) * (2 if blocks < 0 else 1), max(0, -blocks)


def dq_issue(sim):
    p = sim.p
    k = su = ds = dp = 0
    at_s, at_dp, at_dq = At(), At(), At()
    ka, kb, v = Place(p.k_ring), Place(p.k_ring), Place(p.v_ring)
    kept = [0] * (1 if p.mistake == "one_tile_kept" else 4)
    open_ = []                       # second halves of what is half issued, with what follows them
    alive, issued = True, False

    def next_work():
        nonlocal k
        e = yield from next_tile(sim, k)
        k += 1
        n = 0 if e is None else (-e[1] if e[2] else e[1])
        at_s.begin(n)
        kept[at_s.tile % len(kept)] = n

    def go_on(a):
        a.j += 1
        if a.j < a.n:
            return
        a.tile += 1
        a.begin(kept[a.tile % len(kept)])

    def rest():
        for ops in open_:
            yield from ops
        open_.clear()

    def one(op):
        def f():
            yield op
        return f

    def begin_s():
        nonlocal su, ka, issued
        ident, first, buf = (at_s.tile, at_s.j), at_s.j == 0, su & 1
        operands = (("q", ("Q", at_s.tile)), (f"k{ka.at}", ("K", ident)))
        waits = [(f"K{ka.at}", ka.round)] + ([("Q", at_s.tile)] if first else [])
        if not (yield from follow(True, waits, rest, one(over_d(sim, f"S{buf}", ident, 0, *operands)))):
            return False
        issued = True
        ends = at_s.j + 1 == at_s.n
        open_.extend([[over_d(sim, f"S{buf}", ident, 1, *operands), ("commit", f"S{buf}")] + ([("commit", "Q_empty")] if ends else [])])
        su += 1
        ka = ka.next()
        if ends:
            yield from rest()
            at_s.tile += 1
            yield from next_work()
        else:
            at_s.j += 1
        return True

    def begin_dp():
        nonlocal dp, v
        if at_dp.j >= at_dp.skip:
            ident, first = (at_dp.tile, at_dp.j), at_dp.j == at_dp.skip
            operands = (("g", ("G", at_dp.tile)), (f"v{v.at}", ("V", ident)))
            free_dp = [("dP_free", dp - 1)] if dp and p.mistake != "dp_not_awaited" else []
            waits = [(f"V{v.at}", v.round)] + free_dp + ([("G", at_dp.tile)] if first else [])

            if not (yield from follow(dp > 0 and not first, waits, rest, one(over_d(sim, "dP", ident, 0, *operands)))):
                return False
            ends = at_dp.j + 1 == at_dp.n
            open_.extend([[over_d(sim, "dP", ident, 1, *operands), ("commit", "dP"), ("commit", f"V_empty{v.at}")] +
                          ([("commit", "G_empty")] if ends else [])])
            dp += 1
            v = v.next()
        go_on(at_dp)
        return True

    def begin_dq():
        nonlocal ds, kb
        ident, buf = (at_dq.tile, at_dq.j), ds & 1
        mine = (f"dS{buf}", ds >> 1)
        if at_dq.j < at_dq.skip:
            yield from rest()
            if not (yield ("wait", *mine)):
                return False
            yield ("commit", f"K_empty{kb.at}")
        else:
            first = at_dq.j == at_dq.skip
            drained, tile = not first or at_dq.tile == 0, at_dq.tile
            ends = at_dq.j + 1 == at_dq.n

            def half(i):
                return over_rows(sim, "dQ", f"S{buf}", ident, i, (f"k{kb_at}", ("K", ident)), first, ends, tile, WARPS)
            kb_at = kb.at
            waits = [mine] + ([] if drained else [("acc_empty", tile - 1)])
            if not (yield from follow(True, waits, rest, one(half(0)))):
                return False
            open_.extend([[half(1), ("commit", f"K_empty{kb_at}")] + ([("commit", "acc")] if ends else [])])
        ds += 1
        kb = kb.next()
        go_on(at_dq)
        return True

    if p.stall:
        alive = yield ("wait", "stall", 0)
    if alive:
        yield from next_work()
        for a in (at_dp, at_dq):
            a.tile, a.j, a.n, a.skip = at_s.tile, at_s.j, at_s.n, at_s.skip
        if at_s.n:
            alive = (yield from begin_s()) and (yield from begin_dp()) and (at_s.n == 0 or (yield from begin_s()))
    while alive and at_dq.n > 0:
        alive = (at_dp.n == 0 or (yield from begin_dp())) and (yield from begin_dq()) and (at_s.n == 0 or (yield from begin_s()))
    if alive:
        yield from rest()
    yield from shut_down(issued)


def dq_warp(sim, w):
    p = sim.p
    tiles = su = dp = seen = k = 0
    done = False
    alive = True
    upper = w >= WARPS // 2              # not of the first group

    def finish():
        nonlocal done, tiles
        if not done:
            return True
        if not (yield ("wait", "acc", tiles)):
            return False
        yield ("act", lambda t=tiles: take(sim, "dQ", t, WARPS))
        yield ("arrive", "acc_empty")
        done = False
        tiles += 1
        return True

    def logits(ident):
        if not (yield ("wait", f"S{su & 1}", su >> 1)):
            return False
        yield ("act", lambda b=su & 1: sim.expect(f"S{b}.{w}", ("whole", ident), f"logits of {ident}"))
        return True

    def find_delta(tile):
        if not (yield ("wait", "G", k)):
            return False

        def write():
            sim.expect("g", ("G", tile), f"delta of tile {tile}")
            if len(sim.res.get("readers", ())) not in (0, WARPS):
                raise ProtocolError(f"delta of tile {tile} over one that {sim.res['readers']} alone have read")
            sim.res[f"delta.{w}"] = tile
        yield ("act", write)
        yield ("arrive", "delta")
        if p.mistake != "delta_not_awaited" and not (yield ("wait", "delta", k)):
            return False

        def read():
            for x in range(WARPS):
                sim.expect(f"delta.{x}", tile, f"delta of tile {tile}")
            old = sim.res.get("readers", ())
            sim.res["readers"] = (() if len(old) == WARPS else old) + (w,)
        yield ("act", read)
        yield ("arrive", "G_empty")
        return True

    while alive:
        e = yield from next_tile(sim, k)
        if e is None:
            break
        tile, n, twice = e
        if twice:
            for j in range(n):
                alive = yield from logits((tile, j))
                if not alive:
                    break

                def through(b=su & 1, ident=(tile, j)):
                    sim.res[f"S{b}.{w}"] = ("used", ident)
                yield ("act", through)
                yield ("arrive", f"dS{su & 1}")
                if j == 0:
                    alive = yield from finish()
                    if not alive:
                        break
                su += 1
            if not alive:
                break
            if upper:
                def part(t=tile):
                    sim.res[f"part.{w}"] = t
                yield ("act", part)
                yield ("arrive", "parts")
                alive = yield ("wait", "whole", seen)
            else:
                alive = yield ("wait", "parts", seen)
                if alive:
                    def join(t=tile):
                        for x in range(WARPS // 2, WARPS):
                            sim.expect(f"part.{x}", t, f"statistics of tile {t}")
                        sim.res[f"whole.{w}"] = t
                    yield ("act", join)
                    yield ("arrive", "whole")
            if not alive:
                break
            mine = w - WARPS // 2 if upper else w
            yield ("act", lambda t=tile: sim.expect(f"whole.{mine}", t, f"statistics of tile {t}"))
            seen += 1
        for j in range(n):
            ident = (tile, j + n if twice else j)
            alive = yield from logits(ident)
            if not alive:
                break
            if j == 0:
                alive = (yield from finish()) and (yield from find_delta(tile))
                if not alive:
                    break
            alive = yield ("wait", "dP", dp)
            if not alive:
                break

            def hold(ident=ident):
                sim.expect(f"dP.{w}", ("whole", ident), f"dP of {ident}")
                sim.res[f"dP.{w}"] = ("used", ident)
            yield ("act", hold)
            yield ("arrive", "dP_free")

            def left(b=su & 1, ident=ident):
                sim.expect(f"S{b}.{w}", ("whole", ident), f"dS of {ident}")
                sim.res[f"S{b}.{w}"] = ("left", ident)
            yield ("act", left)
            yield ("arrive", f"dS{su & 1}")
            su += 1
            dp += 1
        if not alive:
            break
        done = True
        k += 1
    if alive:
        yield from finish()


# ---------------------------------------------------------------- scheduler

def run(p: Params, seed: int = 0, timeouts: bool = False, bias: float = 0.5, abort_at: int = None, max_steps: int = 400_000):
    """One adversarially scheduled execution; ProtocolError on a violation or a deadlock."""
    sim = Sim(p, random.Random(seed), timeouts=timeouts)
    for name, count in bars(p).items():
        sim.bars[name] = Barrier(name, count)
    roles = (dkv_load, dkv_issue, dkv_warp) if p.kernel == "dkv" else (dq_load, dq_issue, dq_warp)
    procs = [Proc("load", roles[0](sim)), Proc("issue", roles[1](sim))] + [Proc(f"warp{w}", roles[2](sim, w)) for w in range(WARPS)]
    rng = sim.rng
    for pr in procs:
        _advance(pr)
    prio = {name: rng.random() for name in [pr.name for pr in procs] + ["copies", "products"]}

    def runnable(pr):
        if pr.op[0] == "wait":
            return sim.abort or sim.poll(pr.op[1], pr.op[2])
        return pr.op[0] != "drain" or sim.poll(pr.op[1], pr.op[2])

    while not all(pr.done for pr in procs):
        sim.steps += 1
        if sim.steps == abort_at:
            sim.abort = sim.timed_out = True
        if sim.steps > max_steps:
            raise ProtocolError("step limit reached")
        cands = [(pr.name, pr) for pr in procs if not pr.done and runnable(pr)]
        cands += [("copies", i) for i in range(len(sim.inflight))] + ([("products", None)] if sim.mma_queue else [])
        if not cands:
            blocked = [pr for pr in procs if not pr.done]
            waiting = [pr for pr in blocked if pr.op[0] == "wait"]
            if not timeouts or not waiting:
                raise ProtocolError("deadlock: " + ", ".join(f"{pr.name} at {pr.op}" for pr in blocked))
            sim.abort = sim.timed_out = True                    # the bounded wait runs out
            _advance(rng.choice(waiting), False)
            continue
        name, obj = max(cands, key=lambda c: prio[c[0]] + 0.3 * rng.random()) if rng.random() < bias else rng.choice(cands)
        if name == "copies":
            bar, nbytes, res, tag, _ = sim.inflight.pop(obj)
            sim.res[res] = tag
            sim.bars[bar].complete_tx(nbytes)
            continue
        if name == "products":
            item = sim.mma_queue.popleft()
            try:
                item[2]() if item[0] == "mma" else sim.bars[item[1]].arrive()
            except ProtocolError:
                if not sim.abort:                               # (a call that gives up leaves its results undefined)
                    raise
            continue
        op, val = obj.op, None
        if op[0] in ("wait", "probe"):
            val = sim.poll(op[1], op[2])
        elif op[0] == "arrive":
            sim.bars[op[1]].arrive()
        elif op[0] == "expect_tx":
            sim.bars[op[1]].expect_tx(op[2])
            sim.bars[op[1]].arrive()
        elif op[0] == "tma":
            sim.tma_issue(op[1], op[2], op[3], op[4], obj.name)
        elif op[0] in ("mma", "commit"):
            sim.mma_queue.append(op)
        elif op[0] == "act":
            try:
                op[1]()
            except ProtocolError:
                if not sim.abort:
                    raise
        elif op[0] != "drain":
            raise ProtocolError(f"unknown op {op}")
        _advance(obj, val)
        if obj.done and any(f[4] == obj.name for f in sim.inflight):
            raise ProtocolError(f"{obj.name} left with a copy in flight")
    if sim.inflight or sim.mma_queue:
        raise ProtocolError("the kernel ended with copies or products in flight")
    if not sim.abort:
        worked = sum(n > 0 for n in p.tiles)
        for acc, readers in (("dQ", WARPS),) if p.kernel == "dq" else (("dV", WARPS // 2), ("dK", WARPS // 2)):
            if worked and sim.res.get(acc) != ("taken", worked - 1, readers):
                raise ProtocolError(f"{acc} at the end: {sim.res.get(acc)}")
    return sim
