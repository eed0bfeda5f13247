"""Models of two barrier protocols, with the machinery of tests/test_fwd_protocol.py: the windowed forward
up to d = 128 (csrc/fwd.cu compiled by csrc/fwd_window.cu), whose query tiles visit key tiles of their
own and whose K and V tiles have ring places one by one; and the key weights (csrc/weights.cu), with one
Q tile and with several, in turns, whose two warpgroups' sums meet in shared memory.

They model orders, not memory fences."""
import random

import pytest

from test_fwd_protocol import Hazard, Sim
from test_window_schedule import forward_unit

# ---------------------------------------------------------------------------- forward


class Unit:
    """Steps of a unit's query tiles: which of the unit's steps each takes part in."""

    def __init__(self, Lq, Lk, W, S, m):
        st, n, lo, hi, first, nsink, self.nkv = forward_unit(m, Lq, Lk, W, S, 2)
        tile = [j if j < nsink else first + j - nsink for j in range(self.nkv)]
        self.steps = [[j for j in range(self.nkv) if tile[j] < hi[t] and (tile[j] >= lo[t] or tile[j] < st)]
                      for t in (0, 1)]
        assert [len(s) for s in self.steps] == n

    def active(self, t, j):
        return j in self.steps[t]


def run_forward(units, seed, places, mistake=None, warps=1):
    sim = Sim([(u,) for u in units], seed, consumers=1 + 2 * warps)
    for t in (0, 1):
        for name in ("s_full", "o_done"):
            sim.bar(f"{name}{t}")
        for name in ("p_full", "p_hi", "o_free"):
            sim.bar(f"{name}{t}", warps)
    sim.bar("q_full")
    sim.bar("q_empty")
    for s in range(places):
        sim.bar(f"w_full{s}")
        sim.bar(f"w_empty{s}")
    smem = {}
    st = {"S": {}, "P": {}, "O": {0: [], 1: []}, "read": {}, "q_read": True}

    def producer():
        it_sched = it_unit = w_it = 0
        while True:
            unit = yield from sim.grab(it_sched)
            it_sched += 1
            if unit is None:
                return
            uid, u = unit
            while not sim.ready("q_empty", (it_unit & 1) ^ 1, it_unit):
                yield
            if not st["q_read"]:
                raise Hazard(f"Q of {uid} loaded over a Q still read")
            sim.bars["q_full"].expect_tx(sum(len(s) > 0 for s in u.steps))
            for t in (0, 1):
                if u.steps[t]:
                    st["q_read"] = False
                    sim.issue("q_full", f"q{t}", uid)
            it_unit += 1
            for i in range(2 * u.nkv):
                s = w_it % places
                if mistake != "no_place_wait":
                    while not sim.ready(f"w_empty{s}", ((w_it // places) & 1) ^ 1, w_it // places):
                        yield
                if st["read"].get(s) is False:
                    raise Hazard(f"place {s} reloaded before it was read")
                st["read"][s] = False
                sim.load(f"w_full{s}", f"w{s}", ("kv"[i & 1], uid, i >> 1))
                w_it += 1
                yield

    def mma():
        it_sched = it_unit = kv_it = 0
        it, ep = [0, 0], [0, 0]
        while True:
            unit = yield from sim.take(it_sched)
            it_sched += 1
            if unit is None:
                return
            uid, u = unit
            while not sim.ready("q_full", it_unit & 1, it_unit + 1):
                yield

            def place(p):
                while not sim.ready(f"w_full{p % places}", (p // places) & 1, p // places + 1):
                    yield

            begun = [False, False]
            for j in range(-1, u.nkv):
                vp = 2 * (kv_it + j) + 1
                kp = vp + 1
                v_in = k_in = False
                for t in (0, 1):
                    if j >= 0 and u.active(t, j):
                        while not sim.ready(f"p_full{t}", it[t] & 1, it[t] + 1):
                            yield
                        if not v_in:
                            yield from place(vp)
                        v_in = True
                        if not begun[t] and ep[t] > 0:
                            while not sim.ready(f"o_free{t}", (ep[t] - 1) & 1, ep[t]):
                                yield
                        sim.pipe.append(("PV", (uid, t, j, vp % places, 0, not begun[t])))
                        if mistake != "no_p_hi_wait":
                            while not sim.ready(f"p_hi{t}", it[t] & 1, it[t] + 1):
                                yield
                        sim.pipe.append(("PV", (uid, t, j, vp % places, 1, False)))
                        sim.pipe.append(("commit", f"o_done{t}"))
                        it[t] += 1
                        begun[t] = True
                    if j >= 0 and t == (0 if mistake == "v_free_early" else 1):
                        if not v_in and mistake != "unseen_place":
                            yield from place(vp)
                        v_in = True
                        sim.pipe.append(("read", vp % places))
                        sim.pipe.append(("commit", f"w_empty{vp % places}"))
                    if j + 1 < u.nkv:
                        if not k_in:
                            yield from place(kp)
                        k_in = True
                        if u.active(t, j + 1):
                            if it[t] > 0:
                                while not sim.ready(f"o_done{t}", (it[t] - 1) & 1, it[t]):
                                    yield
                            sim.pipe.append(("S", (uid, t, j + 1, kp % places)))
                            sim.pipe.append(("commit", f"s_full{t}"))
                        if t == 1:
                            sim.pipe.append(("read", kp % places))
                            sim.pipe.append(("commit", f"w_empty{kp % places}"))
                            if j + 1 == u.nkv - 1:
                                sim.pipe.append(("commit", "q_empty"))
                    yield
            kv_it += u.nkv
            it_unit += 1
            for t in (0, 1):
                ep[t] += bool(u.steps[t])

    def softmax(t, w):
        it_sched = it = 0
        while True:
            unit = yield from sim.take(it_sched)
            it_sched += 1
            if unit is None:
                return
            uid, u = unit
            if not u.steps[t]:
                continue
            done = []
            for j in u.steps[t]:
                while not sim.ready(f"s_full{t}", it & 1, it + 1):
                    yield
                for _ in range(2):
                    if st["S"].get(t) != (uid, j):
                        raise Hazard(f"softmax {t}.{w} ({uid},{j}) read S = {st['S'].get(t)}")
                    yield
                if done and sim.rnd.random() < 0.3 and st["O"][t] != done:
                    raise Hazard(f"rescale of tile {t} ({uid},{j}) saw O = {st['O'][t]}")
                for hf, bar in ((0, "p_full"), (1, "p_hi")):
                    yield
                    st["P"].setdefault((t, hf), {})[w] = (uid, j)
                    sim.bars[f"{bar}{t}"].arrive((uid, j))
                    done.append((uid, j, hf))
                it += 1
                yield
            while not sim.ready(f"o_done{t}", (it - 1) & 1, it):
                yield
            for _ in range(2):
                if st["O"][t] != done:
                    raise Hazard(f"epilogue of tile {t} of {uid} read O = {st['O'][t]}")
                yield
            if w == 0:
                sim.out.append((uid, t))
            sim.bars[f"o_free{t}"].arrive(uid)

    def execute(op, arg):
        if op == "commit":
            if arg == "q_empty":
                st["q_read"] = True
            sim.bars[arg].arrive()
        elif op == "read":
            st["read"][arg] = True
        elif op == "S":
            uid, t, j, s = arg
            if smem.get(f"q{t}") != uid or smem.get(f"w{s}") != ("k", uid, j):
                raise Hazard(f"S_{t} ({uid},{j}) read Q {smem.get(f'q{t}')}, K {smem.get(f'w{s}')}")
            for hf in (0, 1):
                if any(v != "read" for v in st["P"].get((t, hf), {}).values()):
                    raise Hazard(f"S_{t} ({uid},{j}) overwrote P before PV read it")
                st["P"][(t, hf)] = {}
            st["S"][t] = (uid, j)
        else:
            uid, t, j, s, hf, first = arg
            quarters = st["P"].get((t, hf), {})
            if smem.get(f"w{s}") != ("v", uid, j) or len(quarters) != warps or any(
                    v != (uid, j) for v in quarters.values()):
                raise Hazard(f"PV_{t} ({uid},{j}) half {hf} read V {smem.get(f'w{s}')}, P {quarters}")
            if first:
                st["O"][t] = []
            st["O"][t].append((uid, j, hf))
            st["P"][(t, hf)] = {q: "read" for q in quarters}

    sim.run([producer(), mma()] + [softmax(t, w) for t in (0, 1) for w in range(warps)], execute, smem)
    want = sorted((i, t) for i, u in enumerate(units) for t in (0, 1) if u.steps[t])
    if sorted(sim.out) != want:
        raise Hazard(f"outputs {sorted(sim.out)}, expected {want}")


def random_units(rnd):
    units = []
    for _ in range(rnd.randint(0, 4)):
        Lq = rnd.choice([1, 100, 128, 129, 300, 700, 1000])
        Lk = rnd.choice([0, Lq, Lq, Lq + 200, max(0, Lq - 150)])
        W, S = rnd.choice([1, 60, 128, 250]), rnd.choice([0, 3, 130, 300])
        units.append(Unit(Lq, Lk, W, S, rnd.randrange(-(-Lq // 256))))
    return units


@pytest.mark.parametrize("warps", [1, 4])
@pytest.mark.parametrize("places", [4, 8])
def test_forward_is_hazard_and_deadlock_free(places, warps):
    for seed in range(200 if warps == 1 else 80):
        run_forward(random_units(random.Random(seed * 11 + 5)), seed, places, warps=warps)


@pytest.mark.parametrize("mistake", ["no_place_wait", "no_p_hi_wait", "v_free_early", "unseen_place"])
def test_forward_planted_mistakes(mistake):
    for seed in range(300):
        try:
            run_forward(random_units(random.Random(seed * 11 + 5)), seed, 4, mistake)
        except Hazard:
            return
    raise AssertionError("not caught")


# ------------------------------------------------------------------------ key weights


def run_weights(pieces, seed, many, stages, qbufs, mistake=None, warps=1):
    """pieces: (key tiles, Q tiles) of a turn each."""
    sim = Sim(pieces, seed, consumers=2 + 2 * warps)
    buffers = 2 if many else 4
    for i in range(buffers):
        sim.bar(f"s_full{i}")
        sim.bar(f"s_free{i}", 2 * warps if many else warps)
    for i in range(qbufs):
        sim.bar(f"q_full{i}", 2)
        sim.bar(f"q_empty{i}", 1 + 2 * warps)
    for i in range(stages):
        sim.bar(f"full{i}")
        sim.bar(f"empty{i}")
    for i in range(4):
        sim.bar(f"x_full{i}", warps)
    smem = {}
    st = {"S": {}, "read": {}, "q_read": {}, "lse": {}, "lse_read": {}, "busy": {}, "x": {}, "sum": {}}

    def keys():
        it = f = 0
        while True:
            piece = yield from sim.grab(it)
            it += 1
            if piece is None:
                return
            uid, tiles, _ = piece
            for j in range(tiles):
                s = f % stages
                while not sim.ready(f"empty{s}", ((f // stages) & 1) ^ 1, f // stages):
                    yield
                if st["read"].get(s) is False:
                    raise Hazard(f"stage {s} reloaded before it was read")
                st["read"][s] = False
                sim.load(f"full{s}", f"k{s}", (uid, j))
                f += 1
                yield

    def queries():
        it = g = 0
        while True:
            piece = yield from sim.take(it)
            it += 1
            if piece is None:
                return
            uid, _, nq = piece
            for qt in range(nq):
                s = g % qbufs
                if mistake != "no_q_wait":
                    while not sim.ready(f"q_empty{s}", ((g // qbufs) & 1) ^ 1, g // qbufs):
                        yield
                if st["q_read"].get(s) is False or st["lse_read"].get(s, 2 * warps) != 2 * warps:
                    raise Hazard(f"Q buffer {s} reloaded before it was read")
                st["q_read"][s], st["lse_read"][s] = False, 0
                sim.load(f"q_full{s}", f"q{s}", (uid, qt))
                yield
                st["lse"][s] = (uid, qt)
                sim.bars[f"q_full{s}"].arrive()
                g += 1
                yield

    def mma():
        it = f = g = 0
        cnt = [0, 0]
        while True:
            piece = yield from sim.take(it)
            it += 1
            if piece is None:
                return
            uid, tiles, nq = piece
            for j in range(tiles):
                for qt in range(nq):
                    gq, w = g + qt, 0 if many else j & 1
                    bf = (0 if many else 2 * w) + (cnt[w] & 1)
                    if j == 0:
                        while not sim.ready(f"q_full{gq % qbufs}", (gq // qbufs) & 1, gq // qbufs + 1):
                            yield
                    if qt == 0:
                        while not sim.ready(f"full{f % stages}", (f // stages) & 1, f // stages + 1):
                            yield
                    if cnt[w] >= 2 and mistake != "no_s_wait":
                        while not sim.ready(f"s_free{bf}", ((cnt[w] - 2) >> 1) & 1, ((cnt[w] - 2) >> 1) + 1):
                            yield
                    sim.pipe.append(("S", (uid, j, qt, f % stages, gq % qbufs, bf)))
                    sim.pipe.append(("commit", f"s_full{bf}"))
                    if qt == nq - 1:
                        sim.pipe.append(("read", f % stages))
                        sim.pipe.append(("commit", f"empty{f % stages}"))
                    if j == tiles - 1:
                        sim.pipe.append(("q_read", gq % qbufs))
                        sim.pipe.append(("commit", f"q_empty{gq % qbufs}"))
                    cnt[w] += 1
                    yield
                f += 1
            g += nq

    def sums(w, q):
        it = g = cnt = x_it = 0
        while True:
            piece = yield from sim.take(it)
            it += 1
            if piece is None:
                return
            uid, tiles, nq = piece
            for qt in range(nq):
                s = (g + qt) % qbufs
                while not sim.ready(f"q_full{s}", ((g + qt) // qbufs) & 1, (g + qt) // qbufs + 1):
                    yield
            for j in range(0 if many else w, tiles, 1 if many else 2):
                for qt in range(nq):
                    s, bf = (g + qt) % qbufs, (0 if many else 2 * w) + (cnt & 1)
                    while not sim.ready(f"s_full{bf}", (cnt >> 1) & 1, (cnt >> 1) + 1):
                        yield
                    st["busy"][bf] = st["busy"].get(bf, 0) + 1
                    for _ in range(2):
                        if st["S"].get(bf) != (uid, j, qt) or st["lse"].get(s) != (uid, qt):
                            raise Hazard(f"sums {w}.{q} ({uid},{j},{qt}) read {st['S'].get(bf)}, {st['lse'].get(s)}")
                        yield
                    st["busy"][bf] -= 1
                    sim.bars[f"s_free{bf}"].arrive((uid, j, qt))
                    cnt += 1
                if many:
                    depth = 1 if mistake == "one_x" else 4
                    xs = x_it % depth
                    if w == 1:
                        if st["x"].get((xs, q), "read") != "read":
                            raise Hazard("a sum overwritten before it was read")
                        st["x"][(xs, q)] = (uid, j)
                        sim.bars[f"x_full{xs}"].arrive((uid, j))
                    else:
                        while not sim.ready(f"x_full{xs}", (x_it // depth) & 1, x_it // depth + 1):
                            yield
                        if st["x"].get((xs, q)) != (uid, j):
                            raise Hazard(f"sum of {(uid, j)} met {st['x'].get((xs, q))}")
                        st["x"][(xs, q)] = "read"
                    x_it += 1
                if not many or w == 0:
                    sim.out.append((uid, j, q))
                yield
            for qt in range(nq):
                s = (g + qt) % qbufs
                st["lse_read"][s] += 1
                sim.bars[f"q_empty{s}"].arrive()
                yield
            g += nq

    def execute(op, arg):
        if op == "commit":
            sim.bars[arg].arrive()
        elif op == "read":
            st["read"][arg] = True
        elif op == "q_read":
            st["q_read"][arg] = True
        else:
            uid, j, qt, s, qs, bf = arg
            if smem.get(f"k{s}") != (uid, j) or smem.get(f"q{qs}") != (uid, qt):
                raise Hazard(f"S ({uid},{j},{qt}) read K {smem.get(f'k{s}')}, Q {smem.get(f'q{qs}')}")
            if st["busy"].get(bf):
                raise Hazard(f"S ({uid},{j},{qt}) overwrote scores being read")
            st["S"][bf] = (uid, j, qt)

    sim.run([keys(), queries(), mma()] + [sums(w, q) for w in (0, 1) for q in range(warps)], execute, smem)
    want = sorted((i, j, q) for i, (tiles, _) in enumerate(pieces) for j in range(tiles) for q in range(warps))
    if sorted(sim.out) != want:
        raise Hazard(f"sums {sorted(sim.out)}, expected {want}")


def random_pieces(rnd, many, qbufs):
    return [(rnd.randint(1, 6), rnd.randint(1, qbufs) if many else 1) for _ in range(rnd.randint(0, 6))]


@pytest.mark.parametrize("warps", [1, 4])
@pytest.mark.parametrize("many,stages,qbufs", [(False, 4, 2), (False, 2, 1), (True, 2, 2), (True, 5, 4), (True, 2, 1)])
def test_weights_are_hazard_and_deadlock_free(many, stages, qbufs, warps):
    for seed in range(150 if warps == 1 else 60):
        run_weights(random_pieces(random.Random(seed * 13 + 1), many, qbufs), seed, many, stages, qbufs, warps=warps)


@pytest.mark.parametrize("many,mistake", [(False, "no_q_wait"), (True, "no_q_wait"), (False, "no_s_wait"),
                                          (True, "no_s_wait"), (True, "one_x")])
def test_weights_planted_mistakes(many, mistake):
    for seed in range(400):
        try:
            run_weights(random_pieces(random.Random(seed * 13 + 1), many, 2), seed, many, 4, 2, mistake)
        except Hazard:
            return
    raise AssertionError("not caught")
