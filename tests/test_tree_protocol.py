"""Model of the barrier protocol of the attention over the paged cache
(csrc/tree.cu), run on random pieces and random timings, with the machinery and
the mbarrier semantics of tests/test_fwd_protocol.py: the two loading warps (one
for the pieces, Q and K, one for V, into one ring of stages in the order the
tensor core reads them), the MMA issuer, and two warpgroups of softmax and
epilogue warps.

Layouts modelled:

- alternate: one row tile, two streams that take alternate key tiles, each with
  its own S/P and O; both warpgroups exchange their statistics at the end and
  store half of the columns each, over both O (d <= 128).
- one: one row tile, one stream over two S buffers and one O; the second
  warpgroup only stores (d > 128).
- sep (alternate-sep and pair-sep, d = 64; one-sep, d > 128): P in TMEM columns of its own, so that a
  stream's next scores are issued without waiting for its last PV; the softmax
  waits for that PV before it writes the next P.
- few (few-sep, d = 64): up to 32 rows in all four lane quarters, whose warps hand over P at once
  and add up their O in shared memory.
- pair: two row tiles that share every key tile, one stream each (d <= 128,
  more than 128 rows); the second may have no rows.

Key tiles that reach past the context have their V mended in shared memory by
one warpgroup before its P is handed over; no PV may read such a tile before
every warp of it is done.
"""
import random

import pytest

from test_fwd_protocol import Hazard, Sim


def fifo_k(pair, j):
    return 2 * j if pair else (0 if j == 0 else 2 * j - 1)


def fifo_v(pair, j, n):
    return 2 * j + 1 if pair else (2 * j + 2 if j < n - 1 else 2 * n - 1)


def run_pieces(layout, pieces, seed, stages, mistake=None, warps=1):
    """pieces: list of (n key tiles, row tiles, first ragged tile)."""
    sep = layout.endswith("-sep")
    layout = layout.replace("-sep", "")
    few = layout == "few"
    pair, streams = layout == "pair", 1 if layout == "one" else 2
    sim = Sim(pieces, seed, consumers=2 + 2 * warps)
    for b in (0, 1):
        for name in ("s_full", "o_done"):
            sim.bar(f"{name}{b}")
        for name in ("p_full", "p_hi"):
            sim.bar(f"{name}{b}", warps)
        sim.bar(f"o_free{b}", warps if pair else 2 * warps)
    sim.bar("stat_full", 2 * warps)
    for w in (0, 1):
        sim.bar(f"x_full{w}", warps)
    for name in ("q_full", "q_empty"):
        sim.bar(name)
    for s in range(stages):
        sim.bar(f"full{s}")
        sim.bar(f"empty{s}")
    smem = {}
    st = {"S": {}, "P": {}, "O": {0: [], 1: []}, "read": {}, "q_read": True, "mended": {},
          "stat": {}, "x": {}, "x_read": {}}

    def load(tag, f):
        s = f % stages
        if mistake != "no_empty_wait":
            while not sim.ready(f"empty{s}", ((f // stages) & 1) ^ 1, f // stages):
                yield
        if st["read"].get(s) is False:
            raise Hazard(f"stage {s} reloaded before it was read")
        st["read"][s] = False
        st["mended"][s] = set()
        sim.load(f"full{s}", f"kv{s}", tag)
        yield

    def keys():
        it = f = 0
        while True:
            piece = yield from sim.grab(it)
            if piece is None:
                return
            uid, n, _, _ = piece

            def load_q():
                if mistake != "no_q_empty_wait":
                    while not sim.ready("q_empty", (it & 1) ^ 1, it):
                        yield
                if not st["q_read"]:
                    raise Hazard("Q loaded over a Q still read")
                st["q_read"] = False
                sim.load("q_full", "q", uid)
                yield

            if it == 0:
                yield from load_q()
            for j in range(n):
                yield from load(("k", uid, j), f + fifo_k(pair, j))
                if j == 0 and it > 0:
                    yield from load_q()
            f += 2 * n
            it += 1

    def values():
        it = f = 0
        while True:
            piece = yield from sim.take(it)
            if piece is None:
                return
            uid, n, _, _ = piece
            for j in range(n):
                yield from load(("v", uid, j), f + fifo_v(pair, j, n))
            f += 2 * n
            it += 1

    def mma():
        it = f = 0
        cnt, done = [0, 0], [0, 0]
        while True:
            piece = yield from sim.take(it)
            if piece is None:
                return
            uid, n, ns, _ = piece
            while not sim.ready("q_full", it & 1, it + 1):
                yield

            def stage(no):
                while not sim.ready(f"full{no % stages}", (no // stages) & 1, no // stages + 1):
                    yield

            def there(no):  # a look, without waiting
                return sim.ready(f"full{no % stages}", (no // stages) & 1, no // stages + 1)

            def pv(no, buf, o, c, j, first):
                sim.pipe.append(("PV", (uid, buf, o, j, no % stages, 0, first)))
                if mistake != "no_p_hi_wait" and not few:
                    while not sim.ready(f"p_hi{buf}", c & 1, c + 1):
                        yield
                sim.pipe.append(("PV", (uid, buf, o, j, no % stages, 1, False)))

            if pair:
                for j in range(-1, n):
                    fv, fk = f + 2 * j + 1, f + 2 * j + 2
                    v_in, k_in = j >= 0 and there(fv), j + 1 < n and there(fk)
                    order = list(range(ns)) if mistake != "pair_order" else list(reversed(range(ns)))
                    for s in order:
                        if j >= 0:
                            while not sim.ready(f"p_full{s}", cnt[s] & 1, cnt[s] + 1):
                                yield
                            if s == order[0] and not v_in:
                                yield from stage(fv)
                            if j == 0 and done[s] > 0:
                                while not sim.ready(f"o_free{s}", (done[s] - 1) & 1, done[s]):
                                    yield
                            yield from pv(fv, s, s, cnt[s], j, j == 0)
                            if s == order[-1]:
                                sim.pipe.append(("read", fv % stages))
                                sim.pipe.append(("commit", f"empty{fv % stages}"))
                            sim.pipe.append(("commit", f"o_done{s}"))
                            cnt[s] += 1
                        if j + 1 < n:
                            if s == order[0] and not k_in:
                                yield from stage(fk)
                            if cnt[s] > 0 and not sep:
                                while not sim.ready(f"o_done{s}", (cnt[s] - 1) & 1, cnt[s]):
                                    yield
                            sim.pipe.append(("S", (uid, s, j + 1, fk % stages)))
                            sim.pipe.append(("commit", f"s_full{s}"))
                            if s == order[-1]:
                                sim.pipe.append(("read", fk % stages))
                                sim.pipe.append(("commit", f"empty{fk % stages}"))
                                if j + 1 == n - 1:
                                    sim.pipe.append(("commit", "q_empty"))
                        yield
                for s in range(ns):
                    done[s] += 1
            else:
                def do_s(j, k_in=False):
                    fk, b = f + fifo_k(False, j), j & 1
                    if not k_in:
                        yield from stage(fk)
                    c = cnt[b] + (j >> 1)
                    if c > 0 and not sep and mistake != "no_s_wait":
                        while not sim.ready(f"o_done{b}", (c - 1) & 1, c):
                            yield
                    sim.pipe.append(("S", (uid, b, j, fk % stages)))
                    sim.pipe.append(("read", fk % stages))
                    sim.pipe.append(("commit", f"empty{fk % stages}"))
                    sim.pipe.append(("commit", f"s_full{b}"))
                    if j == n - 1:
                        sim.pipe.append(("commit", "q_empty"))

                yield from do_s(0)
                if n > 1:
                    yield from do_s(1)
                for j in range(n):
                    fv, b = f + fifo_v(False, j, n), j & 1
                    c = cnt[b] + (j >> 1)
                    v_in = there(fv)
                    k_in = j + 2 < n and (mistake == "no_k_wait" or there(f + fifo_k(False, j + 2)))
                    while not sim.ready(f"p_full{b}", c & 1, c + 1):
                        yield
                    if not v_in:
                        yield from stage(fv)
                    if j == 0 and it > 0 and mistake != "no_o_free_wait":
                        while not sim.ready("o_free0", (it - 1) & 1, it):
                            yield
                    yield from pv(fv, b, b if streams == 2 else 0, c, j,
                                  j < 2 if streams == 2 else j == 0)
                    sim.pipe.append(("read", fv % stages))
                    sim.pipe.append(("commit", f"empty{fv % stages}"))
                    sim.pipe.append(("commit", f"o_done{b}"))
                    if j + 2 < n:
                        yield from do_s(j + 2, k_in)
                cnt[0] += (n + 1) // 2
                cnt[1] += n // 2
            f += 2 * n
            it += 1

    def tiles_of(w, n, ns):
        if pair:
            return list(range(n)) if w < ns else []
        if streams == 1:
            return list(range(n)) if w == 0 else []
        return list(range(w, n, 2))

    def softmax(w, q):
        it = f = 0
        cnt = [0, 0]
        while True:
            piece = yield from sim.take(it)
            if piece is None:
                return
            uid, n, ns, ragged = piece
            mine = tiles_of(w, n, ns)
            seen = []
            for j in mine:
                b = w if pair else j & 1
                c = cnt[w] + j if pair else cnt[b] + (j >> 1)
                while not sim.ready(f"s_full{b}", c & 1, c + 1):
                    yield
                if j >= ragged and (not pair or w == 0) and mistake != "no_mend":
                    fv = f + fifo_v(pair, j, n)
                    if mistake != "no_mend_wait":
                        while not sim.ready(f"full{fv % stages}", (fv // stages) & 1,
                                            fv // stages + 1):
                            yield
                    if smem.get(f"kv{fv % stages}") != ("v", uid, j):
                        raise Hazard(f"mending ({uid},{j}) found {smem.get(f'kv{fv % stages}')}")
                    yield
                    st["mended"][fv % stages].add(q)
                if st["S"].get(b) != (uid, j):
                    raise Hazard(f"softmax {w}.{q} ({uid},{j}) read S = {st['S'].get(b)}")
                yield
                if st["S"].get(b) != (uid, j):
                    raise Hazard("S overwritten while the softmax read it")
                if sep and c > 0 and mistake != "no_p_free_wait":
                    while not sim.ready(f"o_done{b}", (c - 1) & 1, c):
                        yield
                if seen and sim.rnd.random() < 0.3:  # rescale O
                    o = w if pair else (b if streams == 2 else 0)
                    if streams == 1 and mistake != "no_rescale_wait":
                        pb = (j - 1) & 1
                        cc = cnt[pb] + ((j - 1) >> 1)
                        while not sim.ready(f"o_done{pb}", cc & 1, cc + 1):
                            yield
                    if st["O"][o] != [(uid, x, h) for x in seen for h in (0, 1)]:
                        raise Hazard(f"rescale of ({uid},{j}) saw O = {st['O'][o]}")
                for hf, bar in ((0, None), (1, "p_full")) if few else ((0, "p_full"), (1, "p_hi")):
                    yield
                    if st["S"].get(b) != (uid, j):
                        raise Hazard("S overwritten while the softmax read it")
                    if sep and st["P"].get((b, hf), {}).get(q, "read") != "read":
                        raise Hazard(f"P of ({uid},{j}) written over one not yet read")
                    st["P"].setdefault((b, hf), {})[q] = (uid, j)
                    if bar:
                        sim.bars[f"{bar}{b}"].arrive((uid, j))
                seen.append(j)
                yield
            # epilogue
            if pair:
                if w < ns:
                    while not sim.ready(f"o_done{w}", (cnt[w] + n - 1) & 1, cnt[w] + n):
                        yield
                    cnt[w] += n
                    reads = [(w, mine)]
                else:
                    reads = []
            else:
                slot = it & 1 if mistake != "one_stat_buffer" else 0
                if w < streams:
                    st["stat"][(slot, w, q)] = uid
                sim.bars["stat_full"].arrive(uid)
                while mistake != "no_stat_wait" and not sim.ready("stat_full", it & 1, it + 1):
                    yield
                yield
                for x in range(streams):
                    if st["stat"].get((slot, x, q)) != uid:
                        raise Hazard(f"statistics of {uid}: {st['stat'].get((slot, x, q))}")
                n0, n1 = (n + 1) // 2, n // 2
                while not sim.ready("o_done0", (cnt[0] + n0 - 1) & 1, cnt[0] + n0):
                    yield
                if n > 1:
                    while not sim.ready("o_done1", (cnt[1] + n1 - 1) & 1, cnt[1] + n1):
                        yield
                cnt[0] += n0
                cnt[1] += n1
                reads = [(x, tiles_of(x, n, ns)) for x in range(streams)]
            for _ in range(2):
                for o, tiles in reads:
                    if tiles and st["O"][o] != [(uid, x, h) for x in tiles for h in (0, 1)]:
                        raise Hazard(f"epilogue {w}.{q} of {uid} read O_{o} = {st['O'][o]}")
                yield
            if few:
                if len(st["x_read"].get((w, q), range(warps))) != warps:
                    raise Hazard(f"O of {uid} written over a quarter that is not read")
                st["x"][(w, q)], st["x_read"][(w, q)] = uid, set()
                sim.bars[f"x_full{w}"].arrive(uid)
                if mistake != "no_x_full_wait":
                    while not sim.ready(f"x_full{w}", it & 1, it + 1):
                        yield
                yield
                for k in range(warps):
                    if st["x"].get((w, k)) != uid:
                        raise Hazard(f"{uid} added up {st['x'].get((w, k))}")
                    yield
                    st["x_read"][(w, k)].add(q)
            if reads:
                if q == 0:
                    sim.out.append((uid, w))
                sim.bars[f"o_free{w if pair else 0}"].arrive(uid)
            f += 2 * n
            it += 1

    def execute(op, arg):
        if op == "commit":
            if arg == "q_empty":
                st["q_read"] = True
            sim.bars[arg].arrive()
        elif op == "read":
            st["read"][arg] = True
        elif op == "S":
            uid, b, j, s = arg
            if smem.get("q") != uid or smem.get(f"kv{s}") != ("k", uid, j):
                raise Hazard(f"S ({uid},{j}) read Q {smem.get('q')}, K {smem.get(f'kv{s}')}")
            for hf in (0, 1):
                if sep:
                    continue
                if any(v != "read" for v in st["P"].get((b, hf), {}).values()):
                    raise Hazard(f"S ({uid},{j}) overwrote P before PV read it")
                st["P"][(b, hf)] = {}
            st["S"][b] = (uid, j)
        elif op == "PV":
            uid, b, o, j, s, hf, first = arg
            quarters = st["P"].get((b, hf), {})
            if smem.get(f"kv{s}") != ("v", uid, j) or len(quarters) != warps or any(
                    v != (uid, j) for v in quarters.values()):
                raise Hazard(f"PV ({uid},{j}) half {hf} read {smem.get(f'kv{s}')}, P {quarters}")
            if j >= pieces[uid][2] and len(st["mended"].get(s, ())) != warps:
                raise Hazard(f"PV ({uid},{j}) read a V that is not mended")
            if first:
                st["O"][o] = []
            st["O"][o].append((uid, j, hf))
            st["P"][(b, hf)] = {x: "read" for x in quarters}

    roles = [keys(), values(), mma()] + [softmax(w, q) for w in (0, 1) for q in range(warps)]
    sim.run(roles, execute, smem)
    want = [(u, w) for u, (n, ns, _) in enumerate(pieces) for w in (0, 1)
            if not pair or w < ns]
    if sorted(sim.out) != sorted(want):
        raise Hazard(f"stored {sorted(sim.out)}, expected {want}")


def random_pieces(rnd, layout):
    pieces = []
    for _ in range(rnd.randint(0, 7)):
        n = rnd.choice([1, 1, 2, 2, 3, 4, 5, 8])
        pieces.append((n, rnd.choice([1, 2, 2]) if layout.startswith("pair") else 1,
                       rnd.choice([0, n - 1, n, max(0, n - 2)])))
    return pieces


LAYOUTS = [("alternate", 5), ("alternate", 8), ("one", 4), ("one", 7), ("pair", 4), ("pair", 8),
           ("alternate-sep", 8), ("pair-sep", 8), ("one-sep", 4), ("one-sep", 7),
           ("few-sep", 5), ("few-sep", 8)]


@pytest.mark.parametrize("warps", [1, 4])
@pytest.mark.parametrize("layout,stages", LAYOUTS)
def test_protocol_is_hazard_and_deadlock_free(layout, stages, warps):
    for seed in range(150 if warps == 1 else 60):
        run_pieces(layout, random_pieces(random.Random(seed * 5 + 1), layout), seed, stages,
                   warps=warps)


# True: the model must catch it; False: another wait implies it (in an in-order
# tensor pipe S runs after the PVs issued before it, so that the P it overwrites,
# or the P before the one it leads to, has been read; the kernel does not rely on
# that order).
MISTAKES = [
    ("alternate", 5, "no_empty_wait", True), ("alternate", 5, "no_q_empty_wait", True),
    ("alternate", 5, "no_p_hi_wait", True), ("alternate", 5, "no_o_free_wait", True),
    ("alternate", 5, "no_s_wait", False), ("alternate", 5, "no_mend", True),
    ("alternate", 5, "no_mend_wait", True), ("alternate", 5, "one_stat_buffer", True),
    ("alternate", 5, "no_k_wait", True),
    ("one", 4, "no_rescale_wait", True), ("one", 4, "no_o_free_wait", True),
    ("alternate-sep", 8, "no_p_free_wait", False), ("pair-sep", 8, "no_p_free_wait", False),
    ("one-sep", 4, "no_p_free_wait", False), ("one-sep", 4, "no_rescale_wait", True),
    ("alternate-sep", 8, "no_p_hi_wait", True),
    ("few-sep", 8, "no_x_full_wait", True), ("few-sep", 8, "no_stat_wait", True),
    ("few-sep", 5, "no_q_empty_wait", True), ("few-sep", 8, "no_mend_wait", True),
    ("few-sep", 8, "no_p_free_wait", False),
    ("pair", 4, "pair_order", True), ("pair", 4, "no_empty_wait", True),
]


@pytest.mark.parametrize("layout,stages,mistake,caught", MISTAKES)
def test_planted_mistakes(layout, stages, mistake, caught):
    for seed in range(400):
        try:
            run_pieces(layout, random_pieces(random.Random(seed * 5 + 1), layout), seed, stages,
                       mistake, warps=2)
        except Hazard:
            assert caught, "a wait thought to be implied by others is needed"
            return
    assert not caught
