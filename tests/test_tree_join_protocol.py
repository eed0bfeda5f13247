"""Model of how the CTAs of the attention over the paged cache (csrc/tree.cu) share items and join
their partials when an item has few rows, run on random lines of key tiles and random timings.

A CTA takes an equal stretch of the line.  A piece of an item that it shares with others leaves a
partial; the CTA then brings it: it counts in the item's word (that of the item's last CTA) under
the call's number, anything else in the word counting as none, and whoever brings the last one
clears the word and joins the partials at the CTA's end.  A first piece whose item began elsewhere is
brought by an idle warp as soon as it is stored (barriers `begun` and `stored`), the others at the
CTA's end.  What a step of the model does is atomic; the steps of all CTAs and warps interleave at
random, so it shows what orders allow, not what a missing fence would.
"""
import random

import pytest

MISTAKES = ("no_stored_wait", "no_clear", "early_brought_twice", "early_never_brought", "stale_count_kept",
            "own_word", "join_at_once")


class Hazard(Exception):
    pass


def pieces(items, ctas, min_tiles=2):
    """What the producer warp computes: per CTA (item, k0, n, first CTA, last CTA, whole)."""
    total = sum(items)
    per = max(-(-total // ctas), min_tiles)
    out = []
    for c in range(ctas):
        at, end = min(total, per * c), min(total, per * (c + 1))
        mine, item, before = [], 0, 0
        while at < end:
            while before + items[item] <= at:
                before += items[item]
                item += 1
            k0 = at - before
            n = min(items[item] - k0, end - at)
            ends = k0 + n == items[item]
            first = (at - k0) // per if k0 > 0 else c
            last = (at - k0 + items[item] - 1) // per if not ends else c
            mine.append((item, k0, n, first, last, k0 == 0 and ends))
            at += n
        out.append(mine)
    return out


def run_call(items, ctas, words, call, rnd, mistake=None):
    """One call on a workspace whose words hold anything; returns how often each item was joined."""
    work = pieces(items, ctas)
    stored, joined = set(), {}
    share = {}  # item -> CTAs, from the pieces themselves
    for c, mine in enumerate(work):
        for item, *_, whole in mine:
            if not whole:
                share.setdefault(item, []).append(c)

    def bring(c, piece):
        """The steps of one thread; returns whether it brought the last partial."""
        item, _, _, first, last, _ = piece
        word = c if mistake == "own_word" else last
        old = 0
        while True:
            yield
            mine = old >> 8 == call or mistake == "stale_count_kept"
            now = old + 1 if mine else (call << 8) + 1
            if words[word] == old:
                words[word] = now
                break
            old = words[word]
        if now & 255 != last - first + 1:
            return False
        yield
        if mistake != "no_clear":
            words[word] = 0
        return True

    def join(c, piece):
        item, _, _, first, last, _ = piece
        assert share[item] == list(range(first, last + 1)), "CTAs disagree on who shares an item"
        for other in range(first, last + 1):
            yield
            if (item, other) not in stored:
                raise Hazard(f"item {item} joined before CTA {other} stored its partial")
        joined[item] = joined.get(item, 0) + 1

    def cta(c):
        mine = work[c]
        shared = [p for p in mine if not p[5]]
        if len(shared) > 2:
            raise Hazard("more than two shared pieces")
        early = bool(mine) and mine[0][1] > 0
        state = {"begun": False, "first_stored": False, "main": False, "idle": False, "last": [False] * 2}

        def main():
            yield
            state["begun"] = True
            for i, p in enumerate(mine):
                for _ in range(rnd.randint(0, 3)):
                    yield
                if not p[5]:
                    stored.add((p[0], c))
                yield
                if i == 0:
                    state["first_stored"] = True
            state["main"] = True

        def idle():
            while not state["begun"]:
                yield
            if early and mistake != "early_never_brought":
                while not state["first_stored"] and mistake != "no_stored_wait":
                    yield
                state["last"][0] = yield from bring(c, shared[0])
                if mistake == "join_at_once" and not state["last"][0]:
                    yield from join(c, shared[0])
            state["idle"] = True

        def end():
            while not (state["main"] and state["idle"]):
                yield
            start = 0 if mistake == "early_brought_twice" else int(early)
            for i in range(start, len(shared)):
                state["last"][i] = yield from bring(c, shared[i])
            for i, p in enumerate(shared):
                if state["last"][i]:
                    yield from join(c, p)

        return [main(), idle(), end()]

    live = [t for c in range(ctas) for t in cta(c)]
    while live:
        # (a random few at a time, so that some threads stay far behind)
        t = live[rnd.randrange(min(len(live), rnd.choice([1, 3, len(live)])))]
        try:
            next(t)
        except StopIteration:
            live.remove(t)
        if rnd.random() < 0.05:
            rnd.shuffle(live)
    if set(joined) != set(share) or any(n != 1 for n in joined.values()):
        raise Hazard(f"joined {joined}, shared {sorted(share)}")


def run(seed, mistake=None, ctas=None):
    rnd = random.Random(seed)
    ctas = ctas or rnd.choice([2, 3, 8, 20])
    call = rnd.getrandbits(56)
    # what a workspace may hold: zeros, anything, another call's counts
    words = [rnd.choice([0, rnd.getrandbits(64), (rnd.getrandbits(56) << 8) + 1]) for _ in range(ctas)]
    for _ in range(3):  # replays of one captured call, whose lengths change in between
        items = [rnd.choice([1, 1, 2, 3, 7, 20, 60]) for _ in range(rnd.randint(1, 12))]
        run_call(items, ctas, words, call, rnd, mistake)
    # another call on the same workspace
    run_call([rnd.randint(1, 30) for _ in range(5)], ctas, words, rnd.getrandbits(56), rnd, mistake)


@pytest.mark.parametrize("block", range(4))
def test_every_shared_item_is_joined_once(block):
    for seed in range(block * 100, block * 100 + 100):
        run(seed)


def test_as_many_ctas_as_the_gpu_runs():
    for seed in range(5):
        run(seed, ctas=152)


@pytest.mark.parametrize("mistake", MISTAKES)
def test_a_mistake_is_found(mistake):
    found = 0
    for seed in range(60):
        try:
            run(seed, mistake)
        except (Hazard, AssertionError):
            found += 1
    assert found > 0
