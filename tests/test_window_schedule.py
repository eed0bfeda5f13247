"""The tiles and units of the windowed attention, restated in Python from csrc/fwd.cu, csrc/bwd.cu and
csrc/sched.cu and held against the mask itself: every visible pair is worked on exactly once, and a
deterministic dQ tile takes its contributions in an order that no unit list can stall."""
import itertools
import random

import numpy as np
import pytest

T = 128
FAR_CHUNK = 16


def cdiv(a, b):
    return -(-a // b)


def visible(Lq, Lk, W, S):
    p = np.arange(Lq)[:, None] + Lk - Lq
    c = np.arange(Lk)[None, :]
    return (c <= p) & ((p - c < W) | (c < S))


def cases():
    rnd = random.Random(7)
    fixed = [(1, 1, 1, 0), (1, 700, 1, 3), (300, 300, 1, 0), (300, 300, 1, 300), (640, 640, 128, 4),
             (640, 640, 129, 128), (640, 900, 127, 129), (700, 200, 50, 10), (5000, 5000, 40, 260),
             (2600, 2600, 300, 0), (129, 2000, 256, 500), (2049, 2049, 2048, 2048)]
    return fixed + [(rnd.randint(1, 1500), rnd.randint(1, 1500), rnd.choice([1, 5, 64, 128, 200, 700]),
                     rnd.choice([0, 1, 4, 127, 128, 129, 400])) for _ in range(40)]


# ------------------------------------------------------------------------------ forward


def forward_unit(m, Lq, Lk, W, S, qtiles):
    """Geometry of unit m: st, per query tile (n, lo, hi), first, nsink, nkv."""
    st, off = cdiv(S, T), Lk - Lq
    n, lo, hi = [0, 0], [0, 0], [0, 0]
    first, end = 1 << 31, 0
    for t in range(2):
        rs = (m * qtiles + t) * T
        if t < qtiles and rs < Lq:
            hi[t] = cdiv(max(min(rs + T, Lq) + off, 0), T)
        if hi[t] == 0:
            continue
        lo[t] = max(rs + off - W + 1, 0) // T
        n[t] = hi[t] - lo[t] + min(st, lo[t])
        first, end = min(first, lo[t]), max(end, hi[t])
    first = min(first, end)
    nsink = min(st, first)
    return st, n, lo, hi, first, nsink, max(end - first + nsink, 1)


@pytest.mark.parametrize("Lq,Lk,W,S", cases())
@pytest.mark.parametrize("qtiles", [1, 2])
def test_forward_tiles(Lq, Lk, W, S, qtiles):
    see = visible(Lq, Lk, W, S)
    for m in range(cdiv(Lq, T * qtiles)):
        st, n, lo, hi, first, nsink, nkv = forward_unit(m, Lq, Lk, W, S, qtiles)
        tile = lambda j: j if j < nsink else first + j - nsink  # noqa: E731
        for t in range(2):
            rows = see[(m * qtiles + t) * T:(m * qtiles + t + 1) * T] if t < qtiles else see[:0]
            want = {c // T for c in np.flatnonzero(rows.any(0))}
            walked = [tile(j) for j in range(nkv)
                      if tile(j) < hi[t] and (tile(j) >= lo[t] or tile(j) < st)]
            s = min(st, lo[t])
            own = [j if j < s else lo[t] + j - s for j in range(n[t])]
            assert walked == own            # the issuer's steps and the softmax warps' are the same
            assert sorted(set(own)) == own and want <= set(own)
            # no tile more than the mask of whole tiles has
            if Lk >= Lq and rows.shape[0] == T:
                assert set(own) == want


# ----------------------------------------------------------------------------- backward


class Unit:
    def __init__(self, j, far, Lq, Lk, W, S, chunk):
        self.j, self.far = j, far
        off, nt, c0 = Lk - Lq, cdiv(Lq, T), j * T
        if far == 0:
            i0 = max(0, (c0 - off) // T)
            i1 = min(nt, (min(c0 + T, Lk) - 2 + W - off) // T + 1)
        else:
            q = far - 1
            i0 = max(q * chunk, (c0 + W - off) // T)
            i1 = min(nt, (q + 1) * chunk)
            if c0 >= min(S, Lk) or c0 + W >= Lk:
                i1 = i0
        self.tiles = list(range(i0, max(i0, i1)))

    def cols(self, c, i, Lq, Lk, W, S):
        r = c - (Lk - Lq)
        lo = r + W if self.far else r
        if self.far:
            hi = Lq if c < min(S, Lk) else 0
        else:
            hi = min(Lq, r + W) if c < Lk else 0
        return max(0, lo - i * T), min(T, hi - i * T)

    def rank(self, i, Lq, Lk, W, S):
        off = Lk - Lq
        last = min((i + 1) * T, Lq) - 1 + off
        before = max(0, min(cdiv(min(S, Lk), T), (last - W) // T + 1))
        if self.far:
            return before - 1 - self.j
        return before + min(cdiv(Lk, T) - 1, ((i + 1) * T + off - 1) // T) - self.j


def units(Lq, Lk, W, S):
    """In the order of a deterministic call's list."""
    st = cdiv(S, T)
    chunk = max(FAR_CHUNK, st)
    far = [Unit(j, 1 + q, Lq, Lk, W, S, chunk) for j in reversed(range(st))
           for q in range(cdiv(cdiv(Lq, T), chunk))]
    return far + [Unit(j, 0, Lq, Lk, W, S, chunk) for j in reversed(range(cdiv(Lk, T)))]


@pytest.mark.parametrize("Lq,Lk,W,S", cases())
def test_backward_pairs(Lq, Lk, W, S):
    W, S = min(W, Lk), min(S, Lk)
    see = visible(Lq, Lk, W, S)
    got = np.zeros((cdiv(Lq, T) * T, cdiv(Lk, T) * T), np.int32)
    for u in units(Lq, Lk, W, S):
        for i in u.tiles:
            for c in range(u.j * T, (u.j + 1) * T):
                lo, hi = u.cols(c, i, Lq, Lk, W, S)
                got[i * T + lo:i * T + max(lo, hi), c] += 1
    assert np.array_equal(got[:Lq, :Lk], see.astype(np.int32))
    assert not got[Lq:].any() and not got[:, Lk:].any()


@pytest.mark.parametrize("Lq,Lk,W,S", cases())
def test_backward_order(Lq, Lk, W, S):
    """A dQ tile's contributions have ranks 0, 1, ..., in the order of the list: each waits only for
    units before it, which never wait for it."""
    W, S = min(W, Lk), min(S, Lk)
    ranks = {}
    for u in units(Lq, Lk, W, S):
        for i in u.tiles:
            ranks.setdefault(i, []).append(u.rank(i, Lq, Lk, W, S))
    for got in ranks.values():
        assert got == list(range(len(got)))


def test_sink_partials_do_not_overlap():
    """Slots of a sequence: tile_off / C + 2 b, one more than it has chunks; and there are enough."""
    rnd = random.Random(3)
    for chunk, B in itertools.product([16, 20], [1, 2, 9]):
        lens = [rnd.choice([0, 1, 128, 2048, 2049, rnd.randint(1, 30000)]) for _ in range(B)]
        off, end = 0, 0
        for b, n in enumerate(lens):
            first = off // chunk + 2 * b
            assert first >= end
            end = first + 1 + cdiv(cdiv(n, T), chunk)
            off += cdiv(n, T)
        assert end <= (cdiv(sum(lens), T) + B) // chunk + 2 * (B + 1)
