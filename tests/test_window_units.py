"""The windowed attention's own geometry (csrc/window.cuh, csrc/fwd.cu) and unit lists (csrc/sched.cu), compiled for
the host and run there, against the mask itself: every visible pair is worked on exactly once, a
deterministic dQ tile takes its contributions in the order of the list, units without rows are not
listed, and the sinks' partials lie apart, within what the workspace has for them."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from test_window_schedule import cases, cdiv, visible

HERE = os.path.dirname(os.path.abspath(__file__))
T = 128


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("emulated") / "window.so")
    src = os.path.join(HERE, "cta_emulator")
    fwd = open(os.path.join(HERE, "..", "bwd_tiled_attention_gb300", "csrc", "fwd.cu")).read()
    first = fwd.index("struct UnitGeom {")
    last = fwd.index("\n}\n", fwd.index("UnitGeom decode_unit(int2 u", first)) + 3
    inc = tmp_path_factory.mktemp("source")
    (inc / "fwd_units.inc").write_text(fwd[first:last])
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I" + src,
                    "-I" + str(inc), os.path.join(src, "window.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.near_place_of.restype = L.far_place_of.restype = ctypes.c_longlong
    L.order_threads.argtypes = [ctypes.c_int, ctypes.c_ulonglong]
    return L


def ptr(x):
    return None if x is None else x.ctypes.data_as(ctypes.c_void_p)


def ends(x):
    return np.cumsum([0] + list(x)).astype(np.int32)


@pytest.mark.parametrize("Lq,Lk,W,S", cases())
@pytest.mark.parametrize("qtiles", [1, 2])
def test_forward_walks(lib, Lq, Lk, W, S, qtiles):
    see = visible(Lq, Lk, W, S)
    n, steps, parts, own = (np.zeros(x, np.int32) for x in (3, 4096, 4096, 8192))
    for m in range(cdiv(Lq, T * qtiles)):
        lib.walk(m, qtiles, Lq, Lk, W, S, ptr(n), ptr(steps), ptr(parts), ptr(own))
        assert 1 <= n[2] < 4096
        for t in range(2):
            rows = see[(m * qtiles + t) * T:(m * qtiles + t + 1) * T] if t < qtiles else see[:0]
            want = {c // T for c in np.flatnonzero(rows.any(0))}
            mine = own[t * 4096:t * 4096 + n[t]].tolist()
            assert mine == [k for k, p in zip(steps[:n[2]].tolist(), parts) if p >> t & 1]
            assert sorted(set(mine)) == mine and want <= set(mine)
            if Lk >= Lq and rows.shape[0] == T:
                assert set(mine) == want


class Batch:
    """A batch, its unit list as the scheduler writes it, and the layout of its workspace."""

    def __init__(self, lib, lq, lk, W, S, H=2, det=True, dense=False, slack=0):
        self.lib, self.lq, self.lk, self.W, self.S, self.H = lib, lq, lk, W, S, H
        self.cu, self.cu_k = ends(lq), ends(lk)
        B, Tq, Tk, d = len(lq), sum(lq), sum(lk), 64
        lay = np.zeros(9, np.int64)
        lib.far_layout(B, H, H, Tq, Tk, d, W, S, ptr(lay))
        self.chunk, self.sink_tiles, self.most_far, self.near, self.rows = lay[:5].tolist()
        self.room = (lay[6] - lay[5]) // (2 * H * d * 4)  # rows that the workspace holds
        ws = np.full(int(lay[7]) // 4 + 4, 0x5a5a5a5a, np.int32)
        units, self.tile_off = np.zeros((int(lay[8]), 2), np.int32), np.zeros(B + 1, np.int32)
        n = lib.schedule(None if dense else ptr(self.cu), max(lq) + slack, Tq, None if dense else ptr(self.cu_k),
                         max(lk) + slack, Tk, B, H, d, int(det), W, S, ptr(ws), ptr(units), ptr(self.tile_off))
        assert n >= 0 and (ws[int(lay[7]) // 4:] == 0x5a5a5a5a).all()
        out = np.zeros(4, np.int32)
        self.units = []
        for x, y in units[:n].tolist():
            lib.unit(x, y, max(1, self.sink_tiles), ptr(out))
            self.units.append(tuple(out.tolist()))   # sequence, tile, 1 + chunk or 0, head

    def tiles(self, b, j, far):
        out = np.zeros(2, np.int32)
        self.lib.span(j, far, self.chunk, self.lq[b], self.lk[b], self.W, self.S, ptr(out))
        return range(out[0], out[0] + out[1])


def batches():
    rnd = random.Random(11)
    some = [(([640], [640]), 129, 128), (([5000], [5000]), 40, 260), (([300, 1, 0, 700], [300, 513, 40, 200]), 50, 10),
            (([2600, 130, 129], [2600, 900, 129]), 128, 4), (([64, 4300], [64, 4300]), 100, 300),
            (([20] * 30 + [3000], [20] * 30 + [3000]), 64, 500), (([0, 0, 5], [9, 0, 700]), 8, 3),
            (([200] * 3, [2500] * 3), 1000, 200)]
    # more sequences than the scheduler has threads
    some += [(([3] * 1500 + [400] + [130] * 40,) * 2, 100, 5), (([1, 200] * 1040 + [900],) * 2, 129, 140)]
    for _ in range(12):
        n = rnd.randint(1, 6)
        lk = [rnd.choice([0, 1, rnd.randint(1, 3000)]) for _ in range(n - 1)] + [rnd.randint(300, 3000)]
        lq = [max(0, x - rnd.choice([0, 0, rnd.randint(0, x)])) + rnd.choice([0, 0, 0, 50]) for x in lk]
        some.append(((lq, lk), rnd.choice([1, 30, 128, 250]), rnd.choice([1, 4, 128, 129, 270])))
    return some


@pytest.mark.parametrize("lens,W,S", batches())
@pytest.mark.parametrize("order", [(0, 0), (1, 0), (2, 5)])
def test_every_pair_once_and_in_order(lib, lens, W, S, order):
    lib.order_threads(*order)
    batch = Batch(lib, *lens, W, S, slack=7)
    lo, hi = np.zeros(T, np.int32), np.zeros(T, np.int32)
    got = [np.zeros((cdiv(a, T) * T, cdiv(b, T) * T), np.int32) for a, b in zip(*lens)]
    ranks = {}
    near = set()
    for b, j, far, h in batch.units:
        L, Lk = batch.lq[b], batch.lk[b]
        tiles = batch.tiles(b, j, far)
        if far:
            assert len(tiles)                    # (listed for its rows)
        else:
            near.add((b, j, h))
        for i in tiles:
            assert not far or i // batch.chunk == far - 1
            ranks.setdefault((b, i, h), []).append(lib.rank_of(j, far, i, L, Lk, W, S))
            if h == 0:
                lib.cols(j, far, i, L, Lk, W, S, ptr(lo), ptr(hi))
                for c in range(T):
                    got[b][i * T + lo[c]:i * T + max(lo[c], hi[c]), j * T + c] += 1
    assert len(set(batch.units)) == len(batch.units)
    assert near == {(b, j, h) for b, n in enumerate(batch.lk) for j in range(cdiv(n, T)) for h in range(batch.H)}
    for b, (L, Lk) in enumerate(zip(*lens)):
        assert np.array_equal(got[b][:L, :Lk], visible(L, Lk, W, S).astype(np.int32))
        assert not got[b][L:].any() and not got[b][:, Lk:].any()
    for x in ranks.values():
        assert x == list(range(len(x)))


@pytest.mark.parametrize("lq,lk,W,S", [(640, 640, 100, 4), (5000, 5000, 300, 300), (130, 900, 128, 1), (3000, 2000, 64, 0),
                                       (20, 700, 600, 500)])
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("det", [False, True])
def test_dense_lists_are_the_packed_ones(lib, lq, lk, W, S, B, det):
    lib.order_threads(0, 0)
    a = Batch(lib, [lq] * B, [lk] * B, W, S, det=det, dense=True)
    b = Batch(lib, [lq] * B, [lk] * B, W, S, det=det)
    assert a.units == b.units and np.array_equal(a.tile_off, b.tile_off)


def places(batch):
    """[first, end) rows of partials that units write and the fold reads, of each sequence and kind."""
    out = []
    for b, (L, Lk) in enumerate(zip(batch.lq, batch.lk)):
        t0, tk0 = int(batch.cu[b]), int(batch.cu_k[b])
        R = batch.lib.far_rows_of(Lk, batch.W, batch.S)
        if R == 0:
            continue
        at = batch.lib.near_place_of(b, tk0, batch.W, batch.S)
        out.append((at, at + R))
        assert at + R <= batch.near
        at = batch.near + batch.lib.far_place_of(b, t0, tk0, batch.chunk, batch.W, batch.S)
        out += [(at + q * R, at + (q + 1) * R) for q in range(cdiv(cdiv(L, T), batch.chunk))]
    return out


@pytest.mark.parametrize("seed", range(40))
def test_partials_lie_apart_and_within_the_workspace(lib, seed):
    rnd = random.Random(seed)
    n = rnd.choice([1, 3, 40, 300])
    top = rnd.choice([30, 300, 5000])
    lk = [rnd.choice([0, 1, rnd.randint(1, top), top]) for _ in range(n)]
    lq = [rnd.choice([x, x, rnd.randint(0, x), x + rnd.randint(0, 200)]) for x in lk]
    W = rnd.choice([1, 7, 64, 128, 1000])
    S = rnd.choice([1, 4, 128, 500, 2100])
    batch = Batch.__new__(Batch)
    batch.lib, batch.lq, batch.lk, batch.W, batch.S = lib, lq, lk, W, S
    batch.cu, batch.cu_k = ends(lq), ends(lk)
    lay = np.zeros(9, np.int64)
    lib.far_layout(n, 2, 2, sum(lq), sum(lk), 64, W, S, ptr(lay))
    batch.chunk, batch.near, batch.rows = int(lay[0]), int(lay[3]), int(lay[4])
    end = 0
    for a, b in sorted(places(batch)):
        assert a >= end
        end = b
    assert end <= batch.rows <= sum(lq) + 2 * sum(lk)
    # far units fit the list
    units = sum(max(0, cdiv(cdiv(a, T), batch.chunk) - lib.far_first_of(j, batch.chunk, a, b, W, S))
                for a, b in zip(lq, lk) for j in range(cdiv(S, T)))
    assert units * 2 <= lay[2]


@pytest.mark.parametrize("lens,longest,W,S", [
    ([8] * 2000 + [20] * 2000 + [8192], 8192, 1024, 128), ([100] * 512 + [8192], 8192, 64, 1023),
    ([32768], 32768, 1024, 4), ([8192] * 4, 8192, 100, 8000)])
def test_workspace_goes_with_the_tokens(lens, longest, W, S):
    """Sequences times sinks do not count where they are more than the tokens are."""
    fabuild.build()
    B, Tk, hq, hkv, d = len(lens), sum(lens), 16, 8, 128
    plain = fa.fa_bwd_kv_workspace_size(B, hq, hkv, longest, Tk, longest, Tk, d)
    size = fa.fa_bwd_window_workspace_size(B, hq, hkv, longest, Tk, longest, Tk, d, W, S)
    rows = 2 * hkv * 2 * d * 4                     # of dK and dV in fp32, for two runs of heads
    assert plain < size <= plain + 3 * Tk * rows + 2 ** 22
    if len(lens) == 1:                             # and few sinks need little
        assert size - plain < Tk * rows // 50


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 1), (128, 2, 2), (256, 2, 1)])
@pytest.mark.parametrize("det", [False, True])
def test_sequences_with_and_without_far_rows(d, hq, hkv, det):
    """More sinks than most sequences have keys, queries behind earlier keys, empty sides."""
    from test_window import run
    fabuild.build()
    run([100] * 40 + [1500, 0, 5] + [70] * 9, [100] * 40 + [1500, 300, 900] + [70] * 9, hq, hkv, d, 64, 1023, det)
    run([3000, 40, 1, 2500], [3000, 40, 700, 4000], hq, hkv, d, 300, 130, det)
