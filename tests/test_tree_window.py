"""Attention over the paged cache within a sliding window and a few first keys, against a 64-bit
implementation: single tokens, chunks and trees, all head layouts and page sizes, windows and sinks on
and off tile boundaries, what stands in hidden places, and what is refused.

The pages hold NaN wherever no token of the test stands."""
import ctypes
import random

import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import attend, f64, within
from test_cache import FAKE, desc, ints
from test_tree import HEADS, Held, queries, random_tree, words_of

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(layer=2), 1), (dict(q=None), 1),
    (dict(scale=0.0), 2), (dict(ws_bytes=1000), 1), (dict(mask=FAKE + 4, words=1), 1), (dict(qt=130), 1)])
def test_bad_calls_are_refused(kw, status):
    a = dict(layer=0, slots=FAKE, B=2, N=3, cu=None, T=6, q=FAKE, Hq=4, qt=256, qh=64, mask=None,
             words=0, o=FAKE, lse=FAKE, scale=0.125, window=5, sinks=1, zero=0, ws=FAKE, ws_bytes=1 << 30,
             stream=None)
    a.update(kw)
    assert fa.lib().fa_tree_fwd_window(ctypes.addressof(desc()), *a.values()) == status


def test_tensor_calls_refuse(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    cache = fa.PagedCache.allocate(1, 3, 2, 16, 64, 2, 2, device="cpu")
    q, slots = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(window=0), dict(window=-3), dict(window=2 ** 31), dict(window=1.5),
               dict(window=4, sinks=-1), dict(window=4, sinks=0.5), dict(sinks=4)):
        with pytest.raises(ValueError, match="window|sinks|whole"):
            fa.tree_attention(q, cache, 0, slots, **kw)


def visible(n, length, W, S, rows=None):
    """[n, length]: what the last n tokens see."""
    ctx = length - n
    see = np.zeros((n, length), bool)
    for t in range(n):
        others = t if rows is None else len([j for j in rows[t] if j < n and j != t])
        pos = ctx + others
        see[t, max(0, min(ctx, pos - W + 1)):ctx] = True
        see[t, :min(S, ctx)] = True
        if rows is None:
            see[t, max(ctx, pos - W + 1):ctx + t + 1] = True
            see[t, ctx:min(ctx + t + 1, max(ctx, S))] = True
        else:
            see[t, [ctx + j for j in rows[t] if j < n]] = True
    return see


def run(h, q, counts, W, S, rows=None, dense=False, **kw):
    words = None if rows is None else words_of(rows, max(1, -(-max(counts + [1]) // 64)))
    cu = None if dense else ints(np.cumsum([0] + counts).tolist())
    got = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), mask=words, cu_seqlens=cu,
                            max_seqlen=None if dense else max(counts + [0]), window=W, sinks=S, **kw)
    h.cache.check()
    return got


def check(h, counts, q, got, W, S, rows=None, sample=12):
    o, lse = f64(got[0]), f64(got[1])
    q64, t = f64(q), 0
    for i, n in enumerate(counts):
        pick = np.arange(n) if n <= sample else np.unique(np.r_[0, n - 1, np.random.RandomState(i).randint(0, n, sample)])
        if n:
            see = visible(n, h.lengths[i], W, S, None if rows is None else rows[t:t + n])[pick]
            k, v = (np.where(see.any(0)[:, None, None], x[i], 0.0) for x in (h.k, h.v))
            ro, rl, bo, bl = attend(q64[t + pick], k, v, see, q.shape[2] ** -0.5)
            within(f"o of {i}", o[t + pick], ro, bo)
            within(f"lse of {i}", lse[:, t + pick], rl, bl)
        t += n


def spoil(h, counts, W, S, rows=None):
    """NaN into K and V of all keys that nobody sees."""
    t = 0
    for i, n in enumerate(counts):
        see = visible(n, h.lengths[i], W, S, None if rows is None else rows[t:t + n])
        for pos in np.flatnonzero(~see.any(0)) if n else ():
            h.put("k", i, int(pos), NAN)
            h.put("v", i, int(pos), NAN)
        t += n


WINDOWS = [(1, 0), (1, 3), (17, 1), (64, 64), (100, 4), (128, 0), (200, 130), (5000, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
@pytest.mark.parametrize("W,S", [(1, 1), (100, 4), (128, 0), (200, 130)])
def test_single_tokens(Hq, heads, d, ps, W, S):
    lengths = [1, 2, ps, ps + 1, 63, 128, 129, 229, 257, 700, 2000]
    h = Held(lengths, heads, d, ps, seed=d + ps)
    counts = [1] * len(lengths)
    spoil(h, counts, W, S)
    q = queries(len(lengths), Hq, d)
    check(h, counts, q, run(h, q, counts, W, S, dense=True), W, S)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
@pytest.mark.parametrize("W,S", [(17, 1), (100, 4), (128, 128)])
def test_chunks(Hq, heads, d, ps, W, S):
    """Causal chunks of any length, empty sequences among them, with and without earlier tokens."""
    counts = [5, 0, 130, 1, 33, 64, 0, 300]
    ctx = [0, 40, 7, 300, 128, 0, 0, 600]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 1)
    spoil(h, counts, W, S)
    q = queries(sum(counts), Hq, d)
    check(h, counts, q, run(h, q, counts, W, S), W, S)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
@pytest.mark.parametrize("W,S", [(3, 2), (100, 4), (200, 130)])
def test_trees(Hq, heads, d, ps, W, S):
    rnd = random.Random(d * ps)
    counts, ctx = [1, 26, 64, 0, 7, 65, 100], [300, 0, 129, 10, 64, 700, 33]
    rows = [r for n in counts for r in random_tree(rnd, n)[1]]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 2)
    spoil(h, counts, W, S, rows)
    q = queries(sum(counts), Hq, d)
    check(h, counts, q, run(h, q, counts, W, S, rows), W, S, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("W,S", WINDOWS)
@pytest.mark.parametrize("Hq,heads,d", [(4, 2, 64), (8, 1, 128), (2, 1, 256)])
def test_windows(W, S, Hq, heads, d):
    counts, ctx = [1, 20, 200], [900, 515, 450]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, 32, seed=W + S)
    q = queries(sum(counts), Hq, d)
    check(h, counts, q, run(h, q, counts, W, S), W, S)
    # masks: rows that see nothing of their own, themselves not, later tokens, bits past the sequence
    rnd = random.Random(W)
    rows = [[], [5, 19], list(range(20))] + [sorted(rnd.sample(range(64), rnd.randint(0, 64))) for _ in range(218)]
    check(h, counts, q, run(h, q, counts, W, S, rows), W, S, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("d,ps,heads,group", [(128, 16, 2, 2), (64, 64, 1, 4), (64, 16, 1, 40), (256, 32, 1, 2)])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("tree", [False, True])
def test_values_of_hidden_places_do_not_matter(d, ps, heads, group, value, tree):
    """A V that is not finite at the window's edge reaches the rows that see it and no other."""
    n, ctx, W, S = 12, 400, 90, 3
    rows = [r for r in random_tree(random.Random(d), n)[1]] if tree else None
    see = visible(n, n + ctx, W, S, rows)
    for pos in (ctx - W + 3, ctx - W + 7, ctx + 4):
        if see[:, pos].all() or not see[:, pos].any():
            continue
        h = Held([n + ctx], heads, d, ps, seed=d)
        h.put("v", 0, pos, value)
        q = queries(n, group * heads, d)
        o = f64(run(h, q, [n], W, S, rows)[0])
        sees = see[:, pos]
        assert np.isfinite(o[~sees]).all() and not np.isfinite(o[sees]).any()
        h.v[0][pos] = 0
        ro, rl, bo, bl = attend(f64(q), h.k[0], h.v[0], see, d ** -0.5)
        within("o", o[~sees], ro[~sees], bo[~sees])


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 4)])
def test_infinite_values_that_all_rows_see(d, Hq):
    for where in (1, 380, 399):
        h = Held([400] * 5, 1, d, 16, seed=d)
        row = torch.randn(d).bfloat16().float()
        row[3], row[33] = INF, NAN
        h.put("v", 2, where, row)
        q = queries(5, Hq, d)
        check(h, [1] * 5, q, run(h, q, [1] * 5, 30, 2), 30, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps,tree", [(8, 2, 128, 64, True), (4, 4, 64, 16, False), (2, 1, 256, 128, False)])
def test_long_contexts(Hq, heads, d, ps, tree):
    """Windows and sinks of many pages (the loaders' page lists), few long items that CTAs share."""
    counts, ctx = [9, 1], [20000, 13000]
    rnd = random.Random(1)
    rows = [r for n in counts for r in random_tree(rnd, n)[1]] if tree else None
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d)
    q = queries(sum(counts), Hq, d)
    for W, S in ((3000, 16), (700, 2500), (9000, 0)):
        check(h, counts, q, run(h, q, counts, W, S, rows), W, S, rows, sample=4)


@pytest.mark.gpu
def test_nothing_hidden_is_the_plain_call():
    h = Held([300, 77], 2, 128, 32)
    q = queries(10, 4, 128)
    plain = fa.tree_attention(q, h.cache, h.layer, ints(h.slots))
    for W, S in ((10000, 0), (3, 10000)):
        got = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), window=W, sinks=S)
        assert all(torch.equal(a, b) for a, b in zip(plain, got))
    # a window that is as long as these sequences, but not as the table
    check(h, [5, 5], q, run(h, q, [5, 5], 305, 0), 305, 0)


@pytest.mark.gpu
def test_calls_agree_to_the_bit_on_streams_and_in_graphs():
    counts, ctx = [1, 30, 7], [3000, 500, 1200]
    h = Held([a + b for a, b in zip(counts, ctx)], 2, 128, 64)
    q, slots = queries(sum(counts), 8, 128), ints(h.slots)
    cu = ints(np.cumsum([0] + counts).tolist())
    call = lambda **kw: fa.tree_attention(q, h.cache, h.layer, slots, cu_seqlens=cu, max_seqlen=30,  # noqa: E731
                                          window=600, sinks=5, **kw)
    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = call()
    for _ in range(3):
        g.replay()
        again = call()
        torch.cuda.synchronize()
        for x in (other, held, again):
            assert all(torch.equal(a, b) for a, b in zip(first, x))
    h.cache.check()


@pytest.mark.gpu
def test_decoding_agrees_with_the_prompt():
    """Tokens appended one by one and looked at within the window, against one windowed pass over all of
    them: the same formula, two kernels."""
    n, W, S, hq, hkv, d = 150, 40, 3, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, x, d, generator=g).bfloat16().cuda() for x in (hq, hkv, hkv))
    table = fa.rotary_table(d, 256)
    cache = fa.PagedCache.allocate(1, 12, hkv, 16, d, 1, 12)
    slots, out = ints([0]), []
    for t in range(n):
        cache.reserve(slots, 1)
        qr = fa.cache_append(cache, 0, slots, k[t:t + 1], v[t:t + 1], q=q[t:t + 1], rotary=table)
        out.append(fa.tree_attention(qr, cache, 0, slots, window=W, sinks=S))
    cache.check()
    qr, kr = fa.rotary(q, k, table, batch=1)
    o, lse = fa.forward(qr, kr, v, causal=True, batch=1, window=W, sinks=S)
    see = visible(n, n, W, S)
    ro, rl, bo, bl = attend(f64(qr), f64(kr), f64(v), see, d ** -0.5)
    within("prompt", f64(o), ro, bo)
    within("decoding", f64(torch.cat([x[0] for x in out])), ro, bo)
    within("lse", f64(torch.cat([x[1] for x in out], 1)), rl, bl)
