"""Drafted trees that may be deeper than the window: the mask and depths of `window_mask`, attention with
them against 64 bits, and verifying a path against decoding it token by token."""
import ctypes
import random

import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import attend, f64, within
from test_cache import FAKE, desc
from test_tree import HEADS, Held, queries, random_tree, words_of

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


@pytest.mark.parametrize("kw,status", [(dict(window=0), 1), (dict(sinks=-1), 1), (dict(mask=None), 1), (dict(depth=None), 1),
                                       (dict(depth=FAKE + 2), 1), (dict(out=FAKE + 4), 1), (dict(words=0), 1),
                                       (dict(T=7), 1), (dict(slots=None), 1), (dict(T=0, B=0), 0)])
def test_bad_masks_are_refused(kw, status):
    a = dict(slots=FAKE, B=2, N=3, cu=None, T=6, mask=FAKE, words=1, window=4, sinks=0, out=FAKE, depth=FAKE, stream=None)
    a.update(kw)
    held = desc()
    assert fa.lib().fa_tree_window_mask(ctypes.addressof(held), *a.values()) == status


@pytest.mark.parametrize("kw,status", [(dict(window=0), 1), (dict(mask=None), 1), (dict(depth=None), 1),
                                       (dict(depth=FAKE + 1), 1), (dict(ws_bytes=10), 1), (dict(scale=0.0), 2)])
def test_bad_calls_are_refused(kw, status):
    a = dict(layer=0, slots=FAKE, B=2, N=3, cu=None, T=6, q=FAKE, Hq=4, qt=256, qh=64, mask=FAKE, words=1, depth=FAKE,
             o=FAKE, lse=FAKE, scale=0.125, window=5, sinks=1, zero=0, ws=FAKE, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    held = desc()
    assert fa.lib().fa_tree_fwd_window_depth(ctypes.addressof(held), *a.values()) == status


def test_tensor_calls_refuse(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    cache = fa.PagedCache.allocate(1, 3, 2, 16, 64, 2, 2, device="cpu")
    q, slots = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    mask, depth = torch.zeros(2, 1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    for kw in (dict(depth=depth), dict(depth=depth, window=4), dict(depth=depth, mask=mask),
               dict(depth=depth[:1], mask=mask, window=4), dict(depth=depth.long(), mask=mask, window=4)):
        with pytest.raises(ValueError, match="depth"):
            fa.tree_attention(q, cache, 0, slots, **kw)
    for kw in (dict(window=0), dict(window=2, sinks=-1), dict(window=1.5), dict(mask=mask.int(), window=2),
               dict(mask=mask[:1], window=2), dict(slots=slots.long(), window=2)):
        with pytest.raises(ValueError):
            fa.window_mask(**{**dict(mask=mask, cache=cache, slots=slots), **kw})


def near(rows, n, ctx, W, S):
    """Depths of a sequence's tokens, and the tokens that the window leaves of those they name."""
    own = [[j for j in row if j < n] for row in rows]
    depth = [len([j for j in row if j != t]) for t, row in enumerate(own)]
    left = [[a for a in row if a == t or depth[t] - depth[a] < W or ctx + depth[a] < S] for t, row in enumerate(own)]
    return depth, left


def visible(n, length, W, S, rows):
    ctx = length - n
    depth, left = near(rows, n, ctx, W, S)
    see = np.zeros((n, length), bool)
    for t in range(n):
        see[t, max(0, min(ctx, ctx + depth[t] - W + 1)):ctx] = True
        see[t, :min(S, ctx)] = True
        see[t, [ctx + a for a in left[t]]] = True
    return see


def deep_tree(rnd, n):
    """Long paths with short branches."""
    rows = []
    for j in range(n):
        p = j - 1 if rnd.random() < 0.8 else j - 1 - rnd.randint(0, 9)
        rows.append((rows[p] if p >= 0 else []) + [j])
    return rows


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("W,S", [(1, 0), (3, 2), (20, 40), (64, 0), (2 ** 31 - 1, 0), (2, 2 ** 31 - 1)])
def test_masks(W, S):
    rnd = random.Random(W)
    counts, ctx = [1, 26, 0, 150, 64], [300, 0, 10, 37, 1]
    h = Held([a + b for a, b in zip(counts, ctx)], 1, 64, 16)
    rows = [r for n in counts for r in deep_tree(rnd, n)]
    rows[3] = [9, 3, 170, 25]                       # not a tree, and bits past the sequence
    words = words_of(rows, 3)
    out, depth = fa.window_mask(words, h.cache, ints(h.slots), W, S, cu_seqlens=ints(np.cumsum([0] + counts).tolist()),
                                max_seqlen=150)
    t, want, deep = 0, [], []
    for n, c in zip(counts, ctx):
        d, left = near(rows[t:t + n], n, c, W, S)
        want, deep, t = want + left, deep + d, t + n
    assert depth.tolist() == deep and torch.equal(out, words_of(want, 3))
    # tokens of no sequence, boundaries that decrease; in place
    again = words.clone()
    depth.fill_(7)
    cu = ints([5, 20, 10, 30, 30, 200])
    fa.lib().fa_tree_window_mask(h.cache._at, ints(h.slots).data_ptr(), 5, 150, cu.data_ptr(), len(rows), again.data_ptr(), 3,
                                 W, S, again.data_ptr(), depth.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert not again[:5].any() and not depth[:5].any() and not again[200:].any() and not depth[200:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
@pytest.mark.parametrize("W,S", [(3, 2), (30, 0), (17, 70)])
def test_deep_trees(Hq, heads, d, ps, W, S):
    rnd = random.Random(d * ps)
    counts, ctx = [1, 26, 64, 0, 7, 65, 100], [300, 0, 129, 10, 64, 700, 33]
    rows = [r for n in counts for r in deep_tree(rnd, n)]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 2)
    sees, t = [], 0
    for i, n in enumerate(counts):
        sees.append(visible(n, h.lengths[i], W, S, rows[t:t + n]))
        for pos in np.flatnonzero(~sees[i].any(0)) if n else ():
            h.put("k", i, int(pos), NAN)
            h.put("v", i, int(pos), NAN)
        t += n
    # a drafted V that is not finite reaches the rows that see it and no other
    h.put("v", 5, ctx[5] + 20, NAN)
    q, cu, slots = queries(sum(counts), Hq, d), ints(np.cumsum([0] + counts).tolist()), ints(h.slots)
    args = dict(cu_seqlens=cu, max_seqlen=100)
    mask, depth = fa.window_mask(words_of(rows, 2), h.cache, slots, W, S, **args)
    o, lse = fa.tree_attention(q, h.cache, h.layer, slots, mask=mask, depth=depth, window=W, sinks=S, **args)
    h.cache.check()
    t = 0
    for i, n in enumerate(counts):
        if n:
            see = sees[i]
            k, v = (np.where(see.any(0)[:, None, None], x[i], 0.0) for x in (h.k, h.v))
            ro, rl, bo, bl = attend(f64(q)[t:t + n], k, v, see, d ** -0.5)
            within(f"o of {i}", f64(o)[t:t + n], ro, bo)
            within(f"lse of {i}", f64(lse)[:, t:t + n], rl, bl)
        t += n


@pytest.mark.gpu
@pytest.mark.parametrize("W,S", [(8, 2), (20, 0), (200, 3)])
def test_verifying_a_path_is_decoding_it(W, S):
    """The rows of a path in a drafted tree, against the same tokens appended one by one."""
    n, ctx, hq, hkv, d, ps = 60, 50, 4, 2, 64, 16
    rnd = random.Random(W)
    rows = deep_tree(rnd, n)
    path = max(rows, key=len)
    assert len(path) > 22
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(ctx + n, x, d, generator=g).bfloat16().cuda() for x in (hq, hkv, hkv))
    cache = fa.PagedCache.allocate(1, 30, hkv, ps, d, 2, 10)
    cache.k.zero_(), cache.v.zero_()
    slots = ints([0])
    cache.reserve(slots, ctx)
    fa.cache_append(cache, 0, slots, k[:ctx], v[:ctx])
    cache.fork(slots, ints([1]))
    cache.reserve(slots, n)
    fa.cache_append(cache, 0, slots, k[ctx:], v[ctx:])
    mask, depth = fa.window_mask(words_of(rows, 1), cache, slots, W, S)
    o, lse = fa.tree_attention(q[ctx:], cache, 0, slots, mask=mask, depth=depth, window=W, sinks=S)
    one = []
    for t in path:
        cache.reserve(ints([1]), 1)
        fa.cache_append(cache, 0, ints([1]), k[ctx + t:ctx + t + 1], v[ctx + t:ctx + t + 1])
        one.append(fa.tree_attention(q[ctx + t:ctx + t + 1], cache, 0, ints([1]), window=W, sinks=S))
    cache.check()
    at = list(range(ctx)) + [ctx + t for t in path]
    m = len(at)
    p, j = np.arange(ctx, m)[:, None], np.arange(m)[None]
    see = (j <= p) & ((p - j < W) | (j < S))
    ro, rl, bo, bl = attend(f64(q)[[ctx + t for t in path]], f64(k)[at], f64(v)[at], see, d ** -0.5)
    within("verified", f64(o)[path], ro, bo)
    within("verified lse", f64(lse)[:, path], rl, bl)
    within("decoded", f64(torch.cat([x[0] for x in one])), ro, bo)
    within("decoded lse", f64(torch.cat([x[1] for x in one], 1)), rl, bl)


@pytest.mark.gpu
def test_streams_and_graphs():
    rnd = random.Random(1)
    counts = [40, 7]
    h = Held([340, 57], 2, 128, 64)
    rows = [r for n in counts for r in deep_tree(rnd, n)]
    q, slots, cu = queries(47, 8, 128), ints(h.slots), ints([0, 40, 47])
    words, args = words_of(rows, 1), dict(cu_seqlens=cu, max_seqlen=40)

    def call(**kw):
        mask, depth = fa.window_mask(words, h.cache, slots, 9, 2, **args, **kw)
        return fa.tree_attention(q, h.cache, h.layer, slots, mask=mask, depth=depth, window=9, sinks=2, **args, **kw)
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
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for x in (other, held):
            assert all(torch.equal(a, b) for a, b in zip(first, x))
    h.cache.check()
