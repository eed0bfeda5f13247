"""Accumulated attention weight of cached keys, against a 64-bit implementation: all head layouts and page
sizes, single tokens, chunks and trees, what lies in pages, and what is refused.

The pages hold NaN wherever no token of the test stands."""
import ctypes
import random

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import U32, f64, within
from test_cache import FAKE, desc, ints
from test_tree import HEADS, Held, queries, random_tree, visible, words_of

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(slots=None), 1), (dict(q=None), 1), (dict(q=FAKE + 8), 1),
    (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hq=2 * 129), 2), (dict(lse=None), 1), (dict(lse=FAKE + 2), 1),
    (dict(w=None), 1), (dict(w=FAKE + 2), 1), (dict(scale=0.0), 2), (dict(scale=NAN), 2), (dict(T=7), 1),
    (dict(N=-1), 1), (dict(qt=0), 1), (dict(qt=130), 1), (dict(qh=65), 1), (dict(mask=FAKE), 1),
    (dict(mask=FAKE + 4, words=1), 1), (dict(cu=FAKE + 2), 1), (dict(B=2 ** 30 + 1, cu=FAKE), 2)])
def test_bad_calls_are_refused(kw, status):
    a = dict(layer=0, slots=FAKE, B=2, N=3, cu=None, T=6, q=FAKE, Hq=4, qt=256, qh=64, lse=FAKE, mask=None,
             words=0, w=FAKE, scale=0.125, stream=None)
    a.update(kw)
    assert fa.lib().fa_cache_weights(ctypes.addressof(desc()), *a.values()) == status


def host_cache(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    return fa.PagedCache.allocate(1, 3, 2, 16, 64, 2, 2, device="cpu")


def test_tensor_calls_refuse(monkeypatch):
    cache = host_cache(monkeypatch)
    slots = torch.zeros(2, dtype=torch.int32)
    good = dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16), lse=torch.zeros(4, 2), cache=cache, layer=0,
                slots=slots, weights=torch.zeros(2, 2, 32))
    for kw in (dict(lse=torch.zeros(2, 4)), dict(lse=torch.zeros(4, 2).double()), dict(weights=torch.zeros(2, 2, 31)),
               dict(weights=torch.zeros(1, 2, 2, 32)), dict(weights=torch.zeros(2, 2, 64)[..., ::2]), dict(layer=1),
               dict(q=torch.zeros(2, 3, 64, dtype=torch.bfloat16)), dict(q=torch.zeros(2, 4, 128, dtype=torch.bfloat16)),
               dict(mask=torch.zeros(1, 1, dtype=torch.int64)), dict(slots=slots.long())):
        with pytest.raises(ValueError):
            fa.cache_weights(**{**good, **kw})
    for name in ("q", "lse", "weights"):
        with pytest.raises(ValueError, match="not differentiable"):
            fa.cache_weights(**{**good, name: good[name].clone().requires_grad_()})
        with forward_ad.dual_level(), pytest.raises(ValueError, match="forward tangent"):
            fa.cache_weights(**{**good, name: forward_ad.make_dual(good[name], good[name])})


# --------------------------------------------------------------------------------- GPU


def expected(h, counts, q, lse, w, rows=None, scale=None):
    """Weights afterwards and their bounds, [slots, heads, places]."""
    q64, l64, out = f64(q), f64(lse), f64(w)
    bound = np.zeros_like(out)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    hq, d, heads = q.shape[1], q.shape[2], h.k[0].shape[1]
    t = 0
    for i, n in enumerate(counts):
        if n:
            see = visible(n, h.lengths[i], None if rows is None else rows[t:t + n])
            for a in range(hq):
                g = a // (hq // heads)
                k, x = h.k[i][:, g], q64[t:t + n, a]
                s = scale * (x @ k.T)
                l = l64[a, t:t + n, None]
                with np.errstate(over="ignore", invalid="ignore"):
                    p = np.where(see & (np.abs(l) < INF), np.exp(s - np.where(np.isinf(l), 0, l)), 0.0)
                # a score sums d products, scaling and subtracting round once each, the
                # exponential has two ulps; a key adds up as many terms as there are rows
                e = scale * 2 * d * U32 * (np.abs(x) @ np.abs(k).T) + 4 * U32 * (np.abs(s) + np.abs(np.where(np.isinf(l), 0, l)))
                at = (h.slots[i], g, slice(0, h.lengths[i]))
                out[at] += p.sum(0)
                bound[at] += (p * (2 * e + 16 * U32 + 2 * U32 * n * (hq // heads))).sum(0) + U32 * p.sum(0)
        t += n
    return out, bound + 2 * U32 * np.abs(out)


def run(h, q, counts, rows=None, dense=False, lse=None, w=None, scale=None, **kw):
    words = None if rows is None else words_of(rows, max(1, -(-max(counts + [1]) // 64)))
    cu = None if dense else ints(np.cumsum([0] + counts).tolist())
    args = dict(mask=words, cu_seqlens=cu, max_seqlen=None if dense else max(counts + [0]), scale=scale)
    if lse is None:
        _, lse = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), **args)
    c = h.cache
    if w is None:
        w = torch.rand(c.slots, c.heads, c.max_pages * c.page_size, device="cuda")
    before = w.clone()
    fa.cache_weights(q, lse, c, h.layer, ints(h.slots), w, **args, **kw)
    c.check()
    ref, bound = expected(h, counts, q, lse, before, rows, scale)
    within("weights", f64(w), ref, bound)
    return lse, before, w


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
def test_single_tokens(Hq, heads, d, ps):
    lengths = [1, 2, ps, ps + 1, 63, 64, 65, 127, 128, 129, 257, 700]
    h = Held(lengths, heads, d, ps, seed=d + ps)
    run(h, queries(len(lengths), Hq, d), [1] * len(lengths), dense=True)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
def test_chunks(Hq, heads, d, ps):
    """Causal chunks of any length, empty sequences among them, with and without earlier tokens."""
    counts = [5, 0, 130, 1, 33, 64, 0, 300]
    ctx = [0, 40, 7, 300, 128, 0, 0, 600]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 1)
    run(h, queries(sum(counts), Hq, d), counts)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
def test_trees(Hq, heads, d, ps):
    rnd = random.Random(d * ps)
    counts, ctx = [1, 26, 64, 0, 7, 65, 100], [300, 0, 129, 10, 64, 700, 33]
    rows = [r for n in counts for r in random_tree(rnd, n)[1]]
    rows[3] = []
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 2)
    run(h, queries(sum(counts), Hq, d), counts, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 64), (256, 128)])
def test_many_and_long_sequences(d, ps):
    rnd = random.Random(d)
    lengths = [rnd.randint(1, 400) for _ in range(500)] + [9000]
    h = Held(lengths, 2, d, ps, seed=d)
    run(h, queries(len(lengths), 4, d), [1] * len(lengths), dense=True)
    h = Held([5000, 12001], 1, d, ps, seed=d + 1)
    run(h, queries(60 + 70, 4, d), [60, 70], scale=0.05)


@pytest.mark.gpu
def test_rows_and_places_that_give_and_get_nothing():
    h = Held([40, 300], 2, 64, 16)
    counts = [7, 3]
    q = queries(10, 4, 64)
    lse = torch.full((4, 10), INF, device="cuda")
    run(h, q, counts, lse=lse)            # exp(s - inf) = 0
    lse = torch.randn(4, 10, device="cuda") + 5
    lse[:, ::2] = -INF
    _, before, w = run(h, q, counts, lse=lse)
    c = h.cache
    for s in range(c.slots):
        n = h.lengths[h.slots.index(s)] if s in h.slots else 0
        assert torch.equal(before[s, :, n:], w[s, :, n:])
    # keys past a length, and drafted ones that a row does not see, may be anything
    h.put("k", 1, 299, NAN)
    lse = torch.randn(4, 10, device="cuda") + 5
    fa.cache_weights(q, lse, c, h.layer, ints(h.slots), w, cu_seqlens=ints([0, 7, 10]), max_seqlen=7)
    mine = w[h.slots[1]]
    assert torch.isfinite(mine[:, :299]).all() and torch.isnan(mine[:, 299]).all()


@pytest.mark.gpu
def test_strided_queries_a_slot_twice_and_streams():
    h = Held([500, 90], 2, 128, 32)
    x = queries(4, 8, 128)
    q = x[:, ::2]
    assert not q.is_contiguous()
    lse, before, w = run(h, q, [2, 2], dense=True)
    both = before.clone()
    s = ints([h.slots[0], h.slots[0]])
    fa.cache_weights(q, lse, h.cache, h.layer, s, both, stream=torch.cuda.current_stream())
    one = torch.zeros_like(both)
    for i in range(2):
        fa.cache_weights(q[2 * i:2 * i + 2], lse[:, 2 * i:2 * i + 2].contiguous(), h.cache, h.layer, s[:1], one)
    assert torch.allclose(both - before, one, rtol=1e-4, atol=1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = before.clone()
    side.wait_stream(torch.cuda.current_stream())
    fa.cache_weights(q, lse, h.cache, h.layer, ints(h.slots), other, stream=side)
    side.synchronize()
    assert torch.equal(other, w)
    held = before.clone()
    slots = ints(h.slots)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.cache_weights(q, lse, h.cache, h.layer, slots, held)
    held.copy_(before)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, w)


@pytest.mark.gpu
@pytest.mark.parametrize("change,bits", [("slot", "slot"), ("length", "length"), ("boundaries", "length"),
                                         ("page", "slot or page")])
def test_refused_on_the_device(change, bits):
    """What does not fit is reported, and the other sequences get their sums."""
    h = Held([100, 60], 2, 64, 16)
    q, lse = queries(4, 4, 64), torch.randn(4, 4, device="cuda") + 4
    slots, cu = list(h.slots), [0, 2, 4]
    w = torch.zeros(h.cache.slots, 2, h.cache.max_pages * 16, device="cuda")
    if change == "slot":
        slots[1] = 77
    elif change == "length":
        h.cache.lengths[slots[1]] = 1
    elif change == "boundaries":
        cu = [0, 2, 9]
    else:
        h.cache.table[slots[1], 1] = 10 ** 6
    fa.cache_weights(q, lse, h.cache, h.layer, ints(slots), w, cu_seqlens=ints(cu), max_seqlen=2)
    with pytest.raises(fa.FAError, match=bits):
        h.cache.check()
    h.cache.check()
    assert w[h.slots[0], :, :100].all()
    if change != "page":
        assert not w[h.slots[1]].any()


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,heads", [(64, 4, 1), (128, 8, 1), (128, 2, 2), (192, 6, 1), (256, 4, 2), (96, 128, 1)])
def test_more_rows_than_stay_in_shared_memory(d, Hq, heads):
    """Several turns over a stretch of keys, with and without a mask, beside a short sequence."""
    counts, ctx = [700, 1], [300, 500]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, 64, seed=d)
    q = queries(sum(counts), Hq, d)
    lse, before, w = run(h, q, counts)
    again = before.clone()
    fa.cache_weights(q, lse, h.cache, h.layer, ints(h.slots), again, cu_seqlens=ints([0, 700, 701]), max_seqlen=700)
    assert torch.equal(again, w)
    rnd = random.Random(d)
    run(h, q, counts, [sorted(rnd.sample(range(700), rnd.randint(0, 5))) for _ in range(700)] + [[0]])


@pytest.mark.gpu
def test_two_calls_at_once():
    """Layers, or sequences, that two streams work on at the same time: what each leaves alone."""
    a, b = Held([3000, 900], 2, 128, 64, seed=1), Held([2500, 40], 2, 64, 16, seed=2)
    work = []
    for h, hq, n in ((a, 8, 1), (b, 4, 40)):
        q = queries(2 * n, hq, h.k[0].shape[2])
        _, lse = fa.tree_attention(q, h.cache, h.layer, ints(h.slots))
        c = h.cache
        w = torch.zeros(c.slots, c.heads, c.max_pages * c.page_size, device="cuda")
        fa.cache_weights(q, lse, c, h.layer, ints(h.slots), w)
        work.append((h, q, lse, ints(h.slots), w, torch.zeros_like(w), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for h, q, lse, s, _, mine, stream in work:
            with torch.cuda.stream(stream):
                mine.zero_()
                fa.cache_weights(q, lse, h.cache, h.layer, s, mine)
    torch.cuda.synchronize()
    for h, _, _, _, want, mine, _ in work:
        assert torch.equal(want, mine)
        h.cache.check()
