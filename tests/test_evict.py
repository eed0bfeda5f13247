"""Eviction on the GPU against the plain form, its refusals, and a run of the serving calls that keeps a
cache within a budget, step by step against a 64-bit model."""
import ctypes
import random

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import bwd_tiled_attention_gb300 as fa
import evict_ref
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import CacheModel, U32, attend, f64, within
from test_cache import FAKE, desc, ints


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(n=5), 1), (dict(slots=None), 1), (dict(slots=FAKE + 2), 1), (dict(keep=FAKE + 1), 1),
    (dict(recent=-1), 1), (dict(sinks=-1), 1), (dict(keep=None, keep_all=6), 1), (dict(w=None), 1),
    (dict(w=FAKE + 2), 1), (dict(recent=2 ** 31 - 1, sinks=1), 1), (dict(n=0), 0)])
def test_bad_calls_are_refused(kw, status):
    a = dict(slots=FAKE, keep=FAKE, keep_all=7, recent=3, sinks=4, w=FAKE, n=2, stream=None)
    a.update(kw)
    assert fa.lib().fa_cache_evict(ctypes.addressof(desc()), *a.values()) == status


def test_too_many_heads_in_all_are_refused():
    big = desc(layers=32767, heads=65535, pages=1, slots=4, max_pages=1)
    assert fa.lib().fa_cache_evict(ctypes.addressof(big), FAKE, None, 9, 1, 1, FAKE, 2, None) in (1, 2)


def test_tensor_calls_refuse(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    cache = fa.PagedCache.allocate(2, 3, 2, 16, 64, 2, 2, device="cpu")
    s, w = torch.zeros(1, dtype=torch.int32), torch.zeros(2, 2, 2, 32)
    good = dict(slots=s, weights=w, keep=9, recent=3, sinks=2)
    for kw in (dict(keep=4), dict(keep=2.5), dict(recent=-1), dict(sinks=-1), dict(weights=w[:1]),
               dict(weights=w.double()), dict(weights=torch.zeros(2, 2, 2, 64)[..., ::2]), dict(slots=s.long()),
               dict(slots=torch.zeros(3, dtype=torch.int32)), dict(keep=torch.zeros(2, dtype=torch.int32)),
               dict(keep=s.long()), dict(recent=2 ** 31 - 2, sinks=5, keep=2 ** 31 - 1)):
        with pytest.raises(ValueError):
            cache.evict(**{**good, **kw})
    with pytest.raises(ValueError, match="not differentiable"):
        cache.evict(s, w.clone().requires_grad_(), 9, 3)
    with forward_ad.dual_level(), pytest.raises(ValueError, match="forward tangent"):
        cache.evict(s, forward_ad.make_dual(w, w), 9, 3)


# --------------------------------------------------------------------------------- GPU


def make(lengths, layers, heads, ps, d, seed=0, kind="spread"):
    rng = np.random.default_rng(seed)
    n = len(lengths)
    width = max(-(-x // ps) for x in lengths) + 1
    cache = fa.PagedCache.allocate(layers, sum(-(-x // ps) for x in lengths) + 2, heads, ps, d, n + 1, width)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    slots = [int(s) for s in rng.permutation(n + 1)[:n]]
    cache.reserve(ints(slots), ints(lengths))
    w = evict_ref.random_weights(rng, (layers, n + 1, heads, width * ps), kind)
    return cache, slots, torch.from_numpy(w).cuda()


def same(cache, model, w, model_w):
    assert np.array_equal(f64(cache.k), model.k) and np.array_equal(f64(cache.v), model.v)
    assert cache.table.tolist() == model.table and cache.lengths.tolist() == model.lengths
    assert cache.refs.tolist() == model.refs
    assert np.array_equal(w.cpu().numpy(), model_w, equal_nan=True)


def evict(cache, slots, w, keep, recent, sinks, bits=0, **kw):
    model = CacheModel(cache.k, cache.v, cache.table, cache.lengths, cache.refs)
    model_w = w.cpu().numpy().copy()
    keeps = keep if isinstance(keep, list) else [keep] * len(slots)
    assert bool(evict_ref.evict(model, model_w, slots, keeps, recent, sinks)) == bool(bits)
    cache.evict(ints(slots), w, ints(keep) if isinstance(keep, list) else keep, recent, sinks=sinks, **kw)
    if bits:
        with pytest.raises(fa.FAError, match=bits):
            cache.check()
    cache.check()
    same(cache, model, w, model_w)


@pytest.mark.gpu
@pytest.mark.parametrize("d,ps,heads,layers", [(64, 16, 3, 2), (96, 32, 1, 3), (128, 64, 2, 1), (192, 128, 1, 2),
                                               (256, 16, 2, 2)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evictions(d, ps, heads, layers, kind):
    cache, slots, w = make([700, 90, 33, 1, 500], layers, heads, ps, d, d, kind)
    evict(cache, slots, w, [300, 90, 20, 13, 499], 10, 3)
    evict(cache, slots, w, 13, 10, 3)
    evict(cache, slots, w, 0, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("recent,sinks", [(0, 0), (1, 0), (0, 5), (128, 4), (196, 4), (90, 110)])
def test_recent_and_sinks(recent, sinks):
    cache, slots, w = make([1000, 205, 201], 2, 2, 32, 64)
    evict(cache, slots, w, 200, recent, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("length,keep,recent", [(9000, 5000, 64), (9000, 8000, 3000), (40000, 1000, 100),
                                                (70000, 34000, 100)])
def test_long_sequences(length, keep, recent):
    """Moves beyond one list, and more candidates than keys in shared memory."""
    cache, slots, w = make([length], 1, 1, 128, 64, length)
    evict(cache, slots, w, keep, recent, 4)


@pytest.mark.gpu
def test_refusals_change_nothing():
    cache, slots, w = make([100, 40, 64], 2, 2, 16, 64)
    a, b, c = slots
    spare = next(s for s in range(4) if s not in slots)
    evict(cache, [a, a], w, 20, 2, 2, "named twice")
    evict(cache, [a, 9], w, 20, 2, 2, "out of range")
    evict(cache, [a, b], w, [20, 3], 2, 2, "length")
    cache.free(ints([c]))
    cache.fork(ints([a]), ints([c]))
    evict(cache, [a], w, 50, 4, 2, "shared")
    evict(cache, [a], w, 96, 0, 96)      # only whole, kept pages are shared
    evict(cache, [c, spare], w, 100, 4, 2)  # nothing to do


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    cache, slots, w = make([400, 300], 2, 2, 32, 128)
    s = ints(slots)
    state = [x.clone() for x in (cache.k, cache.v, cache.table, cache.lengths, cache.refs, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.evict(s, w, 200, 30, sinks=4, stream=side)
    side.synchronize()
    want = [x.clone() for x in (cache.k, cache.v, cache.table, cache.lengths, cache.refs, w)]
    now = (cache.k, cache.v, cache.table, cache.lengths, cache.refs, w)
    for x, y in zip(now, state):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.evict(s, w, 200, 30, sinks=4)
    for _ in range(2):
        for x, y in zip(now, state):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(now, want))
    cache.check()


@pytest.mark.gpu
def test_a_cache_within_a_budget():
    """Prompts and then tokens one by one: append, attention, weights, and an eviction every few steps,
    against the model of the cache and the attention in 64 bits over what it holds."""
    layers, heads, group, d, ps, keep, recent, sinks = 2, 2, 2, 64, 16, 48, 16, 3
    rnd = random.Random(0)
    cache = fa.PagedCache.allocate(layers, 40, heads, ps, d, 3, 10)
    cache.k.zero_()
    cache.v.zero_()
    model = CacheModel(cache.k, cache.v, cache.table, cache.lengths, cache.refs)
    w = torch.zeros(layers, 3, heads, 160, device="cuda")
    table = fa.rotary_table(d, 512)
    slots, prompts = [2, 0], [70, 33]
    seen = [0, 0]

    def step(new):
        cache.reserve(ints(slots), ints(new))
        assert model.reserve(slots, new) == 0
        cu = ints(np.cumsum([0] + new).tolist())
        pos = ints([p + j for p, n in zip(seen, new) for j in range(n)])
        for layer in range(layers):
            g = torch.Generator().manual_seed(sum(seen) * layers + layer)
            q, k, v = (torch.randn(sum(new), x, d, generator=g).bfloat16().cuda() for x in (heads * group, heads, heads))
            before = f64(w[layer])
            q = fa.cache_append(cache, layer, ints(slots), k, v, q=q, rotary=table, positions=pos, cu_seqlens=cu)
            # (the append is tested elsewhere: its rows are taken over)
            model.k[layer], model.v[layer] = f64(cache.k[layer]), f64(cache.v[layer])
            args = dict(cu_seqlens=cu, max_seqlen=max(new))
            o, lse = fa.tree_attention(q, cache, layer, ints(slots), **args)
            fa.cache_weights(q, lse, cache, layer, ints(slots), w[layer], **args)
            t = 0
            for s, n in zip(slots, new):
                length = model.lengths[s]
                kk, vv = model.rows("k", layer, s), model.rows("v", layer, s)
                see = np.tril(np.ones((n, length), bool), length - n)
                ro, rl, bo, bl = attend(f64(q)[t:t + n], kk, vv, see, d ** -0.5)
                within("o", f64(o)[t:t + n], ro, bo)
                within("lse", f64(lse)[:, t:t + n], rl, bl)
                for h in range(heads):
                    got, room = before[s, h, :length].copy(), 0.0
                    for a in range(h * group, (h + 1) * group):
                        x = d ** -0.5 * f64(q)[t:t + n, a] @ kk[:, h].T
                        p = np.where(see, np.exp(x - rl[a][:, None]), 0)
                        got += p.sum(0)
                        e = bl[a][:, None] + 2 * d * U32 * d ** -0.5 * (np.abs(f64(q)[t:t + n, a]) @ np.abs(kk[:, h]).T) + \
                            8 * U32 * (np.abs(x) + np.abs(rl[a][:, None]) + 4)
                        room += (p * 2 * (e + 2 * n * group * U32)).sum(0)
                    within("weights", f64(w[layer, s, h, :length]), got, room + 4 * U32 * np.abs(got))
                t += n
        for i, n in enumerate(new):
            seen[i] += n

    step(prompts)
    for turn in range(6):
        for _ in range(rnd.randint(1, 5)):
            step([1, 1] if turn % 2 else [rnd.randint(1, 3), rnd.randint(1, 3)])
        model_w = w.cpu().numpy().copy()
        evict_ref.evict(model, model_w, slots, [keep] * 2, recent, sinks)
        cache.evict(ints(slots), w, keep, recent, sinks=sinks)
        cache.check()
        same(cache, model, w, model_w)
