"""Weights of cached keys where rows move: accepting drafts and forking take them along.  The kernels on
the host in several orders of their threads, on the GPU, and a run of drafting, verifying, accepting and
evicting against 64 bits."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
import evict_ref
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import U32, CacheModel, attend, f64, within
from test_cache import FAKE, desc
from test_cache_lanes import HERE, ORDERS, Cache, ints as host_ints, load
from test_tree import random_tree, words_of


def move(weights, slots, base, path, accepted, before):
    for s, b, p, m, n in zip(slots, base, path, accepted, before):
        w = weights[:, s]
        w[..., b:b + m] = w[..., [b + x for x in p[:m]]].copy()
        w[..., b + m:n] = 0


def copy(weights, parents, children, lengths):
    for p, c in zip(parents, children):
        weights[:, c] = 0
        weights[:, c, :, :lengths[p]] = weights[:, p, :, :lengths[p]]


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("emulated") / "cache.so")
    src = os.path.join(HERE, "cta_emulator")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I" + src,
                    os.path.join(src, "cache.cpp"), "-o", so], check=True)
    L = load(so)
    for name in ("fa_cache_accept_weights", "fa_cache_fork_weights"):
        getattr(L, name).restype, getattr(L, name).argtypes = fa._SIGS[name]
    return L


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("layers,heads", [(1, 1), (3, 2)])
def test_on_the_host(library, order, layers, heads):
    library.order_threads(*order)
    rnd = random.Random(layers)
    c = Cache(library, layers, 60, heads, 16, 64, 6, 9)
    w = torch.from_numpy(evict_ref.random_weights(np.random.default_rng(1), (layers, 6, heads, 144), "odd"))
    model = w.numpy().copy()
    assert c.reserve([0, 3, 4], [140, 33, 16]) == 0
    p, k = host_ints([0, 4, 0]), host_ints([1, 5, 2])
    assert library.fa_cache_fork_weights(c.at, p.data_ptr(), k.data_ptr(), w.data_ptr(), 3, None) == 0
    copy(model, [0, 4, 0], [1, 5, 2], c.model.lengths)
    assert c.model.fork([0, 4, 0], [1, 5, 2]) == 0 and c.status() == 0
    assert np.array_equal(w.numpy(), model, equal_nan=True)
    c.agree()
    assert c.reserve([3], [100]) == 0 and c.free([5]) == 0   # (4's page is its own again)
    for some, base, got, width, refused in (
            ([3], [33], [67], 70, False), ([3, 1], [5, 128], [1, 2], 2, False), ([1, 3], [129, 5], [0, 0], 0, False),
            ([4], [3], [10], 10, False), ([4, 3], [3, 2], [3, 3], 3, True)):
        path = [sorted(rnd.sample(range(c.model.lengths[s] - b), width)) for s, b in zip(some, base)]
        if refused:
            path[1] = [2, 1, 0]
        before = list(c.model.lengths)
        s, b, a = host_ints(some), host_ints(base), host_ints(got)
        t = host_ints(path).view(len(some), -1)
        assert library.fa_cache_accept_weights(c.at, s.data_ptr(), b.data_ptr(), t.data_ptr() or s.data_ptr(), width,
                                               a.data_ptr(), w.data_ptr(), len(some), None) == 0
        want = c.model.accept(some, base, path, got)
        assert bool(want) == refused and c.status() == want
        if not refused:
            move(model, some, base, path, got, [before[x] for x in some])
        assert np.array_equal(w.numpy(), model, equal_nan=True)
        c.agree()


@pytest.mark.parametrize("kw,status", [(dict(w=None), 1), (dict(w=FAKE + 2), 1), (dict(n=5), 1), (dict(a=None), 1),
                                       (dict(n=0, w=None), 0)])
def test_bad_calls_are_refused(kw, status):
    fabuild.build()
    held = desc()
    c = ctypes.addressof(held)
    x = dict(a=FAKE, b=FAKE, path=FAKE, width=3, acc=FAKE, w=FAKE, n=2)
    x.update(kw)
    assert fa.lib().fa_cache_accept_weights(c, x["a"], x["b"], x["path"], x["width"], x["acc"], x["w"], x["n"], None) == status
    assert fa.lib().fa_cache_fork_weights(c, x["a"], x["b"], x["w"], x["n"], None) == status


def test_tensor_calls_refuse(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    cache = fa.PagedCache.allocate(2, 3, 2, 16, 64, 2, 2, device="cpu")
    s, w = torch.zeros(1, dtype=torch.int32), torch.zeros(2, 2, 2, 32)
    for bad in (w[:1], w.double(), torch.zeros(2, 2, 2, 64)[..., ::2], w[0], w.clone().requires_grad_()):
        with pytest.raises(ValueError, match="weights|differentiable"):
            cache.fork(s, s + 1, weights=bad)
        with pytest.raises(ValueError, match="weights|differentiable"):
            cache.accept(s, s, s[None], s, weights=bad)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("heads,d,ps", [(1, 64, 16), (8, 128, 64)])
def test_accept_and_fork_move_weights(heads, d, ps):
    fabuild.build()
    layers, lengths = 3, [300, 70, 700, 64, 130]
    rng, rnd = np.random.default_rng(d), random.Random(d)
    cache = fa.PagedCache.allocate(layers, 120, heads, ps, d, 9, 800 // ps + 1)
    w = torch.from_numpy(evict_ref.random_weights(rng, (layers, 9, heads, cache.max_pages * ps), "odd")).cuda()
    model = w.cpu().numpy().copy()
    cache.reserve(ints(range(5)), ints(lengths))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.fork(ints([2, 0, 2]), ints([6, 8, 5]), weights=w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    copy(model, [2, 0, 2], [6, 8, 5], lengths)
    assert np.array_equal(w.cpu().numpy(), model, equal_nan=True)
    base = [250, 69, 697, 64, 0]
    path = [sorted(rnd.sample(range(n - b), min(130, n - b))) + [0] * (130 - min(130, n - b))
            for n, b in zip(lengths, base)]
    got = [33, 1, 0, 0, 100]
    cache.free(ints([5, 6, 8]))   # (what is moved may not be shared)
    cache.accept(ints(range(5)), ints(base), ints(path), ints(got), weights=w)
    cache.check()
    move(model, range(5), base, path, got, lengths)
    assert np.array_equal(w.cpu().numpy(), model, equal_nan=True)
    cache.accept(ints([0, 1]), ints([900, 0]), ints([[0], [0]]), ints([1, 1]), weights=w)  # refused whole
    with pytest.raises(fa.FAError):
        cache.check()
    assert np.array_equal(w.cpu().numpy(), model, equal_nan=True)


@pytest.mark.gpu
def test_drafting_with_a_budget():
    """Draft, attend, weigh (rejected rows left out), accept with the weights, evict: weights belong to
    the tokens that hold the places, as if the accepted ones had been decoded one by one."""
    fabuild.build()
    heads, group, d, ps, keep, recent, sinks = 2, 2, 64, 16, 60, 10, 2
    rnd = random.Random(5)
    cache = fa.PagedCache.allocate(1, 40, heads, ps, d, 2, 12)
    cache.k.zero_(), cache.v.zero_()
    model = CacheModel(cache.k, cache.v, cache.table, cache.lengths, cache.refs)
    slots, room = [1, 0], 12 * ps
    w = torch.zeros(1, 2, heads, room, device="cuda")
    want, slack = np.zeros((1, 2, heads, room)), np.zeros((1, 2, heads, room))

    def rows_of(new):
        total = sum(new)
        return [torch.randn(total, x, d, device="cuda").bfloat16() for x in (heads * group, heads, heads)]

    def step(new, rows, keep_rows):
        cache.reserve(ints(slots), ints(new))
        assert model.reserve(slots, new) == 0
        cu = ints(np.cumsum([0] + new).tolist())
        q, k, v = rows_of(new)
        args = dict(cu_seqlens=cu, max_seqlen=max(new))
        q = fa.cache_append(cache, 0, ints(slots), k, v, q=q, cu_seqlens=cu)
        model.k[0], model.v[0] = f64(cache.k[0]), f64(cache.v[0])
        mask = None if rows is None else words_of(rows, 1)
        _, lse = fa.tree_attention(q, cache, 0, ints(slots), mask=mask, **args)
        kept = torch.zeros(sum(new), dtype=torch.bool)
        kept[keep_rows] = True
        fa.cache_weights(q, lse.masked_fill(~kept.cuda(), -np.inf), cache, 0, ints(slots), w[0], mask=mask, **args)
        t = 0
        for s, n in zip(slots, new):
            length = model.lengths[s]
            see = np.tril(np.ones((n, length), bool), length - n)
            if rows is not None:
                see[:, length - n:] = False
                for i in range(n):
                    see[i, [length - n + j for j in rows[t + i]]] = True
            _, rl, _, bl = attend(f64(q)[t:t + n], model.rows("k", 0, s), model.rows("v", 0, s), see, d ** -0.5)
            on = kept[t:t + n].numpy()
            for h in range(heads):
                kk = model.rows("k", 0, s)[:, h]
                for a in range(h * group, (h + 1) * group):
                    x = d ** -0.5 * f64(q)[t:t + n, a] @ kk.T
                    p = np.where(see & on[:, None], np.exp(x - rl[a][:, None]), 0)
                    want[0, s, h, :length] += p.sum(0)
                    e = bl[a][:, None] + 2 * d * U32 * d ** -0.5 * (np.abs(f64(q)[t:t + n, a]) @ np.abs(kk).T) + \
                        8 * U32 * (np.abs(x) + np.abs(rl[a][:, None]) + 4)
                    slack[0, s, h, :length] += (p * 2 * (e + 2 * n * group * U32)).sum(0) + \
                        4 * U32 * want[0, s, h, :length]
            t += n
        within("weights", w.cpu().numpy(), want, slack)

    step([90, 50], None, list(range(140)))
    for _ in range(5):
        new = [rnd.randint(4, 20), rnd.randint(4, 20)]
        base = [model.lengths[s] for s in slots]
        trees = [random_tree(rnd, n)[1] for n in new]
        path = [t[rnd.randrange(n)] for t, n in zip(trees, new)]      # a token and its ancestors
        width = max(map(len, path))
        step(new, trees[0] + trees[1], path[0] + [new[0] + x for x in path[1]])
        wide = [p + [0] * (width - len(p)) for p in path]
        got = [len(p) for p in path]
        before = [model.lengths[s] for s in slots]
        cache.accept(ints(slots), ints(base), ints(wide), ints(got), weights=w)
        assert model.accept(slots, base, wide, got) == 0
        for x in (want, slack):
            move(x, slots, base, wide, got, before)
        within("weights", w.cpu().numpy(), want, slack)
        cache.check()
        mine = w.cpu().numpy().astype(np.float64)  # the eviction goes by the sums that are there
        exact = [mine.copy(), want.copy(), slack.copy()]
        order = mine.astype(np.float32)
        evict_ref.evict(model, order, slots, [keep] * 2, recent, sinks)
        cache.evict(ints(slots), w, keep, recent, sinks=sinks)
        cache.check()
        assert np.array_equal(w.cpu().numpy(), order)
        for s in slots:                 # the exact sums go where the eviction has put theirs
            for h in range(heads):
                lookup = {float(v): j for j, v in reversed(list(enumerate(exact[0][0, s, h])))}
                for x in (1, 2):
                    src = exact[x][0, s, h].copy()
                    out = np.array([src[lookup[float(v)]] if v else 0.0 for v in order[0, s, h]])
                    (want if x == 1 else slack)[0, s, h] = out
