"""Attention over the paged cache against a 64-bit implementation: single tokens, chunks, trees and
arbitrary masks, all head layouts and page sizes, what lies in pages and drafted rows that must not
matter, and what is refused.

The pages hold NaN wherever no token of the test stands."""
import ctypes
import random

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import attend, f64, within
from test_cache import FAKE, desc, ints

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


# ------------------------------------------------------------------------- refusals (CPU)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), 1), (dict(layer=-1), 1), (dict(slots=None), 1), (dict(q=None), 1),
    (dict(q=FAKE + 8), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hq=2 * 129), 2), (dict(o=None), 1),
    (dict(lse=None), 1), (dict(scale=0.0), 2), (dict(scale=NAN), 2), (dict(T=7), 1), (dict(N=-1), 1),
    (dict(qt=0), 1), (dict(qt=130), 1), (dict(qh=0), 1), (dict(qh=65), 1), (dict(mask=FAKE), 1),
    (dict(mask=FAKE, words=1, N=65, B=1, T=65), 1), (dict(mask=FAKE + 4, words=1), 1),
    (dict(ws=None), 1), (dict(ws_bytes=1000), 1), (dict(cu=FAKE + 2), 1)])
def test_bad_calls_are_refused(kw, status):
    a = dict(layer=0, slots=FAKE, B=2, N=3, cu=None, T=6, q=FAKE, Hq=4, qt=256, qh=64, mask=None,
             words=0, o=FAKE, lse=FAKE, scale=0.125, zero=0, ws=FAKE, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    assert fa.lib().fa_tree_fwd(ctypes.addressof(desc()), *a.values()) == status


def test_workspace_and_mask_arguments():
    L = fa.lib()
    assert L.fa_tree_workspace_size(32, 8, 1, 128) < L.fa_tree_workspace_size(32, 8, 64, 128)
    for a in ((0, 8, 1, 128), (32, 5, 1, 128), (32, 8, 0, 128), (129, 1, 1, 64)):
        assert L.fa_tree_workspace_size(*a) == 0
    ok = [FAKE, None, 2, 3, 6, 1, FAKE, None]
    for i, v in ((0, None), (2, -1), (3, 4), (5, 0), (6, None), (6, FAKE + 4), (0, FAKE + 2)):
        bad = list(ok)
        bad[i] = v
        assert L.fa_tree_mask(*bad) == fa.FA_ERR_INVALID_ARG
    assert L.fa_tree_mask(FAKE, FAKE, 2, 65, 10, 1, FAKE, None) == fa.FA_ERR_INVALID_ARG
    assert L.fa_tree_mask(None, None, 0, 0, 0, 1, None, None) == fa.FA_OK


def refuses_lost_gradients(cache, slots, table):
    """Whatever requires a gradient, or has a forward tangent, is refused where it would be cut off."""
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=cache.device)
    leaf, dual_of = x.clone().requires_grad_(), forward_ad.make_dual
    o, lse = x.clone(), torch.zeros(2, 2, device=cache.device)
    append = lambda k=x, v=x, q=x, **kw: fa.cache_append(cache, 0, slots, k, v, q=q, **kw)  # noqa: E731
    attend = lambda q=x, **kw: fa.tree_attention(q, cache, 0, slots, **kw)  # noqa: E731
    calls = [lambda t: append(k=t), lambda t: append(v=t), lambda t: append(q=t), lambda t: attend(q=t),
             lambda t: attend(out=(t, lse))]
    for call in calls:
        with pytest.raises(ValueError, match="not differentiable"):
            call(leaf)
        with forward_ad.dual_level(), pytest.raises(ValueError, match="forward tangent"):
            call(dual_of(x, x))
    with pytest.raises(ValueError, match="not differentiable"):
        attend(out=(o, lse.clone().requires_grad_()))
    for c in (lambda t: append(rotary=t), lambda t: fa.rotary(x, None, t, batch=1)):
        with pytest.raises(ValueError, match="gradient: detach|requires a gradient"):
            c(table.clone().requires_grad_())
    for held in (cache.k, cache.v):
        held.requires_grad_()
        for call in (append, attend):
            with pytest.raises(ValueError, match="not differentiable"):
                call()
        held.requires_grad_(False)
    return append, attend, leaf


def test_lost_gradients_are_refused(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    cache = fa.PagedCache.allocate(1, 3, 2, 16, 64, 2, 2, device="cpu")
    refuses_lost_gradients(cache, torch.zeros(2, dtype=torch.int32), torch.zeros(9, 32, 2))


# ---------------------------------------------------------------------------------- GPU


class Held:
    """A cache that holds `lengths` tokens in slots of its own, pages placed at random, NaN
    everywhere else."""

    def __init__(self, lengths, heads, d, ps, seed=0, layers=2, layer=1, scale_k=1.0):
        rnd = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.layer, self.ps, self.n = layer, ps, len(lengths)
        used = [-(-n // ps) for n in lengths]
        pages = sum(used) + 3
        order = rnd.sample(range(pages), pages)
        slots = rnd.sample(range(self.n + 2), self.n)
        k = torch.full((layers, pages, heads, ps, d), NAN, dtype=torch.bfloat16)
        v = k.clone()
        self.table = np.full((self.n + 2, max(used + [1]) + 1), -1, np.int32)
        lens, refs = [0] * (self.n + 2), [0] * pages
        self.k, self.v = [], []
        for n, u, s in zip(lengths, used, slots):
            mine, order = order[:u], order[u:]
            self.table[s, :u] = mine
            lens[s] = n
            kk = (torch.randn(u * ps, heads, d, generator=g) * scale_k).bfloat16()
            vv = torch.randn(u * ps, heads, d, generator=g).bfloat16()
            kk[n:], vv[n:] = NAN, NAN
            for x, y in ((k, kk), (v, vv)):
                if u:
                    x[layer, mine] = y.view(u, ps, heads, d).transpose(1, 2)
            for p in mine:
                refs[p] = 1
            self.k.append(f64(kk[:n]))
            self.v.append(f64(vv[:n]))
        self.lengths, self.slots = lengths, slots
        self.cache = fa.PagedCache(k.cuda(), v.cuda(), torch.from_numpy(self.table).cuda(), ints(lens),
                                   ints(refs))

    def put(self, which, i, pos, value):
        """Row pos of sequence i, all heads, in the cache and in the copy."""
        x = self.cache.k if which == "k" else self.cache.v
        x[self.layer, int(self.table[self.slots[i], pos // self.ps]), :, pos % self.ps] = value
        (self.k if which == "k" else self.v)[i][pos] = value


def queries(total, Hq, d, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 77)
    return (torch.randn(total, Hq, d, generator=g) * scale).bfloat16().cuda()


def words_of(rows, words):
    """Lists of visible indices -> int64 [T, words]."""
    out = np.zeros((len(rows), words), np.uint64)
    for t, row in enumerate(rows):
        for j in row:
            out[t, j // 64] |= np.uint64(1 << (j % 64))
    return torch.from_numpy(out.view(np.int64)).cuda()


def visible(n, length, rows=None):
    see = np.ones((n, length), bool)
    ctx = length - n
    own = np.tril(np.ones((n, n), bool)) if rows is None else np.zeros((n, n), bool)
    if rows is not None:
        for t, row in enumerate(rows):
            own[t, [j for j in row if j < n]] = True
    see[:, ctx:] = own
    return see


def check(h, counts, q, got, rows=None, sample=None, scale=None):
    """rows: per token of the packed batch, the own tokens that it sees."""
    o, lse = f64(got[0]), f64(got[1])
    scale = q.shape[2] ** -0.5 if scale is None else scale
    q64, t = f64(q), 0
    for i, n in enumerate(counts):
        pick = np.arange(n) if sample is None or n <= sample else \
            np.unique(np.r_[0, n - 1, np.random.RandomState(i).randint(0, n, sample)])
        if n:
            see = visible(n, h.lengths[i], None if rows is None else rows[t:t + n])[pick]
            ro, rl, bo, bl = attend(q64[t + pick], h.k[i], h.v[i], see, scale)
            within(f"o of {i}", o[t + pick], ro, bo)
            within(f"lse of {i}", lse[:, t + pick], rl, bl)
        t += n


def run(h, q, counts, rows=None, dense=False, N=None, **kw):
    words = None if rows is None else words_of(rows, max(1, -(-max(counts + [1]) // 64)))
    cu = None if dense else ints(np.cumsum([0] + counts).tolist())
    got = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), mask=words, cu_seqlens=cu,
                            max_seqlen=None if dense else (N or max(counts + [0])), **kw)
    h.cache.check()
    return got


HEADS = [  # Hq, heads, d, page size
    (4, 4, 64, 16), (8, 2, 128, 64), (3, 1, 128, 128), (8, 8, 128, 16), (12, 2, 96, 32), (5, 1, 192, 64),
    (4, 2, 256, 16), (2, 2, 256, 128), (16, 1, 64, 128), (128, 1, 64, 32), (200, 2, 128, 64), (6, 2, 192, 128),
    (1, 1, 96, 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
def test_single_tokens(Hq, heads, d, ps):
    lengths = [1, 2, ps, ps + 1, 63, 64, 65, 127, 128, 129, 257, 700]
    h = Held(lengths, heads, d, ps, seed=d + ps)
    q = queries(len(lengths), Hq, d)
    check(h, [1] * len(lengths), q, run(h, q, [1] * len(lengths), dense=True))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
def test_chunks(Hq, heads, d, ps):
    """Causal chunks of any length, empty sequences among them, with and without earlier tokens."""
    counts = [5, 0, 130, 1, 33, 64, 0, 300]
    ctx = [0, 40, 7, 300, 128, 0, 0, 100]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 1)
    q = queries(sum(counts), Hq, d)
    check(h, counts, q, run(h, q, counts), sample=12)


def random_tree(rnd, n):
    parents, rows = [], []
    for j in range(n):
        p = j - 1 - rnd.randint(0, 4)
        parents.append(max(p, -1))
        rows.append((rows[p] if p >= 0 else []) + [j])
    return parents, rows


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS)
def test_trees(Hq, heads, d, ps):
    rnd = random.Random(d * ps)
    counts, ctx = [1, 26, 64, 0, 7, 65, 100], [300, 0, 129, 10, 64, 200, 33]
    trees = [random_tree(rnd, n) for n in counts]
    rows = [r for t in trees for r in t[1]]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d + ps + 2)
    q = queries(sum(counts), Hq, d)
    got = run(h, q, counts, rows)
    check(h, counts, q, got, rows, sample=16)
    # the mask that the library makes of the parents is that mask
    parents = ints([p for t in trees for p in t[0]])
    cu = ints(np.cumsum([0] + counts).tolist())
    mask = fa.tree_mask(parents, cu_seqlens=cu, max_seqlen=100)
    assert torch.equal(mask, words_of(rows, 2))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", HEADS[:8])
def test_any_mask(Hq, heads, d, ps):
    """Rows that see nothing of their own, later tokens, bits past the sequence, empty contexts."""
    rnd = random.Random(d + ps)
    counts, ctx = [40, 9, 3], [0, 150, 0]
    rows = [[], [39], [0]] + [sorted(rnd.sample(range(40), rnd.randint(0, 40))) for _ in range(37)]
    rows += [[], [5, 60], list(range(64))] + [[rnd.randint(0, 8)] for _ in range(6)]
    rows += [[], [2], [0, 1, 63]]
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=d)
    q = queries(sum(counts), Hq, d)
    got = run(h, q, counts, rows)
    check(h, counts, q, got, rows)
    assert not got[0][0].any() and got[1][:, 0].eq(-INF).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,ps,heads", [(128, 16, 2), (64, 64, 1), (256, 32, 1)])
def test_values_of_masked_tokens_do_not_matter(d, ps, heads):
    """NaN and infinities in K or V of drafted tokens reach the rows that see them and no other."""
    counts, ctx = [12, 12], [0, 130]
    rows = [[j] if j % 3 else [0, j] for j in range(12)] * 2
    rows[4] = rows[16] = []
    for value in (NAN, INF, -INF):
        h = Held([12, 142], heads, d, ps, seed=d)
        h.put("v", 0, 5, value)
        h.put("v", 1, 130 + 7, value)
        h.put("k", 1, 130 + 2, value)
        q = queries(24, 2 * heads, d).abs()  # (q.k is then infinite, not NaN, for an infinite k)
        got = run(h, q, counts, rows)
        bad = np.zeros(24, bool)
        bad[[5, 12 + 7, 12 + 2]] = True
        keep = [i for i in range(24) if not bad[i]]
        o = f64(got[0])
        assert np.isfinite(o[keep]).all()
        assert not np.isfinite(o[[5, 19]]).any()
        for i in range(2):  # (the rows that see a value are left to the checks above)
            mine = np.arange(12 * i, 12 * i + 12)
            see = visible(12, h.lengths[i], rows[12 * i:12 * i + 12])
            see[bad[mine]] = False
            clean = [np.where(np.isfinite(x[i]), x[i], 0.0) for x in (h.k, h.v)]
            ro, rl, bo, bl = attend(f64(q)[mine], clean[0], clean[1], see, d ** -0.5)
            fine = ~bad[mine]
            within("o", o[mine][fine], ro[fine], bo[fine])
            within("lse", f64(got[1])[:, mine][:, fine], rl[:, fine], bl[:, fine])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("n", [10, 200])
def test_causal_rows_do_not_see_later_values(value, n):
    """The same without a mask, in one and in two row tiles."""
    h = Held([n + 50], 2, 128, 16, seed=n)
    h.put("v", 0, 50 + n - 3, value)
    q = queries(n, 4, 128)
    got = run(h, q, [n])
    o = f64(got[0])
    assert np.isfinite(o[:n - 3]).all() and not np.isfinite(o[n - 3:]).any()
    h.v[0][50 + n - 3] = 0
    ro, rl, bo, bl = attend(f64(q[:n - 3]), h.k[0], h.v[0], visible(n, n + 50)[:n - 3], 128 ** -0.5)
    within("o", o[:n - 3], ro, bo)


@pytest.mark.gpu
def test_values_of_the_context_reach_every_row():
    h = Held([300], 1, 128, 64)
    h.put("v", 0, 10, INF)
    got = run(h, queries(4, 1, 128), [4])
    assert got[0].eq(INF).all() and torch.isfinite(got[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq,n", [(64, 2, 1), (64, 3, 4), (64, 32, 1), (64, 40, 1), (128, 2, 4), (256, 2, 3)])
def test_infinite_values_of_the_context(d, Hq, n):
    """Single columns of V that are infinite or NaN, in one sequence that several CTAs share and in
    many that one CTA has to itself: the same columns come out infinite or NaN, in every row."""
    for lengths in ([700 + n], [130 + n] * 330):
        h = Held(lengths, 1, d, 16, seed=d + n)
        for i in range(0, len(lengths), 3):
            for pos, special in ((9, {3: INF}), (77, {3: INF, 5: -INF, 7: NAN, 33: INF}), (110, {5: INF})):
                row = torch.randn(d).bfloat16().float()
                for c, value in special.items():
                    row[c] = value
                h.put("v", i, pos, row)
        q = queries(n * len(lengths), Hq, d)
        check(h, [n] * len(lengths), q, run(h, q, [n] * len(lengths)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps,tree", [(8, 2, 128, 64, True), (4, 4, 64, 16, False),
                                                (2, 1, 256, 128, True), (32, 8, 128, 128, False)])
def test_long_contexts(Hq, heads, d, ps, tree):
    """Long sequences are split over the CTAs, beside short ones; scores of very different size."""
    counts, ctx = [17, 1, 64, 3], [20000, 3, 9001, 5000]
    rnd = random.Random(1)
    rows = [r for n in counts for r in random_tree(rnd, n)[1]] if tree else None
    h = Held([a + b for a, b in zip(counts, ctx)], heads, d, ps, seed=3, layers=1, layer=0, scale_k=4.0)
    q = queries(sum(counts), Hq, d, scale=2.0)
    check(h, counts, q, run(h, q, counts, rows), rows, sample=5)


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than threads of the kernel, empty ones among them."""
    rnd = random.Random(4)
    counts = [rnd.choice([0, 1, 1, 3]) for _ in range(1500)]
    lengths = [n + rnd.randint(0, 90) for n in counts]
    h = Held(lengths, 1, 64, 16, seed=8, layers=1, layer=0)
    q = queries(sum(counts), 2, 64)
    check(h, counts, q, run(h, q, counts))


@pytest.mark.gpu
def test_strided_queries_and_scale():
    h = Held([90, 200], 2, 64, 16)
    x = torch.randn(6, 8 + 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q = x[:, 2:10]
    check(h, [3, 3], q, run(h, q, [3, 3], dense=True, scale=0.5), scale=0.5)
    odd = torch.randn(6 * 700, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q = odd.as_strided((6, 8, 64), (700, 80, 1), 0)
    with pytest.raises(fa.FAError, match="INVALID"):   # 1400 bytes are no multiple of 16
        run(h, q, [3, 3], dense=True)
    q = odd.as_strided((6, 8, 64), (680, 80, 1), 16)
    check(h, [3, 3], q, run(h, q, [3, 3], dense=True))


@pytest.mark.gpu
def test_rows_of_no_sequence():
    """Rows behind the last sequence: zeros in new tensors, untouched in given ones."""
    h = Held([50, 300], 2, 64, 16)
    q = queries(20, 4, 64)
    cu = ints([0, 2, 9])
    o, lse = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), cu_seqlens=cu, max_seqlen=7)
    check(h, [2, 7], q, (o, lse))
    assert not o[9:].any() and lse[:, 9:].eq(-INF).all()
    out = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    got = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), cu_seqlens=cu, max_seqlen=7, out=out)
    assert got[0] is out[0] and torch.equal(out[0][:9], o[:9]) and torch.equal(out[1][:, :9], lse[:, :9])
    assert out[0][9:].eq(7).all() and out[1][:, 9:].eq(7).all()
    h.cache.check()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,N", [(4, 2, 9), (2, 1, 150)])
def test_rows_before_the_first_sequence(Hq, heads, N):
    """A packed batch that begins behind other tokens: those rows, and the ones behind the last
    sequence, come out empty, or stay as they are in `out`."""
    h = Held([30, 40], heads, 64, 16, seed=8)
    q = queries(25, Hq, 64)
    cu = ints([7, 10, 19])
    part = fa.tree_attention(q[7:19], h.cache, h.layer, ints(h.slots), cu_seqlens=ints([0, 3, 12]),
                             max_seqlen=N)
    junk = [torch.full((25, Hq, 64), NAN, dtype=torch.bfloat16).cuda(), torch.full((Hq, 25), NAN).cuda()]
    del junk  # (what an output's memory is likely to hold)
    o, lse = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), cu_seqlens=cu, max_seqlen=N)
    assert torch.equal(o[7:19], part[0]) and torch.equal(lse[:, 7:19], part[1])
    rest = list(range(7)) + list(range(19, 25))
    assert (o[rest] == 0).all() and (lse[:, rest] == -INF).all()
    out = torch.full_like(o, 3.0), torch.full_like(lse, 5.0)
    fa.tree_attention(q, h.cache, h.layer, ints(h.slots), cu_seqlens=cu, max_seqlen=N, out=out)
    assert torch.equal(out[0][7:19], part[0]) and (out[0][rest] == 3).all() and (out[1][:, rest] == 5).all()
    h.cache.check()


@pytest.mark.gpu
def test_a_slot_read_by_several_sequences():
    h = Held([300], 1, 128, 16)
    q = queries(6, 2, 128)
    one, _ = fa.tree_attention(q[:2].contiguous(), h.cache, h.layer, ints(h.slots))
    three, _ = fa.tree_attention(q[:2].repeat(3, 1, 1), h.cache, h.layer, ints(h.slots * 3))
    for i in range(3):  # (split over the CTAs elsewhere, so not bit for bit)
        assert torch.allclose(three[2 * i:2 * i + 2].float(), one.float(), rtol=2.0 ** -6, atol=2.0 ** -7)


@pytest.mark.gpu
def test_refused_on_the_device():
    """A sequence that does not fit has rows that see nothing; the others are right."""
    h = Held([50, 300, 20], 2, 64, 16)
    q = queries(9, 4, 64)
    cu = ints([0, 3, 6, 9])

    def wrong(first, bits, slots=None, boundaries=cu, N=3):
        o, lse = fa.tree_attention(q, h.cache, h.layer, slots if slots is not None else ints(h.slots),
                                   cu_seqlens=boundaries, max_seqlen=N)
        with pytest.raises(fa.FAError, match=bits):
            h.cache.check()
        assert not o[:first].any() and lse[:, :first].eq(-INF).all()
        return o, lse

    for bad in (-1, 77):
        o, lse = wrong(3, "out of range", slots=ints([bad] + h.slots[1:]))
        ref = run(h, q, [3, 3, 3])
        assert torch.allclose(o[3:].float(), ref[0][3:].float(), rtol=2.0 ** -6, atol=2.0 ** -7)
    keep = h.cache.lengths.clone()
    for n in (2, -5, 10 ** 6):
        h.cache.lengths[h.slots[0]] = n
        wrong(3, "does not fit")
    h.cache.lengths.copy_(keep)
    wrong(9, "does not fit", N=2)                         # longer than the bound
    o, _ = wrong(0, "does not fit", boundaries=ints([0, 3, 2, 9]), N=7)
    o, _ = wrong(0, "does not fit", boundaries=ints([0, 3, 6, 90]), N=90)
    first = int(h.table[h.slots[0], 0])
    h.cache.table[h.slots[0], 0] = 10 ** 6                # a page that is none
    fa.tree_attention(q, h.cache, h.layer, ints(h.slots), cu_seqlens=cu, max_seqlen=3)
    with pytest.raises(fa.FAError, match="out of range"):
        h.cache.check()
    h.cache.table[h.slots[0], 0] = first
    check(h, [3, 3, 3], q, run(h, q, [3, 3, 3]))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d", [(4, 2, 64), (32, 1, 64), (80, 1, 128), (6, 2, 192)])
@pytest.mark.parametrize("cu,N", [([0, 3, 6, 90], 90), ([4, 3, 6, 9], 3), ([-2, 3, 6, 9], 5),
                                  ([0, 5, 2, 2], 5), ([3, 5, 4, 6], 2), ([0, 0, 2 ** 31 - 1, 9], 9),
                                  ([1, 3, 3, 10], 7), ([-5, -1, 12, 20], 13)])
def test_boundaries_that_are_none(cu, N, Hq, heads, d):
    """A sequence whose boundaries decrease or leave the batch owns no tokens: they come out
    empty, or stay as they are where the caller asks for that; the other sequences' are right."""
    T = 9
    h = Held([50, 300, 20], heads, d, 16, seed=11)
    q = queries(T, Hq, d)
    good = [i for i in range(3) if 0 <= cu[i] <= cu[i + 1] <= T]
    names = [[i for i in good if cu[i] <= t < cu[i + 1]] for t in range(T)]
    rest = [t for t in range(T) if not names[t]]
    ws = torch.empty(fa.lib().fa_tree_workspace_size(Hq, heads, N, d), dtype=torch.uint8).cuda()
    slots, bounds = ints(h.slots), ints(cu)
    for zero_rest in (1, 0):
        o = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16).cuda()
        lse = torch.full((Hq, T), 7.0).cuda()
        assert fa.lib().fa_tree_fwd(
            h.cache._at, h.layer, slots.data_ptr(), 3, N, bounds.data_ptr(), T, q.data_ptr(), Hq, Hq * d,
            d, None, 0, o.data_ptr(), lse.data_ptr(), d ** -0.5, zero_rest, ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream) == fa.FA_OK
        with pytest.raises(fa.FAError, match="does not fit"):
            h.cache.check()
        assert (o[rest] == (0 if zero_rest else 7)).all()
        assert (lse[:, rest] == (-INF if zero_rest else 7)).all()
        for i in good:  # (a token that two sequences name holds either's row)
            once = [t for t in range(cu[i], cu[i + 1]) if names[t] == [i]]
            if once:
                see = visible(cu[i + 1] - cu[i], h.lengths[i])[[t - cu[i] for t in once]]
                ro, rl, bo, bl = attend(f64(q[once]), h.k[i], h.v[i], see, d ** -0.5)
                within("o", f64(o[once]), ro, bo)
                within("lse", f64(lse[:, once]), rl, bl)


@pytest.mark.gpu
def test_tensor_api_refuses():
    h = Held([50, 300], 2, 64, 16)
    q, s = queries(6, 4, 64), ints(h.slots)
    go = lambda q=q, layer=h.layer, s=s, **kw: fa.tree_attention(q, h.cache, layer, s, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="multiple"):
        go(q=q[:, :3])
    with pytest.raises(ValueError, match="head dimension"):
        go(q=queries(6, 4, 128))
    with pytest.raises(ValueError, match="bfloat16"):
        go(q=q.float())
    with pytest.raises(ValueError, match="max_seqlen"):
        go(cu_seqlens=ints([0, 3, 6]))
    for bound in (-1, 2 ** 31, 2 ** 33):
        with pytest.raises(ValueError, match="max_seqlen must"):
            go(cu_seqlens=ints([0, 3, 6]), max_seqlen=bound)
    with pytest.raises(ValueError, match="different sizes"):
        go(cu_seqlens=ints([0, 6]), max_seqlen=6)
    with pytest.raises(ValueError, match="B \\* N"):
        go(q=q[:5])
    with pytest.raises(ValueError, match="mask"):
        go(mask=torch.zeros(5, 1, dtype=torch.int64).cuda())
    with pytest.raises(ValueError, match="mask"):
        go(q=queries(130, 4, 64), mask=torch.zeros(130, 1, dtype=torch.int64).cuda())
    with pytest.raises(ValueError, match="out must"):
        go(out=(torch.empty_like(q), torch.empty(6, 4).cuda()))
    with pytest.raises(ValueError, match="layer"):
        go(layer=5)
    with pytest.raises(ValueError, match="on cuda"):
        go(s=s.cpu())
    with pytest.raises(fa.FAError, match="INVALID"):
        go(workspace=torch.empty(1000, dtype=torch.uint8).cuda())
    with pytest.raises(fa.FAError, match="UNSUPPORTED"):
        go(scale=0.0)
    assert go(q=q[:0])[0].shape == (0, 4, 64)


@pytest.mark.gpu
def test_lost_gradients_are_refused_on_the_device():
    """And nothing is lost where no gradient is wanted."""
    cache, slots = fa.PagedCache.allocate(1, 3, 2, 16, 64, 2, 2), ints([0, 1])
    table = fa.rotary_table(64, 9)
    append, attend, leaf = refuses_lost_gradients(cache, slots, table)
    cache.reserve(slots, 1)
    with torch.no_grad():
        q = append(k=leaf, v=leaf, q=leaf, rotary=table.clone().requires_grad_())
        assert attend(q=leaf)[0].shape == q.shape and not q.requires_grad
    with forward_ad.dual_level():
        attend(q=leaf.detach())
    cache.check()


@pytest.mark.gpu
def test_refusals_do_not_depend_on_the_stream():
    h = Held([20], 2, 64, 16)
    side, s, x = torch.cuda.Stream(), ints(h.slots), torch.zeros(1, 2, 64).bfloat16()
    tab = fa.rotary_table(64, 32)
    for kw in ({}, dict(stream=side)):
        with pytest.raises(ValueError, match="must be on"):
            fa.tree_attention(x, h.cache, 0, s, **kw)
        with pytest.raises(ValueError, match="must be on"):
            fa.cache_append(h.cache, 0, s, x, x.cuda(), **kw)
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            fa.cache_append(h.cache, 0, s, x.cuda(), [1.0], **kw)
        with pytest.raises(TypeError, match="must be a PagedCache"):
            fa.cache_append(None, 0, s, x.cuda(), x.cuda(), **kw)
        with pytest.raises(ValueError, match="int32"):
            h.cache.free(s.long(), **kw)
        with pytest.raises((TypeError, ValueError)):
            fa.rotary(x.cuda(), [1.0], tab, batch=1, **kw)
        with pytest.raises(ValueError, match="must be on"):
            fa.rotary(x.cuda(), None, tab, positions=torch.zeros(1, dtype=torch.int32), **kw)
    side.synchronize()
    h.cache.check()


@pytest.mark.gpu
def test_results_do_not_vary():
    counts = [30, 1, 64]
    h = Held([5030, 9000, 700], 2, 128, 64, layers=1, layer=0)
    q = queries(sum(counts), 8, 128)
    ref = run(h, q, counts)
    for _ in range(10):
        got = run(h, q, counts)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    """A captured call follows the lengths as they are at each replay; two graphs with a workspace
    each, and one shared between replays that do not overlap."""
    h = Held([300, 500], 2, 128, 16)
    q, s = queries(2, 4, 128), ints(h.slots)
    ws = torch.empty(fa.lib().fa_tree_workspace_size(4, 2, 1, 128), dtype=torch.uint8).cuda()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa.tree_attention(q, h.cache, h.layer, s, workspace=ws)
        graphs.append((graph, out))
    full = list(h.lengths)
    for cut in (0, 17, 299, 130):
        h.lengths = [n - cut for n in full]
        h.cache.lengths[s.long()] = ints(h.lengths)
        for graph, out in graphs:
            graph.replay()
        for graph, out in graphs:
            kk, vv = h.k, h.v
            h.k = [x[:n] for x, n in zip(kk, h.lengths)]
            h.v = [x[:n] for x, n in zip(vv, h.lengths)]
            check(h, [1, 1], q, out)
            h.k, h.v = kk, vv
    h.cache.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.tree_attention(q, h.cache, h.layer, s, stream=side)
    side.synchronize()
    assert torch.equal(got[0], graphs[0][1][0])


@pytest.mark.gpu
def test_tree_masks():
    cu = ints([0, 4, 4, 7])
    mask = fa.tree_mask(ints([-1, 0, 0, 2, -1, 9, 1, 3, 3]), cu_seqlens=cu, max_seqlen=4)
    # the second sequence's entry 9 is no earlier token: its walk ends there; no sequence owns the last two
    assert mask.flatten().tolist() == [1, 3, 5, 13, 1, 2, 6, 0, 0]
    chain = ints(list(range(-1, 199)))
    mask = fa.tree_mask(chain, batch=1)
    assert torch.equal(mask, words_of([list(range(t + 1)) for t in range(200)], 4))
    assert fa.tree_mask(chain[:0], batch=0).shape == (0, 1)
    with pytest.raises(ValueError, match="int32"):
        fa.tree_mask(chain.long(), batch=1)
    with pytest.raises(ValueError, match="CUDA"):
        fa.tree_mask(chain.cpu(), batch=1)


@pytest.mark.gpu
def test_a_drafted_step():
    """Prompt, branches, a drafted tree with its own rotary positions, acceptance, and a next token:
    every output is that of the plain attention over the tokens that stand at the end."""
    d, heads, Hq, layers = 64, 2, 4, 2
    cache = fa.PagedCache.allocate(layers, 40, heads, 16, d, 6, 10)
    for x in (cache.k, cache.v):
        x.fill_(NAN)
    table = fa.rotary_table(d, 200)
    g = torch.Generator().manual_seed(6)
    made = {}                                   # (slot, layer) -> lists of turned k and of v

    def tokens(slots, counts, positions=None, mask=None):
        cu = ints(np.cumsum([0] + counts).tolist())
        cache.reserve(ints(slots), ints(counts))
        for layer in range(layers):
            x = torch.randn(sum(counts), Hq + 2 * heads, d, generator=g).bfloat16().cuda()
            q, k, v = x[:, :Hq], x[:, Hq:Hq + heads], x[:, Hq + heads:]
            old = [len(made.get((s, layer), ([], []))[0]) for s in slots]
            pos = positions if positions is not None else torch.cat(
                [torch.arange(o, o + n) for o, n in zip(old, counts)]).cuda()
            qr = fa.cache_append(cache, layer, ints(slots), k, v, q=q, rotary=table, cu_seqlens=cu,
                                 positions=pos)
            o, lse = fa.tree_attention(qr, cache, layer, ints(slots), mask=mask, cu_seqlens=cu,
                                       max_seqlen=max(counts))
            q2, kr = fa.rotary(q, k, table, positions=pos)
            assert torch.equal(q2, qr)
            t = 0
            for s, n in zip(slots, counts):
                kk, vv = made.setdefault((s, layer), ([], []))
                kk += list(f64(kr[t:t + n]))
                vv += list(f64(v[t:t + n]))
                see = visible(n, len(kk))
                if mask is not None:
                    see[:, -n:] = (mask[t:t + n, :1].cpu().numpy() >> np.arange(n)) & 1
                ro, rl, bo, bl = attend(f64(qr[t:t + n]), np.stack(kk), np.stack(vv), see, d ** -0.5)
                within("o", f64(o[t:t + n]), ro, bo)
                within("lse", f64(lse[:, t:t + n]), rl, bl)
                t += n

    tokens([0, 1], [37, 16])
    cache.fork(ints([0, 0, 1]), ints([2, 3, 4]))
    for a, b in ((0, 2), (0, 3), (1, 4)):
        for layer in range(layers):
            made[(b, layer)] = tuple(list(x) for x in made[(a, layer)])
    parents = [-1, 0, 0, 1, 2, 4]
    rows = [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [0, 2, 4, 5]]
    depth = torch.tensor([len(r) - 1 for r in rows])
    mask = fa.tree_mask(ints(parents * 3), batch=3)
    assert torch.equal(mask, words_of(rows * 3, 1))
    tokens([3, 2, 4], [6, 6, 6], positions=torch.cat([37 + depth, 37 + depth, 16 + depth]).cuda(), mask=mask)
    cache.accept(ints([3, 2, 4]), ints([37, 37, 16]), ints([[0, 2, 4, 5], [0, 1, 3, 0], [0, 0, 0, 0]]),
                 ints([4, 3, 1]))
    for s, base, keep in ((3, 37, [0, 2, 4, 5]), (2, 37, [0, 1, 3]), (4, 16, [0])):
        for layer in range(layers):
            made[(s, layer)] = tuple(x[:base] + [x[base + j] for j in keep] for x in made[(s, layer)])
    tokens([0, 1, 2, 3, 4], [1, 1, 1, 1, 1])
    cache.free(ints([0, 1, 2, 3, 4]))
    cache.check()
    assert not cache.refs.any() and cache.table.eq(-1).all()


@pytest.mark.gpu
def test_far_pages():
    """Pages whose offsets pass 2^31 elements, written, attended to, copied and moved."""
    heads, d, ps, pages = 8, 256, 128, 8200       # 2^18 elements a page
    cache = fa.PagedCache.allocate(1, pages, heads, ps, d, 3, 4)
    far = [pages - 1, pages - 2, pages - 3]
    cache.refs[:pages - 3] = 1                    # (so that new pages are far ones)
    g = torch.Generator().manual_seed(1)
    n = 150
    cache.reserve(ints([0]), n)
    assert cache.table[0, :2].tolist() == [pages - 3, pages - 2]
    k, v = (torch.randn(n, heads, d, generator=g).bfloat16().cuda() for _ in range(2))
    fa.cache_append(cache, 0, ints([0]), k, v)
    q = queries(n, heads, d)
    o, lse = fa.tree_attention(q, cache, 0, ints([0]))
    pick = [0, 1, 128, 149]
    ro, rl, bo, bl = attend(f64(q)[pick], f64(k), f64(v), visible(n, n)[pick], d ** -0.5)
    within("o", f64(o)[pick], ro, bo)
    within("lse", f64(lse)[:, pick], rl, bl)
    cache.fork(ints([0]), ints([2]))
    assert cache.table[2, :2].tolist() == [pages - 3, far[0]]
    assert torch.equal(cache.k[0, far[0], :, :n - 128], cache.k[0, far[1], :, :n - 128])
    cache.accept(ints([2]), ints([129]), ints([[0, 20]]), ints([2]))
    assert torch.equal(cache.v[0, far[0], :, 2], v[149])
    cache.check()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [5, 64, 5000])
def test_a_bound_far_above_the_tokens(N):
    """max_seqlen may be any bound: row tiles larger than the whole batch, masks with spare words."""
    h = Held([40, 133], 2, 64, 16, seed=5)
    q = queries(7, 2, 64)
    check(h, [2, 5], q, run(h, q, [2, 5], N=N))
    rows = [[0], [1], [0], [0, 1], [2], [1, 3], [4]]
    mask = words_of(rows, -(-N // 64))
    got = fa.tree_attention(q, h.cache, h.layer, ints(h.slots), mask=mask, cu_seqlens=ints([0, 2, 7]),
                            max_seqlen=N)
    check(h, [2, 5], q, got, rows)


@pytest.mark.gpu
def test_calls_back_to_back():
    """Calls of different shapes on one workspace, one after the other without waiting: what one
    leaves in it does not reach the next."""
    a = Held([3000, 900], 2, 128, 64, seed=1, layers=1, layer=0)
    b = Held([70, 5, 4100, 260], 1, 64, 16, seed=2, layers=1, layer=0)
    qa, qb = queries(2, 16, 128), queries(120, 4, 64)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8).cuda()
    ra = run(a, qa, [1, 1], dense=True)
    rb = fa.tree_attention(qb, b.cache, 0, ints(b.slots))
    outs = []
    for _ in range(20):
        outs.append((fa.tree_attention(qa, a.cache, 0, ints(a.slots), workspace=ws), ra))
        outs.append((fa.tree_attention(qb, b.cache, 0, ints(b.slots), workspace=ws), rb))
    for got, ref in outs:
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    a.cache.check()
    # sequence 1 of b holds fewer tokens than the call's 30: reported, and its rows see nothing
    with pytest.raises(fa.FAError, match="does not fit"):
        b.cache.check()
    assert not rb[0][30:60].any()


@pytest.mark.gpu
def test_two_calls_at_once():
    """Two streams read one cache at the same time."""
    h = Held([5000, 77, 3000, 900], 2, 128, 16, seed=3, layers=1, layer=0)
    q = queries(4, 8, 128)
    s = ints(h.slots)
    ref = fa.tree_attention(q, h.cache, 0, s)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for x in streams:
        x.wait_stream(torch.cuda.current_stream())
    outs = [fa.tree_attention(q, h.cache, 0, s, stream=x) for _ in range(10) for x in streams]
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    check(h, [1] * 4, q, ref)
    h.cache.check()
