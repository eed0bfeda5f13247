"""The paged cache: page operations against a plain model, appended rows against a 64-bit rotation,
what is refused on the host and on the device."""
import ctypes
import random

import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from bwd_tiled_attention_gb300.serving import _CacheDesc
from serving_ref import CacheModel, f64, rotary_bound, rotate, within
from test_rotary import table64

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


# ------------------------------------------------------------------------- refusals (CPU)


def desc(**kw):
    a = dict(k=FAKE, v=FAKE, table=FAKE, lengths=FAKE, refs=FAKE, scratch=FAKE, layers=2, pages=10,
             heads=2, page_size=16, d=64, slots=4, max_pages=5)
    a.update(kw)
    return _CacheDesc(**a)


def ops(c):
    """Every call on a cache, with arguments that are fine apart from the cache."""
    L, at = fa.lib(), ctypes.addressof(c)
    yield L.fa_cache_reserve(at, FAKE, None, 1, 0, None)
    yield L.fa_cache_fork(at, FAKE, FAKE, 0, None)
    yield L.fa_cache_free(at, FAKE, 0, None)
    yield L.fa_cache_accept(at, FAKE, FAKE, FAKE, 1, FAKE, 0, None)
    yield L.fa_cache_append(at, 0, FAKE, 0, 0, None, 0, None, None, 0, 0, 0, FAKE, 128, 64, FAKE, 128,
                            64, 0, None, 0, None, 0, 0, None)
    yield L.fa_tree_fwd(at, 0, FAKE, 0, 0, None, 0, FAKE, 2, 128, 64, None, 0, FAKE, FAKE, 0.1, 0, FAKE,
                        1 << 30, None)


def test_nothing_to_do_is_no_error():
    assert set(ops(desc())) == {fa.FA_OK}


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=FAKE + 8), 1), (dict(table=None), 1), (dict(lengths=FAKE + 2), 1),
    (dict(refs=None), 1), (dict(scratch=None), 1), (dict(scratch=FAKE + 4), 1), (dict(layers=0), 1),
    (dict(pages=-1), 1), (dict(heads=0), 1), (dict(slots=0), 1), (dict(max_pages=0), 1),
    (dict(d=80), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2),
    (dict(heads=70000), 2), (dict(layers=40000), 2), (dict(layers=30000, pages=100000), 2),
    (dict(max_pages=1 << 27), 2)])
def test_bad_caches_are_refused(kw, status):
    assert set(ops(desc(**kw))) == {status}


def test_bad_lists_are_refused():
    L, c = fa.lib(), desc()
    at, bad = ctypes.addressof(c), fa.FA_ERR_INVALID_ARG
    assert L.fa_cache_reserve(at, FAKE, None, -1, 2, None) == bad
    assert L.fa_cache_reserve(at, FAKE, FAKE + 1, 0, 2, None) == bad
    assert L.fa_cache_reserve(at, None, None, 1, 2, None) == bad
    assert L.fa_cache_reserve(at, FAKE, None, 1, 5, None) == bad      # 5 entries, 4 slots
    assert L.fa_cache_fork(at, FAKE, None, 2, None) == bad
    assert L.fa_cache_fork(at, FAKE, FAKE, 5, None) == bad
    assert L.fa_cache_fork(at, FAKE, FAKE, -1, None) == bad
    assert L.fa_cache_free(at, None, 1, None) == bad
    assert L.fa_cache_free(at, FAKE + 2, 1, None) == bad
    assert L.fa_cache_accept(at, FAKE, FAKE, None, 1, FAKE, 2, None) == bad
    assert L.fa_cache_accept(at, FAKE, FAKE, FAKE, -1, FAKE, 2, None) == bad
    assert L.fa_cache_accept(at, FAKE, None, FAKE, 1, FAKE, 2, None) == bad
    assert L.fa_cache_check(None, None, None) == bad
    assert fa.lib().fa_cache_scratch_size(0, 1, 1) == 0
    assert fa.lib().fa_cache_scratch_size(10, 4, 5) >= 4 * (10 + 4 * 5 + 4 * 5 + 2)


@pytest.mark.parametrize("kw", [
    dict(layer=2), dict(layer=-1), dict(slots=None), dict(k=None), dict(v=None), dict(k=FAKE + 1),
    dict(q=FAKE, Hq=2), dict(rot=66), dict(rot=64, table=None), dict(rot=64, table_len=0),
    dict(T=7), dict(vt=-1), dict(cu=FAKE + 1), dict(pos_bytes=4)])
def test_bad_appends_are_refused(kw):
    a = dict(layer=0, slots=FAKE, B=2, N=3, cu=None, T=6, q=None, qo=None, Hq=0, qt=0, qh=0, k=FAKE,
             kt=128, kh=64, v=FAKE, vt=128, vh=64, rot=0, table=None, table_len=0, pos=None,
             pos_bytes=0, inter=0, stream=None)
    if "table" in kw or "table_len" in kw:
        a.update(table=FAKE, table_len=5)
    a.update(kw)
    assert fa.lib().fa_cache_append(ctypes.addressof(desc()), *a.values()) == fa.FA_ERR_INVALID_ARG


def test_tensor_api_refuses():
    k = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16)
    table, n, r = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), \
        torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.PagedCache(k, k, table, n, r)
    for args, match in (((k.float(), k, table, n, r), "bfloat16"), ((k, k[:, :2], table, n, r), "shape"),
                        ((k[..., :40].contiguous(),) * 2 + (table, n, r), "head dimension"),
                        ((k[:, :, :, :8].contiguous(),) * 2 + (table, n, r), "page size"),
                        ((k, k, table.long(), n, r), "int32"), ((k, k, table, n[:2], r), "entry a slot"),
                        ((k, k, table, n, r[:3]), "entry a slot"),
                        ((k.transpose(1, 2),) * 2 + (table, n, r), "contiguous")):
        with pytest.raises(ValueError, match=match):
            fa.PagedCache(*args)
    with pytest.raises(TypeError, match="PagedCache"):
        fa.cache_append(None, 0, n, k, k)


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """Each of them would reach the library cut to its low 32 bits."""
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    far = 2 ** 32 + 64

    def new(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    i32, f32, q = torch.int32, torch.float32, new(1, 2, 64)
    cache = fa.PagedCache.allocate(1, 4, 2, 16, 64, 3, 2, device="meta")
    one, table = new(1, dtype=i32), new(9, 32, 2, dtype=f32)
    for call in (lambda: fa.rotary(new(1, 1, far), None, table, batch=1),
                 lambda: fa.rotary(new(1, far, 2), None, table[:, :1].contiguous(), batch=1),
                 lambda: fa.rotary(q, new(1, far, 64), table, batch=1),
                 lambda: fa.rotary(q, None, new(far, 1, 2, dtype=f32), batch=1),
                 lambda: fa.rotary(q, None, table, cu_seqlens=new(far, dtype=i32)),
                 lambda: fa.tree_attention(q, cache, 0, new(far, dtype=i32)),
                 lambda: fa.tree_attention(q, cache, 0, one, mask=new(1, far, dtype=torch.int64)),
                 lambda: fa.cache_append(cache, 0, one, q, q, rotary=new(far, 32, 2, dtype=f32)),
                 lambda: fa.cache_append(cache, 0, one, q, q, q=new(1, far, 64)),
                 lambda: fa.tree_mask(new(3, dtype=i32), cu_seqlens=new(far, dtype=i32), max_seqlen=3),
                 lambda: cache.free(new(far, dtype=i32)),
                 lambda: cache.accept(one, one, new(1, far, dtype=i32), one),
                 lambda: fa.PagedCache(cache.k, cache.v, new(far, 2, dtype=i32), new(far, dtype=i32),
                                       cache.refs),
                 lambda: fa.PagedCache(cache.k, cache.v, new(3, far, dtype=i32), cache.lengths, cache.refs)):
        with pytest.raises(ValueError, match="has a dimension above 2147483647"):
            call()


def test_sizes_that_are_not_whole_are_refused(monkeypatch):
    """A fraction is no count: it must not be cut off."""
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    cache = fa.PagedCache.allocate(1, 4, 2, 16, 64, 3, 2, device="cpu")
    slots, q = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cu, table = torch.zeros(2, dtype=torch.int32), torch.zeros(9, 32, 2)
    called = []
    monkeypatch.setattr(cache, "_call", lambda name, stream, tensors, *a: called.append(a))
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    for call in (lambda: cache.reserve(slots, 1.5),
                 lambda: fa.tree_attention(q, cache, 0, slots, cu_seqlens=cu, max_seqlen=1.5),
                 lambda: fa.tree_mask(slots, cu_seqlens=cu, max_seqlen=1.5),
                 lambda: fa.rotary(q, None, table, batch=0.5)):
        with pytest.raises(ValueError, match="whole number"):
            call()
    assert not called
    cache.reserve(slots, np.int64(3))
    cache.reserve(slots, 2.0)
    cache.reserve(slots, torch.zeros(1, dtype=torch.int32))
    assert [a[2] for a in called] == [3, 2, 0]


def test_more_sequences_than_indexes_hold_are_refused():
    """Bisection adds two indexes, and loops step past the last one: both must stay within 32 bits."""
    L, many = fa.lib(), 2 ** 30 + 1
    c, no = desc(), fa.FA_ERR_UNSUPPORTED
    at = ctypes.addressof(c)
    assert set(ops(desc(slots=many))) == {no}
    assert L.fa_cache_free(at, FAKE, many, None) == no
    assert L.fa_rotary(FAKE, FAKE, 2, 128, 64, None, None, 0, 0, 0, fa.FA_BF16, 5, 64, 64, FAKE, 9, None, 0,
                       many, 0, FAKE, 0, 0, None) == no
    assert L.fa_cache_append(at, 0, FAKE, many, 0, FAKE, 5, None, None, 0, 0, 0, FAKE, 128, 64, FAKE, 128,
                             64, 0, None, 0, None, 0, 0, None) == no
    assert L.fa_tree_fwd(at, 0, FAKE, many, 5, FAKE, 5, FAKE, 2, 128, 64, None, 0, FAKE, FAKE, 0.1, 0, FAKE,
                         1 << 30, None) == no
    assert L.fa_tree_mask(FAKE, FAKE, many, 5, 5, 1, FAKE, None) == no


# ---------------------------------------------------------------------------------- GPU


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def make(layers=2, pages=40, heads=2, ps=16, d=64, slots=9, max_pages=8, seed=0):
    """An empty cache whose pages hold random rows, and its model."""
    c = fa.PagedCache.allocate(layers, pages, heads, ps, d, slots, max_pages)
    g = torch.Generator().manual_seed(seed)
    for x in (c.k, c.v):
        x.copy_(torch.randn(x.shape, generator=g).bfloat16())
    return c, CacheModel(c.k, c.v, c.table, c.lengths, c.refs)


def agree(c, m):
    assert c.table.tolist() == m.table
    assert c.lengths.tolist() == m.lengths
    assert c.refs.tolist() == m.refs
    assert np.array_equal(f64(c.k), m.k) and np.array_equal(f64(c.v), m.v)


def status(c):
    try:
        c.check()
        return 0
    except fa.FAError as e:
        text = str(e)
        return sum(b for b, w in ((1, "out of range"), (2, "does not fit"), (4, "free pages"),
                                  (8, "shared page"), (16, "gave up")) if w in text)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_random_operations(seed):
    """A long run of random operations, some of which are refused, leaves what the model leaves."""
    rnd = random.Random(seed)
    c, m = make(layers=rnd.choice([1, 3]), pages=rnd.choice([25, 60]), ps=rnd.choice([16, 32]),
                d=rnd.choice([64, 96]), seed=seed)
    refused = 0
    for step in range(60):
        some = rnd.sample(range(c.slots), rnd.randint(1, 4))
        op = rnd.choice(["reserve", "reserve", "fork", "free", "accept", "accept"])
        if op == "reserve":
            counts = [rnd.choice([0, 1, 5, 16, 30]) for _ in some]
            if rnd.random() < 0.3:
                counts = [counts[0]] * len(some)
                c.reserve(ints(some), counts[0])
            else:
                c.reserve(ints(some), ints(counts))
            bits = m.reserve(some, counts)
        elif op == "fork":
            empty = [s for s in range(c.slots) if m.lengths[s] == 0]
            kids = rnd.sample(empty, min(len(empty), rnd.randint(1, 3))) or some
            parents = [rnd.choice([s for s in range(c.slots) if s not in kids]) for _ in kids]
            c.fork(ints(parents), ints(kids))
            bits = m.fork(parents, kids)
        elif op == "free":
            c.free(ints(some + some[:1]))
            bits = m.free(some + some[:1])
        else:
            base = [rnd.randint(0, m.lengths[s]) for s in some]
            width = rnd.choice([0, 3, 20])
            path = [sorted(rnd.sample(range(60), width)) for _ in some]
            got = [sum(t < m.lengths[s] - b for t in p) for s, b, p in zip(some, base, path)]
            got = [rnd.randint(0, x) if rnd.random() < 0.8 else x for x in got]
            c.accept(ints(some), ints(base), ints(path).view(len(some), width), ints(got))
            bits = m.accept(some, base, path, got)
        assert status(c) == bits, (step, op)
        refused += bits != 0
        agree(c, m)
    assert refused < 40


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1000, 2500])
def test_many_slots_and_pages(n):
    """More entries than the planning CTA has threads, and a pool that it scans in several steps."""
    c = fa.PagedCache.allocate(1, 9000, 1, 16, 64, 2 * n, 4)
    c.k.zero_()
    c.v.zero_()
    m = CacheModel(c.k, c.v, c.table, c.lengths, c.refs)
    rnd = random.Random(n)
    first = rnd.sample(range(2 * n), n)
    counts = [rnd.randint(0, 40) for _ in first]
    c.reserve(ints(first), ints(counts))
    assert m.reserve(first, counts) == 0
    other = [s for s in range(2 * n) if s not in set(first)]
    c.fork(ints(first), ints(other))
    assert m.fork(first, other) == 0
    gone = rnd.sample(range(2 * n), n)
    c.free(ints(gone))
    m.free(gone)
    assert status(c) == 0
    agree(c, m)


@pytest.mark.gpu
def test_refused_on_the_device():
    c, m = make()
    c.reserve(ints([0, 1, 2]), ints([20, 32, 5]))
    m.reserve([0, 1, 2], [20, 32, 5])
    c.fork(ints([1]), ints([3]))
    m.fork([1], [3])
    e = ints([[0]] * 2)
    for call, bits in (
            (lambda: c.reserve(ints([0, 9]), 1), 1), (lambda: c.reserve(ints([-1, 0]), 1), 1),
            (lambda: c.reserve(ints([2, 2]), 1), 1), (lambda: c.reserve(ints([0, 1]), ints([1, -1])), 2),
            (lambda: c.reserve(ints([0]), 200), 2), (lambda: c.reserve(ints([0]), 2 ** 31 - 1), 2),
            (lambda: c.reserve(ints([0, 1, 2, 4, 5, 6]), 96), 4),
            (lambda: c.fork(ints([0]), ints([1])), 2), (lambda: c.fork(ints([0, 1]), ints([5, 5])), 1),
            (lambda: c.fork(ints([0, 5]), ints([5, 6])), 1), (lambda: c.fork(ints([0]), ints([99])), 1),
            (lambda: c.free(ints([0, 77])), 1),
            (lambda: c.accept(ints([0, 0]), ints([1, 1]), e, ints([0, 0])), 1),
            (lambda: c.accept(ints([0, 2]), ints([21, 1]), e, ints([0, 0])), 2),
            (lambda: c.accept(ints([0, 2]), ints([1, 1]), e, ints([0, 2])), 2),
            (lambda: c.accept(ints([0]), ints([1]), ints([[3, 3]]), ints([2])), 2),
            (lambda: c.accept(ints([0]), ints([1]), ints([[5, 4]]), ints([2])), 2),
            (lambda: c.accept(ints([0]), ints([1]), ints([[-1, 4]]), ints([2])), 2),
            (lambda: c.accept(ints([0]), ints([1]), ints([[4, 19]]), ints([2])), 2),
            (lambda: c.accept(ints([3]), ints([20]), ints([[2]]), ints([1])), 8),
            (lambda: c.accept(ints([3]), ints([20]), ints([[]]).view(1, 0), ints([0])), 8)):
        call()
        assert status(c) == bits
        agree(c, m)
    # dropping whole shared pages is fine, and so is going on in a page of one's own
    c.accept(ints([3]), ints([16]), ints([[]]).view(1, 0), ints([0]))
    assert m.accept([3], [16], [[]], [0]) == 0
    c.reserve(ints([3]), 7)
    assert m.reserve([3], [7]) == 0
    assert status(c) == 0
    agree(c, m)
    with pytest.raises(ValueError, match="named twice"):
        c.reserve(ints(list(range(10))), 1)
    for counts in (-1, 2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="counts must"):
            c.reserve(ints([0]), counts)
    with pytest.raises(ValueError, match="entries"):
        c.fork(ints([0]), ints([5, 6]))
    with pytest.raises(ValueError, match="int32"):
        c.free(torch.tensor([0]).cuda())
    with pytest.raises(ValueError, match="on cuda"):
        c.free(torch.tensor([0], dtype=torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("width,draft", [(1, 4), (8, 64), (21, 40), (40, 40)])
def test_accepted_rows_that_overlap(width, draft):
    """Sources and destinations interleave: every row ends where the path says, in all layers."""
    c, m = make(layers=3, pages=60, ps=16, d=128, slots=4, max_pages=12, seed=width)
    c.reserve(ints([2, 0, 3]), ints([7 + draft, draft, 33 + draft]))
    m.reserve([2, 0, 3], [7 + draft, draft, 33 + draft])
    rnd = random.Random(width)
    path = [sorted(rnd.sample(range(draft), width)) for _ in range(3)]
    got = [width, max(0, width - 1), width]
    c.accept(ints([2, 0, 3]), ints([7, 0, 33]), ints(path), ints(got))
    assert m.accept([2, 0, 3], [7, 0, 33], path, got) == 0
    assert status(c) == 0
    agree(c, m)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,heads,d,rot,ps", [(4, 2, 64, 64, 16), (6, 6, 128, 32, 64), (5, 1, 256, 256, 32),
                                               (0, 3, 96, 96, 16), (12, 4, 192, 40, 128), (2, 2, 64, 0, 16)])
def test_append(Hq, heads, d, rot, ps, interleaved):
    """Prompts of different lengths, one of them empty, then one token each; slots in any order."""
    c, m = make(layers=2, pages=30, heads=heads, ps=ps, d=d, slots=5, max_pages=20, seed=d)
    g = torch.Generator().manual_seed(d + rot)
    slots = [3, 0, 4]
    tab = table64(rot, 400) if rot else None
    dev = torch.from_numpy(tab).cuda() if rot else None
    for counts in ([37, 0, 20], [1, 1, 1], [5, 5, 5]):
        c.reserve(ints(slots), ints(counts))
        m.reserve(slots, counts)
        T = sum(counts)
        x = torch.randn(T, Hq + 2 * heads, d, generator=g).bfloat16().cuda()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + heads], x[:, Hq + heads:]
        cu = None if len(set(counts)) == 1 else ints(np.cumsum([0] + counts).tolist())
        out = fa.cache_append(c, 1, ints(slots), k, v, q=q if Hq else None, rotary=dev,
                              interleaved=interleaved, cu_seqlens=cu)
        pos = np.concatenate([np.arange(m.lengths[s] - n, m.lengths[s]) for s, n in zip(slots, counts)])
        who = np.repeat(slots, counts)
        t64 = tab.astype(np.float64) if rot else np.zeros((400, 0, 2))
        kr, mag = rotate(f64(k), t64, pos, interleaved)
        kb, vb = f64(c.k), f64(c.v)
        for i in range(T):
            page, row = m.place(who[i], int(pos[i]))
            within("k", kb[1, page, :, row], kr[i], rotary_bound(kr[i], mag[i], torch.bfloat16))
            m.k[1, page, :, row] = kb[1, page, :, row]
            m.v[1, page, :, row] = f64(v[i])
        if Hq:
            qr, mag = rotate(f64(q), t64, pos, interleaved)
            within("q", f64(out), qr, rotary_bound(qr, mag, torch.bfloat16))
        else:
            assert out is None
        assert status(c) == 0
        agree(c, m)


@pytest.mark.gpu
def test_append_positions_and_tokens_of_no_sequence():
    c, m = make(d=64)
    c.reserve(ints([5, 6]), ints([3, 4]))
    m.reserve([5, 6], [3, 4])
    g = torch.Generator().manual_seed(9)
    x = torch.randn(10, 6, 64, generator=g).bfloat16().cuda()
    q, k, v = x[:, :2], x[:, 2:4], x[:, 4:]
    tab = table64(64, 100)
    pos = torch.tensor([10, 11, 11, 99, 0, 0, 7, 5, 5, 5])
    out = fa.cache_append(c, 0, ints([5, 6]), k, v, q=q, rotary=torch.from_numpy(tab).cuda(),
                          positions=pos.cuda(), cu_seqlens=ints([0, 3, 7]))
    kr, mag = rotate(f64(k), tab.astype(np.float64), pos.numpy(), False)
    kb = f64(c.k)
    for i in range(7):
        page, row = m.place(5 if i < 3 else 6, i if i < 3 else i - 3)
        within("k", kb[0, page, :, row], kr[i], rotary_bound(kr[i], mag[i], torch.bfloat16))
        m.k[0, page, :, row], m.v[0, page, :, row] = kb[0, page, :, row], f64(v[i])
    agree(c, m)
    assert not out[7:].any() and out[:7].any()
    assert status(c) == 0


@pytest.mark.gpu
def test_append_to_no_sequence():
    """A packed batch without sequences: nothing is written, q comes out as zeros."""
    c, m = make(d=64)
    x = torch.randn(3, 2, 64).bfloat16().cuda()
    q = fa.cache_append(c, 0, ints([]), x, x, q=x, cu_seqlens=ints([0]))
    assert not q.any()
    o, lse = fa.tree_attention(x, c, 0, ints([]), cu_seqlens=ints([0]), max_seqlen=4)
    assert not o.any() and lse.eq(-float("inf")).all()
    assert status(c) == 0
    agree(c, m)


@pytest.mark.gpu
def test_append_refused_on_the_device():
    """A token without a place is not written, wherever the fault lies; the others are."""
    c, m = make(d=64)
    c.reserve(ints([0, 1]), ints([4, 2]))
    m.reserve([0, 1], [4, 2])
    k = torch.ones(3, 2, 64).bfloat16().cuda()
    tab = fa.rotary_table(64, 16)

    def put(slots, counts):
        return fa.cache_append(c, 0, ints(slots), k[:sum(counts)], k[:sum(counts)],
                               cu_seqlens=ints(np.cumsum([0] + counts).tolist()))

    put([1], [3])                               # more tokens than the slot holds
    page, _ = m.place(1, 0)
    m.k[0, page, :, :2] = m.v[0, page, :, :2] = 1.0
    assert status(c) == 2
    agree(c, m)
    put([99, 0], [1, 1])
    page, _ = m.place(0, 0)
    m.k[0, page, :, 3] = m.v[0, page, :, 3] = 1.0
    assert status(c) == 1
    agree(c, m)
    put([-5], [1])
    assert status(c) == 1
    c.table[0, 0] = 1000                        # a page that is none
    put([0], [1])
    assert status(c) == 1
    c.table[0, 0] = m.table[0][0]
    agree(c, m)
    c.lengths[0] = 10 ** 6                      # past the table
    put([0], [1])
    assert status(c) == 2
    c.lengths[0] = m.lengths[0]
    for cu in ([0, 5], [2, 1], [-3, 1]):        # boundaries that are none
        fa.cache_append(c, 0, ints([0]), k, k, cu_seqlens=ints(cu), rotary=tab)
        status(c)
    agree(c, m)
    with pytest.raises(ValueError, match="does not fit"):
        fa.cache_append(c, 0, ints([0]), k[:, :1], k)
    with pytest.raises(ValueError, match="layer"):
        fa.cache_append(c, 2, ints([0]), k, k)
    with pytest.raises(ValueError, match="positions need"):
        fa.cache_append(c, 0, ints([0]), k, k, positions=ints([0, 1, 2]))


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 5], [2, 1], [-3, 1], [0, 5, 2], [0, 3, 9], [3, 2, 3], [-4, -2, 0],
                                [0, 2, 1, 3], [3, 3, 3, 90, 90]])
@pytest.mark.parametrize("d,interleaved", [(64, False), (64, True), (96, False)])
def test_append_reports_boundaries_that_are_none(cu, d, interleaved):
    """Wherever boundaries decrease or leave the batch, whether or not a token lies between them."""
    c, m = make(d=d)
    slots = [4, 0, 6, 2][:len(cu) - 1]
    c.reserve(ints(slots), 40)
    m.reserve(slots, [40] * len(slots))
    x = torch.randn(3, 2, d).bfloat16().cuda()
    tab = fa.rotary_table(32, 64)
    q = fa.cache_append(c, 1, ints(slots), x, x, q=x, rotary=tab, interleaved=interleaved,
                        cu_seqlens=ints(cu))
    assert status(c) == 2
    assert q.shape == x.shape
    # nothing but the sequences' own last rows can have been written
    held = [m.place(s, t) for s in slots for t in range(37, 40)]
    for mine, theirs in ((f64(c.k), m.k), (f64(c.v), m.v)):
        other = np.ones(mine.shape, bool)
        for page, row in held:
            other[1, page, :, row] = False
        assert np.array_equal(mine[other], theirs[other])
    # a batch that is fine reports nothing
    fa.cache_append(c, 1, ints(slots[:1]), x, x, q=x, rotary=tab, cu_seqlens=ints([0, 3]))
    assert status(c) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 96])
def test_append_leaves_shared_pages(d):
    """After a fork the whole pages belong to both: rows of theirs are refused, the page that was
    copied is not, and once the other sequence is gone they are written again."""
    c, m = make(d=d)
    c.reserve(ints([4]), ints([20]))
    c.fork(ints([4]), ints([7]))
    m.reserve([4], [20])
    m.fork([4], [7])
    k = torch.ones(6, 2, d).bfloat16().cuda()
    q = fa.cache_append(c, 1, ints([7]), k, k, q=k)
    page, _ = m.place(7, 16)
    m.k[1, page, :, :4] = m.v[1, page, :, :4] = 1.0
    assert status(c) == 8
    agree(c, m)
    assert torch.equal(q, k)
    c.free(ints([4]))
    m.free([4])
    fa.cache_append(c, 1, ints([7]), k, k)
    page, _ = m.place(7, 14)
    m.k[1, page, :, 14:] = m.v[1, page, :, 14:] = 1.0
    assert status(c) == 0
    agree(c, m)


@pytest.mark.gpu
def test_captured_page_operations():
    """reserve, append, fork, accept and free in one graph, replayed, on lengths that change."""
    c, m = make(layers=2, d=64, pages=60)
    slots, kids, base, got = ints([1, 2]), ints([7, 8]), ints([0, 0]), ints([2, 1])
    path = ints([[0, 3], [2, 3]])
    x = torch.randn(8, 2, 64).bfloat16().cuda()

    def step():
        base.copy_(c.lengths[1:3])
        c.reserve(slots, 4)
        fa.cache_append(c, 0, slots, x, x)
        c.accept(slots, base, path, got)
        c.free(kids)
        c.fork(slots, kids)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(9):
        at = [m.lengths[1], m.lengths[2]]
        graph.replay()
        m.reserve([1, 2], [4, 4])
        for i, sl in enumerate((1, 2)):
            for j in range(4):
                page, row = m.place(sl, at[i] + j)
                m.k[0, page, :, row] = m.v[0, page, :, row] = f64(x[4 * i + j])
        assert m.accept([1, 2], at, [[0, 3], [2, 3]], [2, 1]) == 0
        m.free([7, 8])
        m.fork([1, 2], [7, 8])
    assert status(c) == 0
    agree(c, m)


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [False, True])
def test_on_another_stream(as_int):
    """Every call on a side stream, given as a stream or as its handle."""
    side = torch.cuda.Stream()
    c, m = make(layers=2, d=64)
    x = torch.randn(6, 2, 64).bfloat16().cuda()
    lists = [ints(v) for v in ([3, 4], [2, 4], [5, 6], [0, 0], [1, 1])]
    slots, counts, kids, base, got = lists
    path = ints([[1], [2]])
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(stream=side.cuda_stream if as_int else side)
    c.reserve(slots, counts, **kw)
    fa.cache_append(c, 0, slots, x, x, cu_seqlens=ints([0, 2, 6]), **kw)
    c.fork(slots, kids, **kw)
    c.accept(slots, base, path, got, **kw)
    c.free(kids, **kw)
    c.check(**kw)
    m.reserve([3, 4], [2, 4])
    for s, t0, n in ((3, 0, 2), (4, 2, 4)):
        for j in range(n):
            page, row = m.place(s, j)
            m.k[0, page, :, row] = m.v[0, page, :, row] = f64(x[t0 + j])
    m.fork([3, 4], [5, 6])
    m.accept([3, 4], [0, 0], [[1], [2]], [1, 1])
    m.free([5, 6])
    agree(c, m)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["reserve", "append", "attention"])
def test_memory_is_kept_for_another_stream(call):
    """A cache dropped while a call on another stream is still to run keeps its memory until then."""
    side = torch.cuda.Stream()
    c = fa.PagedCache.allocate(1, 4096, 2, 16, 64, 4, 8)
    slots, x = ints([2]), torch.randn(1, 2, 64).bfloat16().cuda()
    c.reserve(slots, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    if call == "reserve":
        c.reserve(slots, 1, stream=side)
    elif call == "append":
        fa.cache_append(c, 0, slots, x, x, stream=side)
    else:
        fa.tree_attention(x, c, 0, slots, stream=side)
    at, shape = {c.k.data_ptr(), c.v.data_ptr()}, c.k.shape
    del c
    new = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert not side.query()
    assert not at & {t.data_ptr() for t in new}
    side.synchronize()
