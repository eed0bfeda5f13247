"""Causal attention within a sliding window and a few first keys, forward and backward, against a 64-bit
implementation: windows and sinks on and off tile boundaries, all head dimensions and layouts, dense
and packed batches, queries and keys of different lengths, rows that see nothing, and what is refused.

Bounds count roundings: half a step of bf16 (2^-8) for each of P and dS as they enter the tensor core
and for O inside D, fp32 sums, and the stored result's own half step."""
import ctypes
import math

import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild

B16, U32 = 2.0 ** -8, 2.0 ** -24
HALF = {torch.bfloat16: B16, torch.float32: U32}
FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


# ------------------------------------------------------------------------ refusals (CPU)


def _fwd_args(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, dt=0, lse=FAKE, B=1, Hq=2, Hkv=2, Nq=200, tq=200, Nk=200,
             tk=200, d=64, scale=0.125, window=50, sinks=4, cu_q=None, cu_k=None, ws=FAKE,
             ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), 1), (dict(window=-5), 1), (dict(sinks=-1), 1), (dict(d=80), 2), (dict(q=None), 1),
    (dict(scale=-1.0), 2), (dict(Hq=3), 1), (dict(ws_bytes=100), 1), (dict(cu_q=FAKE), 1), (dict(dt=7), 1),
    (dict(tk=100), 1), (dict(o=FAKE + 4), 1)])
def test_bad_forward_calls_are_refused(kw, status):
    assert fa.lib().fa_fwd_window(*_fwd_args(**kw).values()) == status


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), 1), (dict(sinks=-1), 1), (dict(ws_bytes=1000), 1), (dict(d=100), 2), (dict(lse=None), 1),
    # far units of so many sinks do not fit the list's 16 bits
    (dict(Nq=8000000, tq=8000000, Nk=8000000, tk=8000000, sinks=8000000 - 200, Hq=1, Hkv=1, window=9), 2)])
def test_bad_backward_calls_are_refused(kw, status):
    a = _fwd_args(**kw)
    order = [a["q"], a["k"], a["v"], FAKE, a["lse"], FAKE, FAKE, FAKE, FAKE, a["dt"], a["ws"], a["ws_bytes"]] + \
        [a[n] for n in ("B", "Hq", "Hkv", "Nq", "tq", "Nk", "tk", "d", "scale", "window", "sinks", "cu_q", "cu_k")]
    assert fa.lib().fa_bwd_window(*order, 0, None) == status
    pre = [a["o"], a["dt"], FAKE, FAKE if a["lse"] else None, a["ws"], a["ws_bytes"]] + \
        [a[n] for n in ("B", "Hq", "Hkv", "Nq", "tq", "Nk", "tk", "d", "window", "sinks", "cu_q", "cu_k")]
    assert fa.lib().fa_bwd_window_preprocess(*pre, 0, None) == status


def test_workspaces():
    size = fa.fa_bwd_window_workspace_size
    plain = fa.fa_bwd_kv_workspace_size(2, 8, 4, 1000, 2000, 1000, 2000, 64)
    assert size(2, 8, 4, 1000, 2000, 1000, 2000, 64, 100, 0) == plain
    assert size(2, 8, 4, 1000, 2000, 1000, 2000, 64, 1000, 4) == plain      # nothing is hidden
    assert size(2, 8, 4, 1000, 2000, 1000, 2000, 64, 100, 1000) == plain
    assert plain < size(2, 8, 4, 1000, 2000, 1000, 2000, 64, 100, 4)
    assert size(2, 8, 4, 1000, 2000, 1000, 2000, 64, 0, 4) == 0 == size(2, 8, 4, 1000, 2000, 1000, 2000, 64, 9, -1)


def test_tensor_calls_refuse(monkeypatch):
    x = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    lse = torch.zeros(2, 8)
    monkeypatch.setattr(fa, "_check_inputs", lambda *a, **k: None)
    calls = [lambda **k: fa.forward(x, x, x, batch=1, **k), lambda **k: fa.attention(x, x, x, batch=1, **k),
             lambda **k: fa.backward(x, x, x, x, x, lse, batch=1, **k)]
    for call in calls:
        with pytest.raises(ValueError, match="causal"):
            call(window=3)
        with pytest.raises(ValueError, match="sinks need a window"):
            call(causal=True, sinks=3)
        for bad in (0, -1, 2.5, 2 ** 31):
            with pytest.raises(ValueError, match="window must be"):
                call(causal=True, window=bad)
        for bad in (-1, 0.5, 2 ** 31):
            with pytest.raises(ValueError, match="sinks must be"):
                call(causal=True, window=3, sinks=bad)


# --------------------------------------------------------------------------------- GPU


def reference(q, k, v, do, W, S, scale):
    """One sequence, float64 tensors [n, H, d]: outputs and the bounds of their bf16-operand forms."""
    n, hq, d = q.shape
    m, g = k.shape[0], hq // k.shape[1]
    p = torch.arange(n, device=q.device)[:, None] + (m - n)
    c = torch.arange(m, device=q.device)[None]
    see = (c <= p) & ((p - c < W) | (c < S))
    out = {x: torch.zeros_like(y) for x, y in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    bound = {x: torch.zeros_like(y) for x, y in out.items()}
    lse = torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    bl = torch.zeros_like(lse)
    for h in range(hq if m else 0):
        kk, vv, qq, dd = k[:, h // g], v[:, h // g], q[:, h], do[:, h]
        s = (qq @ kk.t()) * scale
        s[~see] = -math.inf
        lse[h] = torch.logsumexp(s, 1)
        pr = torch.exp(s - lse[h][:, None].nan_to_num(neginf=0.0))
        # relative error of a probability: the score's sum of d products, the exponential, the
        # sum over the keys
        ds_ = scale * 2 * d * U32 * (qq.abs() @ kk.abs().t()).amax(1) + 4 * U32 * lse[h].nan_to_num(neginf=0.0).abs()
        rel = (2 * ds_ + 8 * U32 + 2 * m * U32)[:, None]
        bl[h] = rel[:, 0] + 4 * U32 * (1 + lse[h].nan_to_num(neginf=0.0).abs())
        o = pr @ vv
        mag = pr @ vv.abs()
        out["o"][:, h] = o
        bound["o"][:, h] = (B16 * (1 + rel) + rel) * mag
        dp = dd @ vv.t()
        dm = dd.abs() @ vv.abs().t()
        D = (dd * o).sum(1, keepdim=True)
        Dm = (dd * o).abs().sum(1, keepdim=True)
        ds = pr * (dp - D)
        # P enters as bf16 (B16), dS is rounded to bf16 (B16); D is made of the stored O (its
        # bound and its half step), dP of d products in fp32
        bO = bound["o"][:, h] + B16 * o.abs()
        eD = (dd.abs() * bO).sum(1, keepdim=True) + 2 * d * U32 * Dm
        e = (2 * B16 + B16 * B16 + rel) * ds.abs() + (1 + 2 * B16) * pr * (eD + 2 * d * U32 * dm)
        out["dq"][:, h] = scale * (ds @ kk)
        bound["dq"][:, h] = scale * ((e + 2 * m * U32 * ds.abs()) @ kk.abs())
        out["dk"][:, h // g] += scale * (ds.t() @ qq)
        bound["dk"][:, h // g] += scale * ((e + 2 * n * U32 * ds.abs()).t() @ qq.abs())
        out["dv"][:, h // g] += pr.t() @ dd
        bound["dv"][:, h // g] += ((B16 + rel + 2 * n * U32) * pr).t() @ dd.abs()
    return out, bound, lse, bl


def check(name, got, ref, bound, dtype):
    over = (got.double() - ref).abs() - (bound + HALF[dtype] * (ref.abs() + bound))
    assert torch.isfinite(got).all(), name
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 0, f"{name}: {worst:.3e} beyond its bound"


def make(lq, lk, hq, hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    return r(sum(lq), hq, d), r(sum(lk), hkv, d), r(sum(lk), hkv, d), r(sum(lq), hq, d)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ends(x):
    return ints([0] + torch.tensor(x).cumsum(0).tolist())


def layout(lq, lk):
    if len(set(lq)) == 1 and len(set(lk)) == 1:
        return dict(batch=len(lq))
    kw = dict(cu_seqlens=ends(lq), max_seqlen=max(lq) + 3)
    if lq != lk:
        kw.update(cu_seqlens_k=ends(lk), max_seqlen_k=max(lk) + 5)
    return kw


def run(lq, lk, hq, hkv, d, W, S, det=False, dtype=torch.bfloat16, scale=None, seed=0):
    q, k, v, do = make(lq, lk, hq, hkv, d, seed)
    scale = 1 / math.sqrt(d) if scale is None else scale
    kw = dict(causal=True, scale=scale, window=W, sinks=S, **layout(lq, lk))
    o, lse = fa.forward(q, k, v, out_dtype=dtype, **kw)
    got = dict(zip(("dq", "dk", "dv"), fa.backward(q, k, v, o, do, lse, deterministic=det, grad_dtype=dtype,
                                                   check_status=True, **kw)), o=o)
    t = u = 0
    for i, (n, m) in enumerate(zip(lq, lk)):
        if n:
            ref, bound, rl, bl = reference(*(x.double() for x in (q[t:t + n], k[u:u + m], v[u:u + m], do[t:t + n])),
                                           W, S, scale)
            for x in ("o", "dq"):
                check(f"{x} of {i}", got[x][t:t + n], ref[x], bound[x], dtype)
            for x in ("dk", "dv"):
                check(f"{x} of {i}", got[x][u:u + m], ref[x], bound[x], dtype)
            mine = lse[:, t:t + n].double()
            assert torch.equal(torch.isinf(mine), torch.isinf(rl))
            ok = ~torch.isinf(rl)
            assert ((mine - rl).abs() - bl)[ok].max() <= 0 if ok.any() else True
        else:
            assert not got["dk"][u:u + m].any() and not got["dv"][u:u + m].any()
        t, u = t + n, u + m
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("W,S", [(1, 0), (1, 1), (2, 5), (50, 0), (127, 4), (128, 0), (128, 128), (129, 129),
                                 (200, 300), (256, 16), (300, 1), (639, 0), (5, 639)])
def test_windows_and_sinks(W, S):
    run([640], [640], 2, 2, 64, W, S)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 2), (4, 1)])
@pytest.mark.parametrize("det", [False, True])
def test_head_layouts(d, hq, hkv, det):
    run([700, 1, 333], [700, 1, 333], hq, hkv, d, 150, 7, det, seed=d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("W,S", [(40, 3), (200, 0), (130, 260)])
@pytest.mark.parametrize("det", [False, True])
def test_separate_lengths(d, W, S, det):
    """Queries behind earlier keys, alone, more than keys (rows that see nothing), and none."""
    run([100, 1, 500, 0, 260, 3], [700, 300, 200, 129, 260, 0], 4, 2, d, W, S, det, seed=d + W)


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([1], [513]), ([128], [128]), ([129] * 3, [129] * 3),
                                   ([257] * 2, [600] * 2), ([300], [20]), ([255, 256], [255, 256])])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths(lq, lk, d):
    run(lq, lk, 2, 1, d, 33, 2, seed=sum(lq))


@pytest.mark.gpu
@pytest.mark.parametrize("d,n", [(64, 9000), (128, 5000), (192, 4500)])
def test_several_chunks_of_far_rows(d, n):
    """Sinks whose far rows are several units each, over one and three tiles, and runs of heads."""
    run([n, 300, 2100], [n, 300, 2100], 4, 1, d, 256, 4, det=True)
    run([n], [n], 2, 2, d, 100, 300, det=False)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 256])
def test_runs_of_heads(d):
    """Enough units that one walks several query heads (bwd_head_run)."""
    run([2200] * 8, [2200] * 8, 16, 4, d, 140, 5, det=True)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [96, 128, 192])
def test_fp32_outputs(d):
    run([500, 77], [500, 77], 4, 2, d, 130, 9, dtype=torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("W", [300, 5000])
def test_nothing_hidden_is_the_causal_call(W):
    q, k, v, do = make([300, 200], [300, 200], 4, 2, 128)
    kw = dict(causal=True, cu_seqlens=ends([300, 200]), max_seqlen=300)
    o, lse = fa.forward(q, k, v, **kw)
    o2, lse2 = fa.forward(q, k, v, window=W, sinks=3, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a = fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
    b = fa.backward(q, k, v, o, do, lse, deterministic=True, window=7, sinks=W, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
def test_deterministic_runs_agree_to_the_bit(d):
    lens = [1500, 200, 3000]
    q, k, v, do = make(lens, lens, 8, 2, d)
    kw = dict(causal=True, window=400, sinks=20, cu_seqlens=ends(lens), max_seqlen=3000)
    o, lse = fa.forward(q, k, v, **kw)
    first = fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
    for _ in range(5):
        assert torch.equal(o, fa.forward(q, k, v, **kw)[0])
        again = fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.gpu
def test_gradient_against_differences():
    """The slope of L = sum(O dO) along random directions: central differences of the forward in 64 bits
    of the same formula agree with the kernel's gradients to the sum of their bounds."""
    n, d, W, S = 200, 64, 30, 3
    q, k, v, do = make([n], [n], 2, 2, d)
    x = [t.double() for t in (q, k, v)]
    kw = dict(causal=True, window=W, sinks=S, batch=1)
    o, lse = fa.forward(q, k, v, **kw)
    grads = fa.backward(q, k, v, o, do, lse, **kw)
    _, bound, _, _ = reference(*x, do.double(), W, S, 1 / 8)

    def loss(*y):
        return (reference(*y, do.double(), W, S, 1 / 8)[0]["o"] * do.double()).sum()
    g = torch.Generator(device="cuda").manual_seed(1)
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * u, x[i] - h * u
        slope = (loss(*up) - loss(*down)) / (2 * h)
        mine = (grads[i].double() * u).sum()
        room = ((bound[name] + B16 * (grads[i].double().abs() + bound[name])) * u.abs()).sum()
        assert (mine - slope).abs() <= room + 1e-5 * slope.abs() + 1e-5


@pytest.mark.gpu
def test_autograd_streams_and_rotary():
    lens = [300, 90]
    q, k, v, do = make(lens, lens, 4, 2, 64)
    kw = dict(causal=True, window=70, sinks=2, cu_seqlens=ends(lens), max_seqlen=300)
    table = fa.rotary_table(64, 512)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = fa.attention(*leaves, deterministic=True, rotary=table, **kw)
        grads = torch.autograd.grad(out, leaves, do)
    torch.cuda.current_stream().wait_stream(side)
    qr, kr = fa.rotary(q, k, table, cu_seqlens=kw["cu_seqlens"])
    o, lse = fa.forward(qr, kr, v, **kw)
    dq, dk, dv = fa.backward(qr, kr, v, o, do, lse, deterministic=True, **kw)
    assert torch.equal(out, o) and torch.equal(grads[2], dv)
    back = [t.clone().requires_grad_() for t in (q, k)]
    turned = fa.rotary(*back, table, cu_seqlens=kw["cu_seqlens"])
    for a, b in zip(torch.autograd.grad(turned, back, (dq, dk)), grads):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured_calls():
    """One capture of forward and backward, replayed on new values; two captures in turn."""
    lens = [700, 200]
    kw = dict(causal=True, window=90, sinks=5, cu_seqlens=ends(lens), max_seqlen=700)
    graphs = []
    for seed in (1, 2):
        q, k, v, do = make(lens, lens, 4, 2, 128, seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o, lse = fa.forward(q, k, v, **kw)
            fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = fa.forward(q, k, v, **kw)
            grads = fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
        graphs.append((g, (q, k, v, do), (o, lse) + grads))
    for turn in range(2):
        for g, ins, outs in graphs:
            for x, y in zip(ins, make(lens, lens, 4, 2, 128, 10 + turn)):
                x.copy_(y)
            g.replay()
            torch.cuda.synchronize()
            o, lse = fa.forward(*ins[:3], **kw)
            want = (o, lse) + fa.backward(*ins[:3], o, ins[3], lse, deterministic=True, **kw)
            assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.gpu
def test_boundaries_that_do_not_fit_are_reported():
    q, k, v, do = make([300], [300], 2, 2, 64)
    kw = dict(causal=True, window=20, sinks=4, max_seqlen=300)
    ws = torch.zeros(fa.fa_bwd_window_workspace_size(2, 2, 2, 300, 300, 300, 300, 64, 20, 4),
                     dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(2, 300, device="cuda")
    for cu in ([0, 200, 310], [0, 301, 300], [1, 5, 300]):
        with pytest.raises(fa.FAError, match="INVALID_ARG"):
            fa.backward(q, k, v, o, do, lse, workspace=ws, check_status=True, cu_seqlens=ints(cu), **kw)


@pytest.mark.gpu
def test_a_short_workspace_is_refused():
    """One of the plain call does not hold the sinks' partials."""
    q, k, v, do = make([300], [300], 2, 2, 64)
    kw = dict(causal=True, batch=1, window=20, sinks=4)
    o, lse = fa.forward(q, k, v, **kw)
    plain = torch.zeros(fa.fa_bwd_workspace_size(1, 2, 2, 300, 300, 64), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        fa.backward(q, k, v, o, do, lse, workspace=plain, **kw)
    with pytest.raises(ValueError, match="workspace"):
        fa.forward(q, k, v, workspace=plain[:100], **kw)
    size = fa.fa_bwd_window_workspace_size(1, 2, 2, 300, 300, 300, 300, 64, 20, 4)
    whole = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    a = fa.backward(q, k, v, o, do, lse, workspace=whole[:size], deterministic=True, **kw)
    b = fa.backward(q, k, v, o, do, lse, deterministic=True, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and whole[size:].eq(77).all()


@pytest.mark.gpu
def test_empty_sides():
    q, k, v, do = make([0], [50], 2, 2, 64)
    kw = dict(causal=True, window=7, sinks=1, cu_seqlens=ints([0, 0]), max_seqlen=0,
              cu_seqlens_k=ints([0, 50]), max_seqlen_k=50)
    o, lse = fa.forward(q, k, v, **kw)
    dq, dk, dv = fa.backward(q, k, v, o, do, lse, **kw)
    assert o.shape == (0, 2, 64) and not dk.any() and not dv.any()
    q, k, v, do = make([50], [0], 2, 2, 64)
    kw.update(cu_seqlens=ints([0, 50]), max_seqlen=50, cu_seqlens_k=ints([0, 0]), max_seqlen_k=0)
    o, lse = fa.forward(q, k, v, **kw)
    assert not o.any() and (lse == -math.inf).all()
    assert not fa.backward(q, k, v, o, do, lse, **kw)[0].any()


@pytest.mark.gpu
def test_two_calls_at_once():
    work = []
    for seed, lens, d, W, S in ((1, [2500, 300], 128, 200, 4), (2, [900] * 3, 64, 40, 130)):
        q, k, v, do = make(lens, lens, 4, 2, d, seed)
        kw = dict(causal=True, window=W, sinks=S, cu_seqlens=ends(lens), max_seqlen=max(lens))
        o, lse = fa.forward(q, k, v, **kw)
        work.append(((q, k, v, do), kw, (o, lse) + fa.backward(q, k, v, o, do, lse, deterministic=True, **kw),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (q, k, v, do), kw, want, stream in work:
            with torch.cuda.stream(stream):
                o, lse = fa.forward(q, k, v, **kw)
                got.append(((o, lse) + fa.backward(q, k, v, o, do, lse, deterministic=True, **kw), want))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for a, b in got for x, y in zip(a, b))


@pytest.mark.gpu
def test_more_queries_than_one_batch_index():
    """Many short sequences: far units and partials of each, dense and packed."""
    for lens in ([130] * 300, [1 + 7 * (i % 40) for i in range(400)]):
        run(lens[:40], lens[:40], 2, 1, 64, 20, 3, det=True)
        q, k, v, do = make(lens, lens, 2, 1, 64)
        kw = dict(causal=True, window=20, sinks=3, **layout(lens, lens))
        o, lse = fa.forward(q, k, v, **kw)
        whole = fa.backward(q, k, v, o, do, lse, deterministic=True, check_status=True, **kw)
        n = sum(lens[:40])
        part = dict(causal=True, window=20, sinks=3, **layout(lens[:40], lens[:40]))
        few = fa.backward(*(x[:n].contiguous() for x in (q, k, v, o, do)), lse[:, :n].contiguous(),
                          deterministic=True, **part)
        assert all(torch.equal(x[:n], y) for x, y in zip(whole, few))
