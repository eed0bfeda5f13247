"""Rotary positions against a 64-bit implementation: layouts, part of the head, strides, types,
positions, gradients, and what is refused."""
import math

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from serving_ref import f64, rotary_bound, rotate, within

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


def table64(rot, length, base=10000.0):
    a = np.arange(length)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


# ------------------------------------------------------------------------- refusals (CPU)


def call(**kw):
    a = dict(q=FAKE, q_out=FAKE, Hq=4, qt=256, qh=64, k=FAKE, k_out=FAKE, Hkv=2, kt=128, kh=64,
             dtype=fa.FA_BF16, T=10, d=64, rot=64, table=FAKE, table_len=100, positions=None,
             pos_bytes=0, B=2, N=5, cu=None, interleaved=0, backward=0, stream=None)
    a.update(kw)
    return fa.lib().fa_rotary(*a.values())


@pytest.mark.parametrize("kw", [
    dict(rot=66), dict(rot=63), dict(rot=-2), dict(d=0), dict(T=-1), dict(Hq=-1), dict(qt=-1),
    dict(kh=-8), dict(table=None), dict(table_len=0), dict(table_len=-1), dict(q=None),
    dict(k_out=None), dict(dtype=5), dict(pos_bytes=4), dict(positions=FAKE), dict(B=3),
    dict(positions=FAKE, pos_bytes=2), dict(positions=FAKE + 4, pos_bytes=8), dict(q=FAKE + 1),
    dict(cu=FAKE + 2), dict(N=-5, B=-2), dict(d=70000, rot=64)])
def test_bad_arguments_are_refused(kw):
    assert call(**kw) == fa.FA_ERR_INVALID_ARG


def test_tokens_too_wide_for_the_indexes_are_refused():
    assert call(Hq=65535, Hkv=60000, d=65536) == fa.FA_ERR_UNSUPPORTED


def test_nothing_to_do_is_no_error():
    assert call(T=0, N=0) == fa.FA_OK
    assert call(Hq=0, Hkv=0, q=None, k=None) == fa.FA_OK
    assert fa.lib().fa_rotary_table(FAKE, 8, 0, 1.0, FAKE, None) == fa.FA_OK


@pytest.mark.parametrize("args", [
    (FAKE, 0, 4, 1.0, FAKE), (FAKE, 8, -1, 1.0, FAKE), (None, 8, 4, 1.0, FAKE),
    (FAKE, 8, 4, 1.0, None), (FAKE, 8, 4, 1.0, FAKE + 8), (FAKE + 4, 8, 4, 1.0, FAKE),
    (FAKE, 8, 4, math.nan, FAKE), (FAKE, 8, 1 << 40, 1.0, FAKE)])
def test_bad_table_arguments_are_refused(args):
    assert fa.lib().fa_rotary_table(*args, None) == fa.FA_ERR_INVALID_ARG


def test_tensor_api_refuses():
    q, tab = torch.zeros(6, 2, 64, dtype=torch.bfloat16), torch.zeros(9, 32, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rotary(q, q, tab, batch=2)
    with pytest.raises(ValueError, match="batch"):
        fa.rotary(q, q, tab)
    with pytest.raises(ValueError, match="B \\* N"):
        fa.rotary(q, q, tab, batch=4)
    with pytest.raises(ValueError, match="one type"):
        fa.rotary(q, q.float(), tab, batch=2)
    with pytest.raises(ValueError, match="same tokens"):
        fa.rotary(q, q[:3], tab, batch=2)
    with pytest.raises(ValueError, match="last dimension"):
        fa.rotary(q.transpose(1, 2), None, tab, batch=2)
    with pytest.raises(ValueError, match="more columns"):
        fa.rotary(q, q, torch.zeros(9, 33, 2), batch=2)
    with pytest.raises(ValueError, match="float32"):
        fa.rotary(q, q, tab.double(), batch=2)
    with pytest.raises(ValueError, match="entry a token"):
        fa.rotary(q, q, tab, positions=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="bfloat16"):
        fa.rotary(q.half(), None, tab, batch=2)
    with pytest.raises(TypeError):
        fa.rotary(None, None, tab, batch=2)
    for kw in (dict(rot=7), dict(scaling="other"), dict(factor=0.5), dict(scaling="by_parts"),
               dict(frequencies=[1.0]), dict(device="cpu"), dict(length=-1),
               dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            fa.rotary_table(**dict(dict(rot=8, length=4), **kw))
    with pytest.raises(ValueError, match="positions"):
        fa.attention(q, q, q, batch=1, rotary=tab, positions_k=torch.zeros(6, dtype=torch.int32))
    with pytest.raises(ValueError, match="rotary table"):
        fa.attention(q, q, q, batch=1, positions=torch.zeros(6, dtype=torch.int32))


def test_a_raised_base_with_frequencies_is_refused():
    with pytest.raises(ValueError, match="base"):
        fa.rotary_table(8, 4, scaling="ntk", factor=4.0, frequencies=[1.0, 0.5, 0.2, 0.1])


def test_frequencies_that_require_a_gradient_are_refused():
    f = torch.ones(4, requires_grad=True)
    with pytest.raises(ValueError, match="not differentiable"):
        fa.rotary_table(8, 4, frequencies=f)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        fa.rotary_table(8, 4, frequencies=f, device="cpu")


def refuses_forward_tangents(q, k, table):
    """A tangent must not be dropped without a word, in the rotation or in its gradient."""
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(q, torch.ones_like(q))
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                for a, b, t in ((dual, k, table), (dual, None, table), (None, dual, table),
                                (k, None, forward_ad.make_dual(table, table))):
                    with pytest.raises(NotImplementedError, match="forward"):
                        fa.rotary(a, b, t, batch=1)
                assert fa.rotary(k, None, table, batch=1)[0].shape == k.shape  # (no tangent, no error)
        x = q.clone().requires_grad_()
        y, _ = fa.rotary(x, None, table, batch=1)
        with pytest.raises(NotImplementedError, match="forward"):
            torch.autograd.grad(y, x, forward_ad.make_dual(torch.ones_like(q), torch.ones_like(q)))
    assert fa.rotary(q, None, table, batch=1)[0].shape == q.shape


def test_forward_tangents_are_refused(monkeypatch):
    monkeypatch.setattr(fa.serving, "_cuda", lambda name, t: None)
    monkeypatch.setattr(fa.serving, "_here", lambda device, stream: True)
    monkeypatch.setattr(fa.serving, "_rotate",
                        lambda q, k, *a: [None if t is None else torch.zeros(t.shape) for t in (q, k)])
    refuses_forward_tangents(torch.ones(6, 2, 64), torch.ones(6, 2, 64), torch.zeros(9, 32, 2))


# ---------------------------------------------------------------------------------- GPU


CASES = [  # T, Hq, Hkv, d, rot
    (1, 1, 1, 64, 64), (7, 4, 2, 128, 128), (33, 5, 3, 192, 64), (130, 32, 8, 128, 96),
    (19, 6, 1, 256, 256), (11, 3, 3, 40, 20), (5, 2, 2, 7, 6), (9, 9, 1, 80, 2), (4, 2, 2, 96, 0),
    (3, 1, 0, 64, 32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot", CASES)
def test_rotary_forward(T, Hq, Hkv, d, rot, interleaved, dtype):
    g = torch.Generator().manual_seed(T * 1000 + d)
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(dtype).cuda()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv] if Hkv else None   # slices of one projection
    pos = torch.randint(0, 500, (T,), generator=g)
    tab = table64(rot, 500) if rot else np.zeros((500, 0, 2), np.float32)
    dt = torch.int64 if d % 3 else torch.int32
    got = fa.rotary(q, k, torch.from_numpy(tab).cuda(), positions=pos.to(dt).cuda(),
                    interleaved=interleaved)
    for name, a, b in (("q", got[0], q), ("k", got[1], k)):
        if b is None:
            assert a is None
            continue
        assert a.is_contiguous() and a.dtype == dtype
        ref, mag = rotate(f64(b), tab.astype(np.float64), pos.numpy(), interleaved)
        within(name, f64(a), ref, rotary_bound(ref, mag, dtype))
        assert torch.equal(a[..., rot:], b[..., rot:])


@pytest.mark.gpu
def test_positions_of_sequences():
    """Without positions every sequence counts from 0; tokens behind the last one are zeros."""
    tab = table64(64, 64)
    q = torch.randn(40, 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dense, _ = fa.rotary(q, None, torch.from_numpy(tab).cuda(), batch=4)
    cu = torch.tensor([0, 3, 3, 20, 33], dtype=torch.int32).cuda()
    packed, _ = fa.rotary(q, None, torch.from_numpy(tab).cuda(), cu_seqlens=cu)
    pos = np.r_[np.arange(3), np.arange(17), np.arange(13)]
    for got, p in ((dense, np.arange(40) % 10), (packed[:33], pos)):
        ref, mag = rotate(f64(q[:len(p)]), tab.astype(np.float64), p, False)
        within("q", f64(got), ref, rotary_bound(ref, mag, torch.bfloat16))
    assert not packed[33:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 40])
def test_positions_outside_the_table(d):
    tab = torch.from_numpy(table64(32, 10)).cuda()
    q = torch.ones(4, 3, d, dtype=torch.bfloat16).cuda()
    for dt, far in ((torch.int32, 2 ** 31 - 1), (torch.int64, 2 ** 40)):
        got, _ = fa.rotary(q, None, tab, positions=torch.tensor([9, 10, -1, far], dtype=dt).cuda())
        assert torch.isfinite(got[0]).all() and got[1:, :, :32].isnan().all()
        assert torch.equal(got[:, :, 32:], q[:, :, 32:])


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_unaligned_inputs(offset):
    """Any base, token and head stride: what 16-byte accesses cannot take runs element by element."""
    tab = table64(64, 50)
    flat = torch.randn(offset + 12 * 331, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q = flat.as_strided((12, 4, 64), (331, 71, 1), offset)
    got, _ = fa.rotary(q, None, torch.from_numpy(tab).cuda(), batch=1)
    ref, mag = rotate(f64(q), tab.astype(np.float64), np.arange(12), False)
    within("q", f64(got), ref, rotary_bound(ref, mag, torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(interleaved, dtype):
    """The gradient is the transposed rotation; checked against the formula, and in fp32 against
    differences."""
    tab = table64(32, 64)
    t = torch.from_numpy(tab).cuda()
    g = torch.Generator().manual_seed(5)
    q = torch.randn(24, 3, 64, generator=g).to(dtype).cuda().requires_grad_()
    k = torch.randn(24, 1, 64, generator=g).to(dtype).cuda().requires_grad_()
    gq, gk = torch.randn(24, 3, 64, generator=g).to(dtype).cuda(), torch.randn(24, 1, 64, generator=g).to(dtype).cuda()
    a, b = fa.rotary(q, k, t, batch=2, interleaved=interleaved)
    dq, dk = torch.autograd.grad((a, b), (q, k), (gq, gk))
    pos = np.arange(24) % 12
    for name, got, up in (("dq", dq, gq), ("dk", dk, gk)):
        ref, mag = rotate(f64(up), tab.astype(np.float64), pos, interleaved, back=True)
        within(name, f64(got), ref, rotary_bound(ref, mag, dtype))
    if dtype == torch.float32:
        u = torch.randn(24, 3, 64, generator=g).cuda()
        eps = 2.0 ** -6  # the map is linear: a difference has no error but rounding
        up, _ = fa.rotary(q.detach() + eps * u, None, t, batch=2, interleaved=interleaved)
        dn, _ = fa.rotary(q.detach() - eps * u, None, t, batch=2, interleaved=interleaved)
        num = ((f64(up) - f64(dn)) / (2 * eps) * f64(gq)).sum()
        ana = (f64(dq) * f64(u)).sum()
        # each of the 4608 values rounds in 7 places of 2^-24 relative to at most ~8, over 2 eps
        assert abs(num - ana) <= 4608 ** 0.5 * 4 * 7 * 8 * 2.0 ** -24 / (2 * eps)


@pytest.mark.gpu
def test_gradients_of_one_output_and_expanded_gradients():
    t = torch.from_numpy(table64(64, 64)).cuda()
    q = torch.randn(8, 2, 64).cuda().requires_grad_()
    k = torch.randn(8, 1, 64).cuda().requires_grad_()
    a, b = fa.rotary(q, k, t, batch=1)
    a.sum().backward()                       # an expanded gradient, and none for k
    ref, mag = rotate(np.ones((8, 2, 64)), table64(64, 64).astype(np.float64), np.arange(8), False, True)
    within("dq", f64(q.grad), ref, rotary_bound(ref, mag, torch.float32))
    assert k.grad is None
    # twice: |rotary(q)|^2 = |q|^2, so the gradient is 2q and the gradient of its sum 2; each
    # value passes two rotations of magnitudes up to ~10 in fp32
    a, _ = fa.rotary(q, None, t, batch=1)
    (dq,) = torch.autograd.grad((a * a).sum(), q, create_graph=True)
    (dd,) = torch.autograd.grad(dq.sum(), q)
    assert torch.allclose(dq, 2 * q, rtol=0, atol=1e-5)
    assert torch.allclose(dd, torch.full_like(dd, 2.0), rtol=0, atol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    {}, dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="by_parts", factor=16.0, original_length=4096),
    dict(frequencies=[1.0, 0.5, 0.25, 1e-6])])
def test_tables(kw):
    """Far positions keep their phase: cos and sin are those of the 64-bit angle."""
    rot, n = 8 if "frequencies" in kw else 64, 131072
    got = f64(fa.rotary_table(rot, n, **kw))
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    scale = 1.0
    if kw.get("scaling") == "linear":
        f = f / 4
    elif kw.get("scaling") == "ntk":
        f = (10000.0 * 8.0 ** (64 / 62)) ** (-np.arange(0, 64, 2) / 64)
        assert np.isclose(f[-1] * 8, 10000.0 ** (-62 / 64)) and f[0] == 1
    elif kw.get("scaling") == "by_parts":
        turns = 4096 * f / (2 * np.pi)
        keep = np.clip((turns - 1) / 31, 0, 1)
        f = f * keep + f / 16 * (1 - keep)
        scale = 1 + 0.1 * np.log(16)
    elif "frequencies" in kw:
        f = np.array(kw["frequencies"])
    a = np.arange(n)[:, None] * f
    ref = scale * np.stack([np.cos(a), np.sin(a)], -1)
    # the frequencies may differ in their last places (powers), which a position multiplies
    within("table", got, ref, 2.0 ** -24 * np.abs(ref) + np.maximum(a, 1)[..., None] * 2.0 ** -48 + 2.0 ** -50)


@pytest.mark.gpu
def test_forward_tangents_are_refused_on_the_device():
    x = torch.randn(6, 2, 64).cuda()
    refuses_forward_tangents(x, x + 1, fa.rotary_table(64, 9))


@pytest.mark.gpu
def test_attention_with_rotary():
    """attention(rotary=) is rotary followed by attention, and so are its gradients."""
    t = fa.rotary_table(64, 200)
    g = torch.Generator().manual_seed(3)
    x = [torch.randn(300, h, 64, generator=g).bfloat16().cuda().requires_grad_() for h in (4, 2, 2)]
    cu = torch.tensor([0, 101, 300], dtype=torch.int32).cuda()
    kw = dict(causal=True, cu_seqlens=cu, max_seqlen=199, deterministic=True)
    o = fa.attention(*x, rotary=t, **kw)
    q, k = fa.rotary(x[0], x[1], t, cu_seqlens=cu)
    o2 = fa.attention(q, k, x[2], **kw)
    assert torch.equal(o, o2)
    w = torch.randn(o.shape, generator=g).bfloat16().cuda()
    for a, b in zip(torch.autograd.grad(o, x, w), torch.autograd.grad(o2, x, w)):
        assert torch.equal(a, b)
    pos = torch.cat([torch.arange(101), torch.arange(199)]).cuda()
    with torch.no_grad():
        assert torch.equal(o, fa.attention(*x, rotary=t, positions=pos, **kw))
        assert torch.equal(o, fa.attention(*x, rotary=t, positions=pos, positions_k=pos, **kw))


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    t = fa.rotary_table(128, 100)
    q = torch.randn(50, 4, 128).bfloat16().cuda()
    ref, _ = fa.rotary(q, None, t, batch=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = fa.rotary(q, None, t, batch=1, stream=s)
    s.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = fa.rotary(q, None, t, batch=1)
    q.copy_(q.flip(0))
    ref, _ = fa.rotary(q, None, t, batch=1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.gpu
def test_captured_gradients():
    """Forward and backward in one graph, replayed on other values."""
    t = fa.rotary_table(64, 100)
    q = torch.randn(60, 4, 64).cuda().requires_grad_()
    k = torch.randn(60, 2, 64).cuda().requires_grad_()
    gq, gk = torch.randn(60, 4, 64).cuda(), torch.randn(60, 2, 64).cuda()

    def step():
        out = fa.rotary(q, k, t, batch=3)
        return out + torch.autograd.grad(out, (q, k), (gq, gk))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    with torch.no_grad():
        q.copy_(torch.randn_like(q))
        gk.copy_(torch.randn_like(gk))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_attention_with_rotary_and_different_lengths():
    """Queries at the end of longer keys: positions for each side."""
    t = fa.rotary_table(64, 200)
    g = torch.Generator().manual_seed(8)
    q = torch.randn(40, 4, 64, generator=g).bfloat16().cuda().requires_grad_()
    k = torch.randn(130, 2, 64, generator=g).bfloat16().cuda().requires_grad_()
    v = torch.randn(130, 2, 64, generator=g).bfloat16().cuda().requires_grad_()
    kw = dict(causal=True, batch=1, deterministic=True)
    pos = dict(positions=torch.arange(90, 130).cuda(), positions_k=torch.arange(130).cuda())
    o = fa.attention(q, k, v, rotary=t, interleaved=True, **pos, **kw)
    qr, _ = fa.rotary(q, None, t, positions=pos["positions"], interleaved=True)
    _, kr = fa.rotary(None, k, t, positions=pos["positions_k"], interleaved=True)
    o2 = fa.attention(qr, kr, v, **kw)
    assert torch.equal(o, o2)
    w = torch.randn(o.shape, generator=g).bfloat16().cuda()
    for a, b in zip(torch.autograd.grad(o, (q, k, v), w), torch.autograd.grad(o2, (q, k, v), w)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="positions and positions_k"):
        fa.attention(q, k, v, rotary=t, **kw)


@pytest.mark.gpu
def test_more_tokens_than_one_launch_takes():
    """Past 2^27 tokens of one head the call runs as several launches."""
    T, d = (1 << 27) + 1000, 64
    t = torch.from_numpy(table64(d, 97)).cuda()
    q = torch.empty(T, 1, d, dtype=torch.bfloat16, device="cuda")
    q.view(torch.int16).random_(0x3C00, 0x4000)         # finite values
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 97
    got, _ = fa.rotary(q, None, t, positions=pos)
    for a in (0, (1 << 27) - 300, T - 500):
        ref, mag = rotate(f64(q[a:a + 500]), table64(d, 97).astype(np.float64), pos[a:a + 500].cpu().numpy(), False)
        within("q", f64(got[a:a + 500]), ref, rotary_bound(ref, mag, torch.bfloat16))
