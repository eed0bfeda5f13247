"""Rotary positions, the paged key/value cache, and attention over it.

The tensor API of the second half of ``include/fa.h``: like the rest of the
package it marshals arguments and launches the library's kernels on the
current stream (or ``stream``).  q ``[T, Hq, d]`` and k, v ``[T, Hkv, d]`` may be
slices of a fused projection: the last dimension must be contiguous, token and
head strides are free (for `tree_attention`, positive multiples of 8 elements, and
the first element on a 16-byte boundary).  Sequences are a dense batch (T = B * N) or a packed one
(``cu_seqlens`` int32 ``[B+1]``).

A serving step::

    cache.reserve(slots, new)                        # room for the step's tokens
    for layer in range(layers):
        q = fa.cache_append(cache, layer, slots, k, v, q=q, rotary=table)
        o, lse = fa.tree_attention(q, cache, layer, slots, mask=mask)
    cache.accept(slots, base, path, accepted)        # after verifying a drafted tree
    cache.check()                                    # now and then: errors found on the device
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch
from torch.autograd import forward_ad

from . import FA_BF16, FA_FP32, FA_OK, FAError, lib

__all__ = ["PagedCache", "rotary", "rotary_table", "cache_append", "tree_attention", "tree_mask"]

_INT = (torch.int32,)
_BF16 = (torch.bfloat16,)
_HEAD_DIMS = (64, 96, 128, 192, 256)
_PAGE_SIZES = (16, 32, 64, 128)
_MOST = 2 ** 31 - 1  # counts are 32 bits


class _CacheDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "table", "lengths", "refs", "scratch")] + \
               [(n, ctypes.c_int) for n in ("layers", "pages", "heads", "page_size", "d", "slots",
                                            "max_pages")]


def _check(status, what):
    if status != FA_OK:
        raise FAError(status, what)


def _want(name, t, dtypes, ndim, device=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(x) for x in dtypes)}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _heads_tensor(name, t, dtypes, device=None):
    """A [T, H, d] tensor with free token and head strides."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == 3 and t.stride(2) == 1 and
            (device is None or t.device == device)):
        return
    _want(name, t, dtypes, 3, device, contiguous=False)
    if t.shape[2] > 1 and t.stride(2) != 1 and t.numel():
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _too_far(name, t):
    """The library's sizes are 32 bits."""
    raise ValueError(f"{name} has a dimension above {_MOST}: shape {tuple(t.shape)}")


def _not_differentiable(what, *tensors):
    """A gradient, or a forward tangent, that a call would drop is refused."""
    grad, forward = torch.is_grad_enabled(), forward_ad._current_level >= 0
    for t in tensors:
        if t is None:
            continue
        if grad and t.requires_grad:
            raise ValueError(f"{what} is not differentiable: call it under torch.no_grad(), or "
                             "detach what requires a gradient")
        if forward and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{what} is not differentiable, and an input has a forward tangent")


def _cuda(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")


@contextlib.contextmanager
def _on(device, stream, tensors):
    """The device made current and `stream`, when one is given, as its current
    stream: what is allocated inside belongs to it, and `tensors` are kept from
    reuse until it is done with them."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            for t in tensors:
                if isinstance(t, torch.Tensor) and t.is_cuda:  # (what else is given is refused later)
                    t.record_stream(stream)
            yield


def _here(device, stream):
    """Nothing to switch: the usual call."""
    return stream is None and device.index == torch._C._cuda_getDevice()


def _raw_stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _whole(name, x):
    if type(x) is int:
        return x
    n = int(x)
    if n != x:
        raise ValueError(f"{name} must be a whole number, got {x}")
    return n


def _sequences(T, batch, cu_seqlens, max_seqlen, device, need_max=True):
    """(B, N) of the call: N is the dense length, or the bound of a packed batch."""
    if T > _MOST:
        raise ValueError(f"{T} tokens: a call takes at most {_MOST}")
    if cu_seqlens is None:
        if batch is None:
            raise ValueError("dense inputs need batch (B); T = B * N")
        batch = _whole("batch", batch)
        if batch < 0 or (batch == 0 and T) or (batch and T % batch):
            raise ValueError("T must equal B * N for a dense batch")
        return batch, T // batch if batch else 0
    _want("cu_seqlens", cu_seqlens, _INT, 1, device)
    B = cu_seqlens.numel() - 1
    if B > _MOST:
        _too_far("cu_seqlens", cu_seqlens)
    if B < 0:
        raise ValueError("cu_seqlens must have B + 1 entries")
    if batch is not None and batch != B:
        raise ValueError("cu_seqlens and the batch name different sizes")
    if max_seqlen is None:
        if need_max:
            raise ValueError("variable-length inputs need max_seqlen")
        return B, 0
    max_seqlen = _whole("max_seqlen", max_seqlen)
    if not 0 <= max_seqlen <= _MOST:
        raise ValueError(f"max_seqlen must be from 0 to {_MOST}, got {max_seqlen}")
    return B, max_seqlen


# ------------------------------------------------------------------------------- rotary


def rotary_table(rot, length, base=10000.0, scaling=None, factor=1.0, original_length=None,
                 low_turns=1.0, high_turns=32.0, frequencies=None, device="cuda"):
    """cos and sin of positions 0 .. length-1: fp32 ``[length, rot/2, 2]``, angles in 64 bits.

    Pair i turns by ``base ** (-2i / rot)`` a position, or by ``frequencies[i]``.
    Scalings for contexts ``factor`` times as long as the trained one:

    - ``"linear"``: every frequency divided by factor;
    - ``"ntk"``: the base raised by ``factor ** (rot / (rot - 2))``, so that the slowest
      pair is divided by factor and the fastest stays (not with ``frequencies``);
    - ``"by_parts"``: pairs that turn fewer than ``low_turns`` times over
      ``original_length`` are divided by factor, those with more than ``high_turns`` stay,
      those between are mixed; cos and sin are stretched by ``1 + 0.1 ln(factor)``.
    """
    if rot <= 0 or rot % 2:
        raise ValueError("rot must be positive and even")
    if length < 0:
        raise ValueError("length must not be negative")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    if scaling not in (None, "linear", "ntk", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    scale = 1.0
    if frequencies is not None:
        freq = torch.as_tensor(frequencies, dtype=torch.float64)
        _not_differentiable("rotary_table", freq)
        if freq.shape != (rot // 2,):
            raise ValueError("frequencies must have rot / 2 entries")
        if scaling == "ntk":
            raise ValueError("ntk scaling raises the base, which frequencies take the place of")
    else:
        if scaling == "ntk":
            if rot < 4:
                raise ValueError("ntk scaling needs rot >= 4")
            base = base * factor ** (rot / (rot - 2))
        freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if original_length is None:
            raise ValueError("by_parts scaling needs original_length")
        if not low_turns < high_turns:
            raise ValueError("low_turns must be below high_turns")
        turns = original_length * freq / (2 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
        scale = 1.0 + 0.1 * math.log(factor)
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("the table must be on a CUDA device")
    with torch.cuda.device(device):
        freq = freq.to(device="cuda").contiguous()
        table = torch.empty((length, rot // 2, 2), dtype=torch.float32, device="cuda")
        _check(lib().fa_rotary_table(freq.data_ptr(), rot // 2, length, scale, _ptr(table) or None,
                                     _raw_stream(table.device)), "fa_rotary_table")
    return table


def _rotary_args(table, positions, T, device):
    _want("rotary table", table, (torch.float32,), 3, device)
    length, _, pair = table.shape
    if pair != 2:
        raise ValueError("the rotary table must be [length, rot / 2, 2]")
    if length > _MOST:
        _too_far("rotary table", table)
    if table.requires_grad and torch.is_grad_enabled():
        raise ValueError("the rotary table gets no gradient: detach it")
    if positions is None:
        return 0
    _want("positions", positions, (torch.int32, torch.int64), 1, device)
    if positions.shape[0] != T:
        raise ValueError("positions must have one entry a token")
    return 4 if positions.dtype == torch.int32 else 8


def _rotate(q, k, table, positions, pos_bytes, B, N, cu_seqlens, interleaved, backward):
    first = q if q is not None else k
    T, d = first.shape[0], first.shape[2]
    dev = first.device
    args = []
    outs = []
    for t in (q, k):
        if t is None:
            args += [None, None, 0, 0, 0]
            outs.append(None)
            continue
        o = torch.empty(t.shape, dtype=t.dtype, device=dev)
        s = t.stride()
        args += [t.data_ptr(), o.data_ptr(), t.shape[1], s[0], s[1]]
        outs.append(o)
    dt = FA_BF16 if first.dtype is torch.bfloat16 else FA_FP32
    if first.numel() or (k is not None and k.numel()):
        _check(lib().fa_rotary(*args, dt, T, d, table.shape[1] * 2, table.data_ptr(), table.shape[0],
                               _ptr(positions), pos_bytes, B, N, _ptr(cu_seqlens),
                               1 if interleaved else 0, backward, _raw_stream(dev)), "fa_rotary")
    return outs


def _last_contiguous(g):
    return g if g is None or g.shape[2] <= 1 or g.stride(2) == 1 else g.contiguous()


class _Rotary(torch.autograd.Function):
    """how: (pos_bytes, B, N, interleaved, backward); positions and cu_seqlens travel in `where`."""

    @staticmethod
    def forward(ctx, q, k, table, where, how):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(table, *where)
        ctx.how = how
        pos_bytes, B, N, interleaved, backward = how
        return tuple(_rotate(q, k, table, where[0], pos_bytes, B, N, where[1], interleaved, backward))

    @staticmethod
    def backward(ctx, gq, gk):
        if gq is None and gk is None:
            return None, None, None, None, None
        table, positions, cu_seqlens = ctx.saved_tensors
        pos_bytes, B, N, interleaved, back = ctx.how
        gq, gk = _last_contiguous(gq), _last_contiguous(gk)
        dev = (gq if gq is not None else gk).device
        with contextlib.nullcontext() if _here(dev, None) else torch.cuda.device(dev):
            # the transposed rotation, itself differentiable (a forward tangent is refused there)
            if torch.is_grad_enabled() or forward_ad._current_level >= 0:
                dq, dk = _Rotary.apply(gq, gk, table, (positions, cu_seqlens),
                                       (pos_bytes, B, N, interleaved, 1 - back))
            else:
                dq, dk = _rotate(gq, gk, table, positions, pos_bytes, B, N, cu_seqlens, interleaved,
                                 1 - back)
        return dq, dk, None, None, None


def rotary(q, k, table, positions=None, cu_seqlens=None, batch=None, interleaved=False,
           stream=None):
    """q and k (or one of them, the other None) turned to their tokens' positions; differentiable
    in reverse, any number of times (forward tangents are refused, as by `attention`).

    ``table`` is that of `rotary_table`; its rot columns of each head turn, the others are
    copied.  Pairs are columns (i, i + rot/2), or (2i, 2i + 1) when interleaved.  Without
    ``positions`` (int32 or int64 ``[T]``) each sequence counts from 0: pass ``batch`` or
    ``cu_seqlens``; tokens no packed sequence owns then come out as zeros.  A position
    outside the table makes the token's turned columns NaN.  bf16 or fp32.
    Returns new contiguous tensors (q, k).
    """
    first = q if q is not None else k
    if first is None:
        raise TypeError("rotary needs q or k")
    both = (torch.bfloat16, torch.float32)
    _heads_tensor("q" if q is not None else "k", first, both)
    if q is not None and k is not None:
        _heads_tensor("k", k, both)
        if k.dtype != q.dtype or k.device != q.device:
            raise ValueError("q and k must have one type and device")
        if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
            raise ValueError("q and k must have the same tokens and head dimension")
    (T, H, d), dev = first.shape, first.device
    if H > _MOST or d > _MOST:
        _too_far("q" if q is not None else "k", first)
    if k is not None and k.shape[1] > _MOST:
        _too_far("k", k)
    pos_bytes = _rotary_args(table, positions, T, dev)
    if 2 * table.shape[1] > d:
        raise ValueError("the table turns more columns than a head has")
    if positions is not None:
        _sequences(T, 1, None, None, dev)
        B, N, cu_seqlens = 1, T, None
    else:
        B, N = _sequences(T, batch, cu_seqlens, None, dev, need_max=False)
    _cuda("q" if q is not None else "k", first)
    # (inside a dual level an input may have a forward tangent, which the function refuses)
    grad = torch.is_grad_enabled() and ((q is not None and q.requires_grad) or
                                        (k is not None and k.requires_grad)) or \
        forward_ad._current_level >= 0

    if not _here(dev, stream):
        with _on(dev, stream, (q, k, table, positions, cu_seqlens)):
            return rotary(q, k, table, positions, cu_seqlens, batch, interleaved)
    if grad:
        return _Rotary.apply(q, k, table, (positions, cu_seqlens), (pos_bytes, B, N, interleaved, 0))
    return tuple(_rotate(q, k, table, positions, pos_bytes, B, N, cu_seqlens, interleaved, 0))


# -------------------------------------------------------------------------------- cache


class PagedCache:
    """Keys and values of several sequences ("slots") in shared pages, for all layers.

    ``k``, ``v``: bf16 ``[layers, pages, heads, page_size, d]``; ``table``: int32
    ``[slots, max_pages]``, -1 past the pages in use; ``lengths``: int32 ``[slots]``;
    ``refs``: int32 ``[pages]``, the sequences that hold a page (0 = free).  `allocate` makes
    an empty cache.  Lists of slots are int32 tensors on the device; nothing synchronises.
    What is wrong in them (a slot out of range or named twice, too long a sequence, no free
    pages, a shared page that would be written) is found on the device: the call then changes
    nothing, and `check` raises.  Page operations on one cache must be ordered on one stream,
    and appends and attention ordered behind those whose rows they touch.
    """

    def __init__(self, k, v, table, lengths, refs):
        bf16 = (torch.bfloat16,)
        _want("k", k, bf16, 5)
        _want("v", v, bf16, 5, k.device)
        if k.shape != v.shape:
            raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} differ in shape")
        layers, pages, heads, page_size, d = k.shape
        if d not in _HEAD_DIMS:
            raise ValueError(f"the head dimension must be one of {_HEAD_DIMS}, got {d}")
        if page_size not in _PAGE_SIZES:
            raise ValueError(f"the page size must be one of {_PAGE_SIZES}, got {page_size}")
        _want("table", table, _INT, 2, k.device)
        _want("lengths", lengths, _INT, 1, k.device)
        _want("refs", refs, _INT, 1, k.device)
        slots, max_pages = table.shape
        if lengths.shape[0] != slots or refs.shape[0] != pages:
            raise ValueError("lengths must have an entry a slot, refs one a page")
        if not (layers and pages and heads and slots and max_pages):
            raise ValueError("the cache has no room")
        for name, t in (("k", k), ("table", table)):
            if max(t.shape) > _MOST:
                _too_far(name, t)
        _cuda("k", k)
        self.k, self.v, self.table, self.lengths, self.refs = k, v, table, lengths, refs
        self.layers, self.pages, self.heads, self.page_size, self.d = layers, pages, heads, page_size, d
        self.slots, self.max_pages, self.device = slots, max_pages, k.device
        size = lib().fa_cache_scratch_size(pages, slots, max_pages)
        self.scratch = torch.zeros(size // 4, dtype=torch.int32, device=k.device)
        self._desc = _CacheDesc(k.data_ptr(), v.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                                refs.data_ptr(), self.scratch.data_ptr(), layers, pages, heads,
                                page_size, d, slots, max_pages)
        self._at = ctypes.addressof(self._desc)
        self._tensors = (k, v, table, lengths, refs, self.scratch)

    @classmethod
    def allocate(cls, layers, pages, heads, page_size, d, slots, max_pages, device="cuda"):
        """An empty cache; its pages are not initialised."""
        shape = (layers, pages, heads, page_size, d)
        ints = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.full((slots, max_pages), -1, **ints), torch.zeros(slots, **ints),
                   torch.zeros(pages, **ints))

    def _list(self, name, t, n=None, ndim=1):
        _want(name, t, _INT, ndim, self.device)
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
        return t

    def _few(self, n):
        if n > self.slots:
            raise ValueError(f"{n} entries for {self.slots} slots: some slot is named twice")

    def _call(self, name, stream, tensors, *args):
        fn = getattr(lib(), name)
        if _here(self.device, stream):
            return _check(fn(self._at, *args, _raw_stream(self.device)), name)
        with _on(self.device, stream, self._tensors + tensors):
            _check(fn(self._at, *args, _raw_stream(self.device)), name)

    def reserve(self, slots, counts, stream=None):
        """Room for counts (an int, or int32 ``[n]``) more tokens at the end of each slot: pages are
        taken lowest index first and lengths raised.  Slots must differ."""
        n = self._list("slots", slots).shape[0]
        self._few(n)
        many = counts if isinstance(counts, torch.Tensor) else None
        if many is not None:
            self._list("counts", many, n)
            counts = 0
        else:
            counts = _whole("counts", counts)
            if not 0 <= counts <= _MOST:
                raise ValueError(f"counts must be from 0 to {_MOST}, got {counts}")
        self._call("fa_cache_reserve", stream, (slots, many), slots.data_ptr(), _ptr(many),
                   counts, n)

    def fork(self, parents, children, stream=None):
        """children[i], which must be empty, becomes a copy of parents[i]: whole pages are shared,
        a partly filled last page is copied."""
        n = self._list("parents", parents).shape[0]
        self._list("children", children, n)
        self._few(n)
        self._call("fa_cache_fork", stream, (parents, children), parents.data_ptr(),
                   children.data_ptr(), n)

    def free(self, slots, stream=None):
        """Empties slots; pages that no other slot holds are free again."""
        n = self._list("slots", slots).shape[0]
        if n > _MOST:
            _too_far("slots", slots)
        self._call("fa_cache_free", stream, (slots,), slots.data_ptr(), n)

    def accept(self, slots, base, path, accepted, stream=None):
        """Of the tokens behind position base[i], keeps path[i, :accepted[i]] (strictly ascending
        indices behind base, int32 ``[n, width]``), moved together, and drops the others."""
        n = self._list("slots", slots).shape[0]
        self._few(n)
        self._list("base", base, n)
        self._list("path", path, n, 2)
        if path.shape[1] > _MOST:
            _too_far("path", path)
        self._list("accepted", accepted, n)
        self._call("fa_cache_accept", stream, (slots, base, path, accepted), slots.data_ptr(),
                   base.data_ptr(), path.data_ptr(), path.shape[1], accepted.data_ptr(), n)

    def check(self, stream=None):
        """Synchronises the stream, and raises if a call on this cache has been refused on the
        device or failed there since the last check.  What a call on another stream finds while
        this one waits is kept for the next check."""
        bits = ctypes.c_int(0)
        with _on(self.device, stream, self._tensors):
            st = lib().fa_cache_check(self._at, ctypes.addressof(bits), _raw_stream(self.device))
        if st != FA_OK:
            told = [w for b, w in ((1, "a slot or page index out of range, or a slot named twice"),
                                   (2, "a length, count or path that does not fit"),
                                   (4, "not enough free pages"),
                                   (8, "a shared page would be written"),
                                   (16, "a wait in a kernel gave up")) if bits.value & b]
            raise FAError(st, "paged cache (" + "; ".join(told) + ")")


def _of_cache(cache, layer, slots):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    if not 0 <= layer < cache.layers:
        raise ValueError(f"layer {layer} of {cache.layers}")
    _want("slots", slots, _INT, 1, cache.device)
    n = slots.shape[0]
    if n > _MOST:
        _too_far("slots", slots)
    return n


def cache_append(cache, layer, slots, k, v, q=None, rotary=None, positions=None,
                 interleaved=False, cu_seqlens=None, stream=None):
    """Writes new keys and values ``[T, heads, d]`` to one layer of the cache, as the last tokens of
    ``slots``, which must differ (reserve them first: that checks it).  A token whose place is in
    a page that several slots share is not written, and `PagedCache.check` raises.

    With ``rotary`` (a `rotary_table`) k, and q if given, are turned to ``positions``, by
    default the tokens' places in their sequences.  Returns the turned q (contiguous), or
    None.  Sequence i is slots[i]: T = n * N tokens, or ``cu_seqlens``.  Not differentiable:
    inputs that require a gradient are refused outside ``torch.no_grad()``.
    """
    n = _of_cache(cache, layer, slots)
    dev = cache.device
    if not _here(dev, stream):
        with _on(dev, stream, cache._tensors + (slots, k, v, q, rotary, positions, cu_seqlens)):
            return cache_append(cache, layer, slots, k, v, q, rotary, positions, interleaved, cu_seqlens)
    _heads_tensor("k", k, _BF16, dev)
    _heads_tensor("v", v, _BF16, dev)
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1] != cache.heads or k.shape[2] != cache.d:
        raise ValueError(f"k {tuple(k.shape)} or v {tuple(v.shape)} does not fit the cache")
    if q is not None:
        _heads_tensor("q", q, _BF16, dev)
        Tq, Hq, d = q.shape
        if Tq != T or d != cache.d:
            raise ValueError(f"q {tuple(q.shape)} does not fit the cache or k")
        if Hq > _MOST:
            _too_far("q", q)
    if (k.requires_grad or v.requires_grad or (q is not None and q.requires_grad) or
            cache.k.requires_grad or cache.v.requires_grad or forward_ad._current_level >= 0):
        _not_differentiable("cache_append", k, v, q, rotary, cache.k, cache.v)
    B, N = _sequences(T, n, cu_seqlens, None, dev, need_max=False)
    rot = rows = pos_bytes = 0
    if rotary is not None:
        pos_bytes = _rotary_args(rotary, positions, T, dev)
        rows, rot = rotary.shape[0], 2 * rotary.shape[1]
        if rot > cache.d:
            raise ValueError("the table turns more columns than a head has")
    elif positions is not None:
        raise ValueError("positions need a rotary table")

    out = None
    if q is not None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        qt, qh, _ = q.stride()
    else:
        Hq = qt = qh = 0
    kt, kh, _ = k.stride()
    vt, vh, _ = v.stride()
    if T:
        _check(lib().fa_cache_append(
            cache._at, layer, slots.data_ptr(), B, N, _ptr(cu_seqlens), T, _ptr(q), _ptr(out), Hq,
            qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, rot, _ptr(rotary), rows,
            _ptr(positions), pos_bytes, 1 if interleaved else 0, _raw_stream(dev)), "fa_cache_append")
    return out


# ---------------------------------------------------------------------------- attention


def tree_mask(parents, cu_seqlens=None, max_seqlen=None, batch=None, stream=None):
    """Ancestor bits of drafted trees for `tree_attention`: int64 ``[T, words]``.

    ``parents``: int32 ``[T]``, the index within its sequence of each token's parent, -1 for
    none; parents come before their children."""
    _want("parents", parents, _INT, 1)
    T = parents.shape[0]
    B, N = _sequences(T, batch, cu_seqlens, max_seqlen, parents.device)
    _cuda("parents", parents)
    words = max(1, -(-N // 64))
    with _on(parents.device, stream, (parents, cu_seqlens)):
        mask = torch.empty((T, words), dtype=torch.int64, device=parents.device)
        _check(lib().fa_tree_mask(_ptr(parents), _ptr(cu_seqlens), B, N, T, words, _ptr(mask),
                                  _raw_stream(parents.device)), "fa_tree_mask")
    return mask


@functools.lru_cache(maxsize=256)
def _workspace_bytes(Hq, Hkv, N, d):
    return int(lib().fa_tree_workspace_size(Hq, Hkv, N, d))


def tree_attention(q, cache, layer, slots, mask=None, scale=None, cu_seqlens=None, max_seqlen=None,
                   out=None, workspace=None, stream=None):
    """Attention of new tokens over one layer of the cache; returns (o, lse).

    The tokens of q ``[T, Hq, d]`` are the last ones of ``slots`` (`cache_append` comes first).
    ``scale`` is positive, by default 1 / sqrt(d).
    Each sees all earlier tokens of its sequence, and of the call's own ones those that its
    row of ``mask`` names (`tree_mask`, or any int64 ``[T, words]``), or without a mask
    itself and those before it.  A row that sees nothing gives o = 0 and lse = -inf.
    Calls that may run at the same time need a ``workspace`` each.  Not differentiable:
    inputs that require a gradient are refused outside ``torch.no_grad()``.
    Sequence i is slots[i]: T = n * N tokens, or ``cu_seqlens`` and ``max_seqlen``.
    Tokens no packed sequence owns give o = 0 and lse = -inf, or are left as they are in
    ``out``, a pair (o, lse) to write to; a sequence whose boundaries decrease or are not
    within [0, T] owns none, and `PagedCache.check` raises.  ``workspace``: uint8, at least
    ``fa_tree_workspace_size`` bytes.
    """
    n = _of_cache(cache, layer, slots)
    dev = cache.device
    if not _here(dev, stream):
        with _on(dev, stream, cache._tensors + (q, slots, mask, cu_seqlens, workspace) +
                 (tuple(out) if out is not None else ())):
            return tree_attention(q, cache, layer, slots, mask, scale, cu_seqlens, max_seqlen, out,
                                  workspace)
    _heads_tensor("q", q, _BF16, dev)
    T, Hq, d = q.shape
    if Hq > _MOST:
        _too_far("q", q)
    if d != cache.d:
        raise ValueError("q and the cache differ in head dimension")
    if Hq % cache.heads or Hq == 0:
        raise ValueError("the query heads must be a multiple of the key/value heads")
    B, N = _sequences(T, n, cu_seqlens, max_seqlen, dev)
    words = 0
    if mask is not None:
        _want("mask", mask, (torch.int64,), 2, dev)
        rows, words = mask.shape
        if rows != T or 64 * words < N:
            raise ValueError("mask must be [T, words] with 64 bits a word for every new token")
        if words > _MOST:
            _too_far("mask", mask)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is not None:
        _want("out[0]", out[0], (torch.bfloat16,), 3, dev)
        _want("out[1]", out[1], (torch.float32,), 2, dev)
        if out[0].shape != q.shape or tuple(out[1].shape) != (Hq, T):
            raise ValueError("out must be ([T, Hq, d], [Hq, T])")
    if workspace is not None:
        _want("workspace", workspace, (torch.uint8,), 1, dev)
    if (q.requires_grad or cache.k.requires_grad or cache.v.requires_grad or out is not None or
            forward_ad._current_level >= 0):
        _not_differentiable("tree_attention", q, cache.k, cache.v, *(out or ()))

    if out is not None:
        o, lse = out
    else:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        lse = torch.empty((Hq, T), dtype=torch.float32, device=dev)
    if T == 0:
        return o, lse
    if workspace is not None:
        ws, size = workspace, workspace.numel()
    else:
        size = max(_workspace_bytes(Hq, cache.heads, N or 1, d), 16)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    qt, qh, _ = q.stride()
    _check(lib().fa_tree_fwd(
        cache._at, layer, slots.data_ptr(), B, N, _ptr(cu_seqlens), T, q.data_ptr(), Hq, qt, qh,
        _ptr(mask), words, o.data_ptr(), lse.data_ptr(), scale, 1 if out is None else 0,
        ws.data_ptr(), size, _raw_stream(dev)), "fa_tree_fwd")
    return o, lse
