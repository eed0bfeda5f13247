"""The page operations' kernels run on the host in several orders of their threads, against the plain
model: what they leave must not depend on how far a lane has come when its neighbours follow.

tests/cta_emulator compiles csrc/cache.cu as it is; a thread runs until it waits for others."""
import ctypes
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300.serving import _CacheDesc
from serving_ref import CacheModel, f64

HERE = os.path.dirname(os.path.abspath(__file__))
ASCENDING, DESCENDING, RANDOM = 0, 1, 2
ORDERS = [(ASCENDING, 0), (DESCENDING, 0), (RANDOM, 1), (RANDOM, 2)]
CALLS = ("fa_cache_scratch_size", "fa_cache_reserve", "fa_cache_fork", "fa_cache_free", "fa_cache_accept",
         "fa_cache_check")


def load(so):
    L = ctypes.CDLL(so)
    for name in CALLS:
        getattr(L, name).restype, getattr(L, name).argtypes = fa._SIGS[name]
    L.order_threads.argtypes = [ctypes.c_int, ctypes.c_ulonglong]
    L.at_stream_wait.argtypes = [ctypes.c_void_p]
    return L


@pytest.fixture(scope="module")
def emulated(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("emulated") / "cache.so")
    src = os.path.join(HERE, "cta_emulator")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I" + src,
                    os.path.join(src, "cache.cpp"), "-o", so], check=True)
    return so


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


class Cache:
    """The cache's calls on host memory."""

    def __init__(self, L, layers, pages, heads, ps, d, slots, max_pages, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.L = L
        self.k, self.v = (torch.randn(layers, pages, heads, ps, d, generator=g).bfloat16() for _ in range(2))
        self.table = torch.full((slots, max_pages), -1, dtype=torch.int32)
        self.lengths, self.refs = torch.zeros(slots).int(), torch.zeros(pages).int()
        self.scratch = torch.zeros(L.fa_cache_scratch_size(pages, slots, max_pages) // 4 + 4).int()
        at = self.scratch.data_ptr()
        self.scratch = self.scratch[(-at % 16) // 4:]
        self.slots = slots
        self.desc = _CacheDesc(self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr(),
                               self.lengths.data_ptr(), self.refs.data_ptr(), self.scratch.data_ptr(),
                               layers, pages, heads, ps, d, slots, max_pages)
        self.at = ctypes.addressof(self.desc)
        self.model = CacheModel(self.k, self.v, self.table, self.lengths, self.refs)

    def reserve(self, slots, counts):
        s, c = ints(slots), ints(counts)
        assert self.L.fa_cache_reserve(self.at, s.data_ptr(), c.data_ptr(), 0, len(slots), None) == 0
        return self.model.reserve(slots, counts)

    def fork(self, parents, children):
        p, c = ints(parents), ints(children)
        assert self.L.fa_cache_fork(self.at, p.data_ptr(), c.data_ptr(), len(parents), None) == 0
        return self.model.fork(parents, children)

    def free(self, slots):
        s = ints(slots)
        assert self.L.fa_cache_free(self.at, s.data_ptr(), len(slots), None) == 0
        return self.model.free(slots)

    def accept(self, slots, base, path, accepted):
        s, b, a = ints(slots), ints(base), ints(accepted)
        p = ints(path).view(len(slots), -1)
        assert self.L.fa_cache_accept(self.at, s.data_ptr(), b.data_ptr(), p.data_ptr(), p.shape[1],
                                      a.data_ptr(), len(slots), None) == 0
        return self.model.accept(slots, base, path, accepted)

    def status(self):
        bits = ctypes.c_int(-1)
        st = self.L.fa_cache_check(self.at, ctypes.addressof(bits), None)
        assert st == (fa.FA_OK if bits.value == 0 else fa.FA_ERR_TIMEOUT if bits.value & 16
                      else fa.FA_ERR_INVALID_ARG)
        return bits.value

    def agree(self):
        assert self.table.tolist() == self.model.table
        assert self.lengths.tolist() == self.model.lengths
        assert self.refs.tolist() == self.model.refs
        assert np.array_equal(f64(self.k), self.model.k) and np.array_equal(f64(self.v), self.model.v)


@pytest.mark.parametrize("order,seed", ORDERS)
def test_random_operations(emulated, order, seed):
    L = load(emulated)
    L.order_threads(order, seed)
    rnd = random.Random(order * 10 + seed)
    c = Cache(L, rnd.choice([1, 5]), rnd.choice([25, 60]), 2, 16, 64, 9, 8, seed)
    refused = 0
    for _ in range(30):
        some = rnd.sample(range(9), rnd.randint(1, 4))
        op = rnd.choice(["reserve", "reserve", "fork", "free", "accept", "accept"])
        if op == "reserve":
            bits = c.reserve(some, [rnd.choice([0, 1, 5, 16, 30]) for _ in some])
        elif op == "fork":
            empty = [s for s in range(9) if c.model.lengths[s] == 0]
            kids = rnd.sample(empty, min(len(empty), rnd.randint(1, 3))) or some
            bits = c.fork([rnd.choice([s for s in range(9) if s not in kids]) for _ in kids], kids)
        elif op == "free":
            bits = c.free(some + some[:1])
        else:
            base = [rnd.randint(0, c.model.lengths[s]) for s in some]
            width = rnd.choice([1, 3, 20])
            path = [sorted(rnd.sample(range(60), width)) for _ in some]
            got = [sum(t < c.model.lengths[s] - b for t in p) for s, b, p in zip(some, base, path)]
            got = [rnd.randint(0, x) for x in got]
            bits = c.accept(some, base, path, got)
        assert c.status() == bits, op
        refused += bits != 0
        c.agree()
    assert refused < 25


def many_entries(L, n, order, seed):
    L.order_threads(order, seed)
    c = Cache(L, 1, 5000, 1, 16, 64, 2 * n, 5, n)
    rnd = random.Random(n)
    first = rnd.sample(range(2 * n), n)
    other = [s for s in range(2 * n) if s not in set(first)]
    assert c.reserve(first, [rnd.randint(0, 70) for _ in first]) == 0
    assert c.fork(first, other) == 0
    assert c.status() == 0
    c.agree()
    length = c.model.lengths
    base = [rnd.randint(0, length[s] // 16) * 16 for s in other]
    got = [min(length[s] - b, rnd.choice([0, 1])) if length[s] // 16 * 16 == b else 0
           for s, b in zip(other, base)]
    assert c.accept(other, base, [[0]] * n, got) == 0
    assert c.free(rnd.sample(range(2 * n), n)) == 0
    assert c.status() == 0
    c.agree()


@pytest.mark.parametrize("order,seed", ORDERS)
@pytest.mark.parametrize("n", [300, 1100])
def test_many_entries(emulated, n, order, seed):
    """Groups of four lanes, and more entries than the planning CTA has threads: its lists then lie in
    the scratch words, the copying kernel's records among them.  In a process of its own, since a lane
    that takes a record for a count writes out of range."""
    code = (f"import sys; sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]\n"
            f"import test_cache_lanes as t\nt.many_entries(t.load({emulated!r}), {n}, {order}, {seed})")
    subprocess.run([sys.executable, "-c", code], check=True)


@pytest.mark.parametrize("before", [0, 2])
def test_errors_found_during_a_check_are_kept(emulated, before):
    """A bit that a call on another stream sets while the check waits, after it has copied the status
    word, is there for the next check."""
    L = load(emulated)
    c = Cache(L, 1, 4, 1, 16, 64, 2, 2)
    c.scratch[0] = before
    late = [8]

    def other_stream():
        if late:
            c.scratch[0] |= late.pop()

    hook = ctypes.CFUNCTYPE(None)(other_stream)
    L.at_stream_wait(ctypes.cast(hook, ctypes.c_void_p))
    try:
        assert c.status() == before
    finally:
        L.at_stream_wait(None)
    assert c.status() == 8 and c.status() == 0
