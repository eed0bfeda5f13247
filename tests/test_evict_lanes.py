"""Eviction's kernels run on the host in several orders of their threads, against the plain form: with
keys in shared memory and without, more moves than are listed at once, runs of recent rows that
overlap their new places.

tests/cta_emulator compiles csrc/evict.cu as it is; a thread runs until it waits for others."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
import evict_ref
from serving_ref import f64
from test_cache_lanes import HERE, ORDERS, Cache, ints, load


@pytest.fixture(scope="module", params=[32768, 300])
def library(request, tmp_path_factory):
    """Keys in shared memory, or more than it is said to hold."""
    so = str(tmp_path_factory.mktemp("emulated") / f"evict{request.param}.so")
    src = os.path.join(HERE, "cta_emulator")
    text = open(os.path.join(src, "evict.cpp")).read()
    if request.param != 32768:  # the kernels' own constant, and a short list of moves
        own = open(os.path.join(HERE, "..", "bwd_tiled_attention_gb300", "csrc", "evict.cu")).read()
        assert "kMostKeys = 32768" in own and "kPairs = 2048" in own
        own = own.replace("kMostKeys = 32768", f"kMostKeys = {request.param}").replace("kPairs = 2048", "kPairs = 60")
        path = os.path.join(HERE, "..", "bwd_tiled_attention_gb300", "csrc")
        own = own.replace('#include "../../include/fa.h"', f'#include "{path}/../../include/fa.h"')
        for name in ("cache.cuh", "cache_plan.cuh", "common.cuh", "internal.h"):
            own = own.replace(f'#include "{name}"', f'#include "{path}/{name}"')
        at = str(tmp_path_factory.mktemp("source") / "evict.cu")
        open(at, "w").write(own)
        text = text.replace("../../bwd_tiled_attention_gb300/csrc/evict.cu", at)
    cpp = str(tmp_path_factory.mktemp("source") / "evict.cpp")
    open(cpp, "w").write(text)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-I" + src,
                    f"-DFA_MOST_KEYS={request.param}", os.path.join(src, "cache.cpp"), cpp, "-o", so], check=True)
    L = load(so)
    L.fa_cache_evict.restype, L.fa_cache_evict.argtypes = fa._SIGS["fa_cache_evict"]
    return L


def evicted(L, c, w, slots, keep, recent, sinks):
    """The call, and the plain form, on one cache; returns the status bits of both."""
    s, k = ints(slots), ints(keep)
    model_w = w.numpy().copy()
    want = evict_ref.evict(c.model, model_w, slots, keep, recent, sinks)
    before = [x.clone() for x in (c.k, c.v, w, c.table, c.lengths, c.refs)]
    assert L.fa_cache_evict(c.at, s.data_ptr(), k.data_ptr(), 0, recent, sinks, w.data_ptr(), len(slots), None) == 0
    bits = ctypes.c_int(0)
    L.fa_cache_check(c.at, ctypes.addressof(bits), None)
    if want:
        assert bits.value & want
        for a, b in zip(before, (c.k, c.v, w, c.table, c.lengths, c.refs)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        return bits.value
    assert bits.value == 0
    assert np.array_equal(f64(c.k), c.model.k) and np.array_equal(f64(c.v), c.model.v)
    assert c.table.tolist() == c.model.table and c.lengths.tolist() == c.model.lengths
    assert c.refs.tolist() == c.model.refs
    assert np.array_equal(w.numpy(), model_w, equal_nan=True)
    return 0


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lengths,keep,recent,sinks", [
    ([700, 90, 33], [128, 90, 20], 10, 3), ([500, 480], [450, 440], 200, 4), ([640, 17], [400, 17], 0, 0),
    ([600, 600], [40, 599], 30, 5), ([300], [299], 150, 149), ([64, 1], [0, 0], 0, 0)])
def test_evictions(library, order, kind, lengths, keep, recent, sinks):
    library.order_threads(*order)
    if min(keep) < recent + sinks:
        recent, sinks = min(recent, 3), min(sinks, 2)
    rng = np.random.default_rng(len(lengths) + keep[0])
    n = len(lengths)
    c = Cache(library, 2, sum(-(-x // 16) for x in lengths) + 3, 2, 16, 64, n + 1, max(-(-x // 16) for x in lengths))
    slots = list(rng.permutation(n + 1)[:n])
    assert c.reserve([int(s) for s in slots], lengths) == 0
    w = torch.from_numpy(evict_ref.random_weights(rng, (2, n + 1, 2, c.table.shape[1] * 16), kind))
    assert evicted(library, c, w, [int(s) for s in slots], keep, recent, sinks) == 0


@pytest.mark.parametrize("order", ORDERS[:3])
def test_refusals_change_nothing(library, order):
    library.order_threads(*order)
    c = Cache(library, 1, 30, 1, 16, 64, 5, 8)
    assert c.reserve([0, 1, 2], [100, 40, 64]) == 0
    assert c.fork([0], [3]) == 0
    w = torch.rand(1, 5, 1, 128)
    for slots, keep, recent, sinks, bits in (
            ([1, 1], [20, 20], 2, 2, 1), ([1, 9], [20, 20], 2, 2, 1), ([-1], [20], 2, 2, 1),
            ([1, 2], [20, 3], 2, 2, 2), ([0], [50], 4, 2, 8), ([3, 1], [99, 20], 4, 2, 8)):
        assert evicted(library, c, w, slots, keep, recent, sinks) & bits
    # shared pages before the sinks' end, and behind the budget, are no matter; kept whole ones neither
    assert evicted(library, c, w, [0], [96], 0, 96) == 0
    assert evicted(library, c, w, [3, 1], [100, 40], 4, 2) == 0
    assert evicted(library, c, w, [1, 2], [20, 3], 1, 2) == 0
