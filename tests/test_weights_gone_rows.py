"""Rows whose lse is -inf give nothing to any key, whatever their q holds: padding that was never
written, rejected drafts."""
import numpy as np
import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from test_cache import ints
from test_tree import Held, queries, words_of


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,heads,d,ps", [(4, 2, 64, 16), (8, 2, 128, 64), (2, 2, 256, 128), (12, 2, 96, 32)])
@pytest.mark.parametrize("n,ctx", [(1, 300), (9, 200), (150, 300), (40, 0)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("mask", [False, True])
def test_q_that_is_not_finite(Hq, heads, d, ps, n, ctx, value, mask):
    h = Held([n + ctx, n + ctx], heads, d, ps, seed=n)
    cache, slots = h.cache, ints(h.slots)
    q = queries(2 * n, Hq, d)
    words = words_of([list(range(t + 1)) for _ in range(2) for t in range(n)], -(-n // 64)) if mask else None
    _, lse = fa.tree_attention(q, cache, h.layer, slots, mask=words)
    gone = torch.zeros(2 * n, dtype=torch.bool, device="cuda")
    gone[::3] = True
    gone[-1] = True
    lse[:, gone] = -np.inf
    room = cache.max_pages * ps
    got = []
    for fill in (0.0, value):
        q[gone] = fill
        w = torch.zeros(cache.slots, heads, room, device="cuda")
        fa.cache_weights(q, lse, cache, h.layer, slots, w, mask=words)
        got.append(w)
    cache.check()
    # the same positive terms, n times the group's heads at most, added up in fp32 in two orders:
    # each sum is off by that many steps of 2^-24 at most, relative to it
    steps = n * (Hq // heads)
    assert torch.isfinite(got[1]).all()
    assert ((got[1] - got[0]).abs() <= 2 * steps * 2.0 ** -24 * got[0]).all()
    # the others' sums are there: every row of a head gives 1 in all
    total = got[1].double().sum(-1).sum(0)
    assert (total - (~gone).sum() * (Hq // heads)).abs().max() <= 2 * n * Hq * 1e-4
