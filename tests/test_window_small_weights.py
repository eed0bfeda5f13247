"""Gradients of windowed attention where most probabilities are small: a first key that takes nearly
all of the weight, and attention that is flat over hundreds of thousands of keys.  A probability's
error is relative to it at any size, so the bounds are those of test_window.py, element by element."""
import math

import pytest
import torch

import bwd_tiled_attention_gb300 as fa
from bwd_tiled_attention_gb300 import build as fabuild
from test_window import check, make, reference


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()


def gradients(q, k, v, do, W, S, det, dtype):
    kw = dict(causal=True, batch=1, window=W, sinks=S)
    o, lse = fa.forward(q, k, v, out_dtype=dtype, **kw)
    got = fa.backward(q, k, v, o, do, lse, deterministic=det, grad_dtype=dtype, check_status=True, **kw)
    ref, bound, _, _ = reference(*(x.double() for x in (q, k, v, do)), W, S, 1 / math.sqrt(q.shape[2]))
    for name, x in zip(("dq", "dk", "dv"), got):
        check(name, x, ref[name], bound[name], dtype)
    return dict(zip(("dq", "dk", "dv"), got)), ref


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("lift", [12, 16, 20, 40])
@pytest.mark.parametrize("hq,hkv,det,dtype", [(2, 2, False, torch.bfloat16), (4, 1, True, torch.float32)])
def test_a_first_key_that_takes_nearly_everything(d, lift, hq, hkv, det, dtype):
    """The others' probabilities are about e^-lift (2^-17 to 2^-58)."""
    q, k, v, do = make([500], [500], hq, hkv, d, seed=lift)
    q[:, :, 0], k[:, :, 0] = 8.0, 0.0
    k[0, :, 0] = lift * math.sqrt(d) / 8
    got, ref = gradients(q, k, v, do, 200, 1, det, dtype)
    # far from the first key's own gradients, which are as large as ever
    assert ref["dk"][200:].norm() < 1e-3 * ref["dv"][0].norm() * math.exp(12 - lift) * 8
    off = (got["dk"][1:].double() - ref["dk"][1:]).norm() / ref["dk"][1:].norm()
    assert off < 2.0 ** -7, off   # dS's half step, and that of the stored value


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 192])
def test_flat_over_many_keys(d):
    """Probabilities of about 2^-19."""
    q, k, v, do = make([130], [600000], 1, 1, d)
    gradients(q * 0.01, k, v, do, 500000, 3, False, torch.float32)
