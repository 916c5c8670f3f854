"""The fp64 attention oracle against hand-worked values and invariants (CPU), and the
host-side frequency table of the library."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from kv_token_compressor_b200 import kvc
from oracle import attention as AT


@pytest.fixture(scope="module")
def L():
    from kv_token_compressor_b200 import build

    build.build()
    return kvc.lib()


def test_attend_worked_values():
    K = np.array([[1.0, 0.0], [0.0, 2.0]])
    q = np.array([[math.log(3.0), 0.0], [0.0, 0.0]])
    out, lse, mag, top = AT.attend(q, K, 1.0)
    assert np.allclose(out[0], [0.75, 0.5]) and np.allclose(out[1], [0.5, 1.0])
    assert np.allclose(lse, [math.log(4.0), math.log(2.0)])
    out, lse, _, _ = AT.attend(q, K, 1.0, sink=np.array([math.log(4.0), -math.inf]))
    assert np.allclose(out[0], [3 / 8, 2 / 8]) and np.allclose(lse[0], math.log(8.0))
    assert np.allclose(out[1], [0.5, 1.0])
    out, lse, _, _ = AT.attend(q, K[:0], 1.0)
    assert np.all(out == 0) and np.all(np.isneginf(lse))
    out, lse, _, _ = AT.attend(q, K[:0], 1.0, sink=np.array([0.5, 0.5]))
    assert np.all(out == 0) and np.allclose(lse, 0.5)


def test_e4m3_table_against_torch():
    b = torch.arange(256, dtype=torch.uint8)
    t = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, AT.e4m3_values(), equal_nan=True)


@pytest.mark.parametrize("half", [False, True])
def test_rope_invariants(half):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 24))
    f = AT.rope_frequencies(16)
    pos = np.array([0, 5, 1000003])
    y = AT.partial_rope(x, pos, f, 16, half=half)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., :8], x[..., :8])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    back = AT.partial_rope(y, pos, f, 16, half=half, inverse=True)
    assert np.allclose(back, x, atol=1e-12)
    # inverse is the transpose: <g, R x> = <R^T g, x>
    g = rng.standard_normal(x.shape)
    lhs = (g * AT.partial_rope(x, pos, f, 16, half=half, magnitude=1.3)).sum()
    rhs = (AT.partial_rope(g, pos, f, 16, half=half, inverse=True, magnitude=1.3) * x).sum()
    assert abs(lhs - rhs) < 1e-10
    # products of two rotated vectors depend on the distance of their positions only
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    d = [(AT.partial_rope(q, [p], f, 16, half=half) * AT.partial_rope(k, [p - 7], f, 16, half=half)
          ).sum() for p in (7, 4000)]
    assert abs(d[0] - d[1]) < 1e-9


@pytest.mark.parametrize("args", [
    (64,), (8, 500000.0), (64, 10000.0, 4.0, 4096.0, 32.0, 1.0), (64, 10000.0, 40.0, 4096.0),
    (128, 160000.0, 16.0, 65536.0, 32.0, 1.0), (16, 10000.0, 2.0, 10.0, 1.5, 0.01),
    (16, 1.5, 8.0, 1e9, 64.0, 32.0),
])
def test_rope_frequencies_match_the_definition(L, args):
    got = kvc.rope_frequencies(*args, device="cpu").double().numpy()
    ref = AT.rope_frequencies(*args)
    # one rounding to fp32 (half a step, 2^-24); the fp64 arithmetic adds far less
    assert np.all(np.abs(got - ref) <= 2.0 ** -24 * ref + 1e-13 * ref)


def test_rope_frequencies_scaling_by_parts(L):
    f1 = kvc.rope_frequencies(64, device="cpu").double()
    f8 = kvc.rope_frequencies(64, factor=8.0, original_len=4096.0, device="cpu").double()
    turns = 4096.0 * f1 / (2 * math.pi)
    assert torch.equal(f8[turns > 40.0], f1[turns > 40.0])          # fast pairs keep theirs
    slow = turns < 0.7
    assert torch.allclose(f8[slow], f1[slow] / 8, rtol=1e-6)        # slow ones are interpolated
    assert bool(torch.all(f8 <= f1)) and bool(torch.all(f8 >= f1 / 8 * (1 - 1e-6)))


@pytest.mark.parametrize("kw", [
    dict(r=0), dict(r=4), dict(r=12), dict(base=1.0), dict(base=math.nan), dict(factor=0.5),
    dict(factor=math.inf), dict(factor=2.0, original_len=0.0), dict(factor=2.0, beta_slow=0.0),
    dict(factor=2.0, beta_fast=1.0, beta_slow=1.0), dict(factor=2.0, original_len=math.nan),
])
def test_rope_frequencies_refusals(L, kw):
    a = dict(r=64, device="cpu")
    a.update(kw)
    with pytest.raises(kvc.KvcError) as e:
        kvc.rope_frequencies(**a)
    assert e.value.status == kvc.KVC_ERR_SHAPE
    assert L.kvc_rope_frequencies(64, 10000.0, 1.0, 0.0, 0.0, 0.0, None) == kvc.KVC_ERR_NULL
