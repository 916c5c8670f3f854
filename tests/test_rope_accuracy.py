"""partial_rope's sines and cosines by themselves, and its smallest shapes at angles that are not
zero (GPU).

Tolerances, derived before the first run.  Rotating (1, 0) or (0, 1) returns the kernel's cosine
and sine as they are (fma of exact products).  pos * inv_freq is exact in fp64 (24 + 28 bits at
most), its remainder modulo 2 pi is off by 2^-51 or less, and with the remainder as h + l (fp32 h,
|l| <= 2^-23) sin h and cos h are within CUDA's stated 2 units in the last place, the correction
l cos h (l sin h) leaves l^2 / 2 <= 2^-47, and the sum is rounded by half a unit:
    |got - ref| <= 2.5 * 2^-23 |ref| + 2^-46 .
Without the correction a sine next to a multiple of pi is off by all of l, thousands of units."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_token_compressor_b200 import kvc
from oracle import attention as AT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 28) - 4096, -4096])
def test_sines_and_cosines_to_their_last_places(half, inverse, start):
    T, r = 4096, 64
    pos = torch.arange(start, start + T)
    f = kvc.rope_frequencies(r)
    x = torch.zeros((T, 2, r))
    a, b = (slice(0, r // 2), slice(r // 2, r)) if half else (slice(0, r, 2), slice(1, r, 2))
    x[:, 0, a] = 1.0
    x[:, 1, b] = 1.0
    y = kvc.partial_rope(x.cuda(), pos.cuda(), f, r, layout="half" if half else "interleaved",
                         inverse=inverse).double().cpu().numpy()
    ang = pos.double().numpy()[:, None] * f.double().cpu().numpy()[None]
    cs, sn = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
    for got, ref in ((y[:, 0, a], cs), (y[:, 0, b], sn), (y[:, 1, a], -sn), (y[:, 1, b], cs)):
        over = np.abs(got - ref) - (2.5 * 2.0 ** -23 * np.abs(ref) + 2.0 ** -46)
        assert over.max() <= 0, (np.argwhere(over > 0)[:3], over.max())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("H,c,r", [(1, 8, 8), (3, 8, 8), (1, 24, 8), (1, 64, 24), (128, 512, 64)])
@pytest.mark.parametrize("pos", [1, 12345, -7])
def test_one_token_is_turned(dt, half, inverse, H, c, r, pos):
    """A single token, at an angle that is not zero; a turned value is a sum of two products of
    factors within 2.5 * 2^-23, each rounded: 2^-21 (|a| + |b|) is above all of it."""
    g = torch.Generator().manual_seed(H + c + r)
    x = torch.randn((1, H, c), generator=g).to(dt)
    f = kvc.rope_frequencies(r)
    got = kvc.partial_rope(x.cuda(), torch.tensor([pos]).cuda(), f, r,
                           layout="half" if half else "interleaved", inverse=inverse)
    got, x64 = got.double().cpu().numpy(), x.double().numpy()
    ref = AT.partial_rope(x64, np.array([pos]), f.double().cpu().numpy(), r, half, inverse)
    assert np.abs(ref - x64)[..., c - r:].max() > 0.1  # it does turn
    p = np.abs(x64)[..., c - r:]
    s = p[..., : r // 2] + p[..., r // 2:] if half else p[..., 0::2] + p[..., 1::2]
    pair = np.concatenate([s, s], -1) if half else np.repeat(s, 2, -1)
    step = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    assert np.array_equal(got[..., : c - r], x64[..., : c - r])
    err = np.abs(got - ref)[..., c - r:]
    assert np.all(err <= step * np.abs(ref[..., c - r:]) + 2.0 ** -21 * pair)
    assert kvc.device_status() == kvc.KVC_OK
