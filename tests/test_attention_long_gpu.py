"""Every row of very long queries counted exactly once (GPU).

With scale 0 every weight is the same power of two, and with integers up to 8 as entries every
partial sum is an integer times it, exact in fp32 (below 2^24, checked with a factor of 8 beside
what the parts of a query add).  So out is the exact mean, rounded: its factors 1 / n and the weights' power of
two cost 2^-22, bf16 2^-8, of a mean that is a small integer over n: one row more or less shows.
lse = ln n to 2^-20 (1 + ln n)."""

from __future__ import annotations

import math

import pytest
import torch

from kv_token_compressor_b200 import kvc

pytestmark = pytest.mark.gpu


def _integers(rows, c, r, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-8, 9, (rows, c), generator=g, device="cuda", dtype=torch.int32)
    return v, v[:, : c - r].float().to(torch.float8_e4m3fn), v[:, c - r:].bfloat16()


def _check(out, lse, t, sums, n):
    mean = sums.double() / n
    assert float(sums.abs().max()) < 2 ** 20
    err = (out[t].double() - mean).abs()
    assert bool(torch.all(err <= (2.0 ** -8 + 2.0 ** -20) * mean.abs())), (t, n)
    L = math.log(n)
    assert float((lse[t].double() - L).abs().max()) <= 2.0 ** -20 * (1 + L), (t, n)


def _prefix_bound(v):
    """Largest partial sum in row order (each part of a query has at most twice that)."""
    return int(v.long().cumsum(0).abs().max())


@pytest.mark.parametrize("c,r", [(128, 64), (128, 0), (64, 64)])
@pytest.mark.parametrize("H,lens", [
    (64, [8_000_000]),                       # among all CTAs
    (5, [3, 2_000_003, 64, 1]),              # beside short ones, split
    (128, [1_000_001] + [70] * 73),          # whole queries, CTA by CTA
    (1, [65_537 * k for k in range(1, 12)]),
])
def test_all_rows_of_long_queries(c, r, H, lens):
    rows = max(lens)
    v, nope, rope = _integers(rows, c, r, seed=c + r + rows)
    assert 2 * 8 * _prefix_bound(v) < 2 ** 24
    T = len(lens)
    q = torch.randn((T, H, c), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    nv = torch.tensor(lens, dtype=torch.int64, device="cuda")
    out, lse = kvc.shared_kv_attention(q, nope, rope, torch.zeros_like(nv), nv, rows, r, 0.0,
                                       want_lse=True)
    assert kvc.device_status() == kvc.KVC_OK
    for t, n in enumerate(lens):
        _check(out, lse, t, v[:n].long().sum(0), n)


@pytest.mark.parametrize("T", [1, 3])
def test_all_entries_of_the_longest_list(T):
    """2^20 listed entries of three million, in no order, and a window."""
    k, rows, c, r, w = 1 << 20, 3_000_000, 128, 64, 1000
    v, nope, rope = _integers(rows, c, r, seed=T)
    wv, wnope, wrope = _integers(w, c, r, seed=99)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.stack([torch.randperm(rows, generator=g, device="cuda")[:k] for _ in range(T)])
    idx[:, 77] = -1
    i64 = dict(dtype=torch.int64, device="cuda")
    q = torch.randn((T, 64, c), generator=g, device="cuda").bfloat16()
    win = (wnope, wrope, torch.zeros(T, **i64), torch.full((T,), w, **i64), w)
    out, lse = kvc.shared_kv_attention_topk(q, nope, rope, torch.zeros(T, **i64),
                                            torch.full((T,), rows, **i64), idx.int(), r, 0.0,
                                            window=win, want_lse=True)
    assert kvc.device_status() == kvc.KVC_OK
    for t in range(T):
        at = idx[t][idx[t] >= 0]
        assert 2 * 8 * _prefix_bound(v[at]) < 2 ** 24
        _check(out, lse, t, v[at].long().sum(0) + wv.long().sum(0), k - 1 + w)
