"""Calls at the ends of what the attention entry points document: the longest padded batches and
the sizes that are refused."""

from __future__ import annotations

import pytest
import torch

from kv_token_compressor_b200 import kvc


@pytest.mark.gpu
def test_a_padded_batch_of_seconds_is_no_timeout():
    """2^28 queries of one head, six of them with rows at both ends: the walk over the rest takes
    seconds, longer than a bounded wait that no longer makes progress, and must not end it.  (Every
    K is 1, E4M3 0x38, so every attended query's output is exactly 1 and its lse is
    q.K scale + ln n = 8 + ln 5.)"""
    T, H, c = 1 << 28, 1, 8
    q = torch.ones((T, H, c), dtype=torch.bfloat16, device="cuda")
    nope = torch.full((64, c), 0x38, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(T, dtype=torch.int64, device="cuda")
    nv = torch.zeros(T, dtype=torch.int64, device="cuda")
    full = torch.tensor([0, 1, 148, 149, 300, T - 3], device="cuda")
    nv[full] = 5
    out = torch.full_like(q, 7.0)
    _, lse = kvc.shared_kv_attention(q, nope, None, ks, nv, 60, 0, 1.0, out=out, want_lse=True)
    assert kvc.device_status() == kvc.KVC_OK
    assert bool(torch.all(out[full] == 1.0))
    want = 8.0 + torch.log(torch.tensor(5.0, dtype=torch.float64))
    # x and lse are sums of a few exact products and one logarithm, each within 2^-22 of 9.6
    assert bool(torch.all((lse[full].double().cpu() - want).abs() <= 2.0 ** -18))
    out[full] = 0.0
    assert torch.count_nonzero(out).item() == 0
