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


A, B = 0x7F0000000000, 0x7F0000000000 + (1 << 44)  # addresses that nothing reads


@pytest.fixture(scope="module")
def L():
    from kv_token_compressor_b200 import build

    build.build()
    return kvc.lib()


def _dense(L, T, H, most):
    """Status of a dense call whose sizes alone are looked at: with no query tensor a call that
    would be taken ends in KVC_ERR_NULL before anything runs."""
    return L.shared_kv_attention(None, T, H, 512, 64, A, A, 1000, 1.0, A, A, most, None, None, 0,
                                 None, None, 0, None, 0.1, B, None, A, 1 << 50, None)


@pytest.mark.parametrize("T,H,most", [
    (1, 64, (1 << 31) - 63), (1, 64, 1 << 31), (1, 64, 1 << 38), (4, 128, 1 << 40),
    (1, 64, (1 << 63) - 1), (1, 64, (1 << 63) - 64), (3, 1, (1 << 31) + 1000),
    ((1 << 31) - 300, 64, 10), (1 << 30, 128, 10), (1 << 31, 1, 10), (1 << 45, 1, 1 << 30),
    (1, (1 << 31) - 1, 1 << 32),
])
def test_workspace_size_refuses_what_the_call_refuses(L, T, H, most):
    assert _dense(L, T, H, most) == kvc.KVC_ERR_UNSUPPORTED
    assert kvc.shared_kv_attention_workspace_bytes(T, H, 512, 64, most) == -1


@pytest.mark.parametrize("T,H,most", [
    (1, 64, (1 << 31) - 64), (1, 1, 1), (1 << 20, 128, 1 << 20), ((1 << 31) - 301, 64, 10),
    ((1 << 31) - 301, 64, (1 << 31) - 64), (1, (1 << 31) - 1, 100), (4, 128, 1000),
])
def test_workspace_size_answers_what_the_call_takes(L, T, H, most):
    assert _dense(L, T, H, most) == kvc.KVC_ERR_NULL
    # two slots of 64 heads x 512 channels fp32 and a pair of fp32 each, a CTA, at most
    assert 0 <= kvc.shared_kv_attention_workspace_bytes(T, H, 512, 64, most) <= 148 * 2 * 64 * 2056


def test_workspace_size_without_queries(L):
    """A call without queries does nothing, whatever its rows: no workspace."""
    assert _dense(L, 0, 64, 1 << 40) == kvc.KVC_OK
    assert kvc.shared_kv_attention_workspace_bytes(0, 64, 512, 64, 1 << 40) == 0
