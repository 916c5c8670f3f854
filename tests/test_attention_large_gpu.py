"""partial_rope and the attention calls on tensors of more than 2^31 elements (GPU): values on both
sides of the 32-bit borders of element and byte offsets."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_token_compressor_b200 import kvc
from oracle import attention as AT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("half", [False, True])
def test_rope_past_32_bit_offsets(in_place, half):
    """33000 x 128 heads of 512 bf16 channels: 2.16e9 elements.  Each turned value is off by
    2^-21 (|a| + |b|) at most and rounded to bf16."""
    T, H, c, r = 33000, 128, 512, 64
    x = torch.randn((1, H, c), generator=torch.Generator().manual_seed(1)).bfloat16()
    xd = x.cuda().expand(T, H, c).contiguous()
    pos = torch.arange(T)
    f = kvc.rope_frequencies(r)
    got = kvc.partial_rope(xd, pos.cuda(), f, r, layout="half" if half else "interleaved",
                           out=xd if in_place else None)
    x64 = x.double().numpy()
    for t in (0, 16383, 16384, 32767, 32768, T - 1):
        ref = AT.partial_rope(x64, np.array([t]), f.double().cpu().numpy(), r, half)
        y = got[t: t + 1].double().cpu().numpy()
        p = np.abs(x64)[..., c - r:]
        s = p[..., : r // 2] + p[..., r // 2:] if half else p[..., 0::2] + p[..., 1::2]
        pair = np.concatenate([s, s], -1) if half else np.repeat(s, 2, -1)
        assert np.array_equal(y[..., : c - r], x64[..., : c - r])
        err = np.abs(y - ref)[..., c - r:]
        assert np.all(err <= 2.0 ** -8 * np.abs(ref[..., c - r:]) + 2.0 ** -21 * pair), t
    # the copied channels of all tokens, whole
    assert bool(torch.all(got[..., : c - r] == x.cuda()[..., : c - r]))


@pytest.mark.parametrize("listed", [False, True])
def test_attention_past_32_bit_offsets(listed):
    """33000 queries x 128 heads of 512 channels; query t sees the one row t % 50 (twice, in a list
    or as two equal rows), so its output is that row to one bf16 rounding and its lse q.K scale +
    ln 2."""
    T, H, c, r, rows = 33000, 128, 512, 64, 50
    g = torch.Generator().manual_seed(2)
    nope = torch.randn((rows, c - r), generator=g).to(torch.float8_e4m3fn)
    rope = torch.randn((rows, r), generator=g).bfloat16()
    q1 = torch.randn((1, H, c), generator=g).bfloat16()
    q = q1.cuda().expand(T, H, c).contiguous()
    at = torch.arange(T, device="cuda") % rows
    i64 = dict(dtype=torch.int64, device="cuda")
    scale = 0.05
    if listed:
        idx = torch.stack([at, torch.full_like(at, -1), at], 1).int()
        out, lse = kvc.shared_kv_attention_topk(
            q, nope.cuda(), rope.cuda(), torch.zeros(T, **i64), torch.full((T,), rows, **i64), idx, r,
            scale, want_lse=True)
    else:
        out, lse = kvc.shared_kv_attention(
            q, nope.cuda().repeat_interleave(2, 0), rope.cuda().repeat_interleave(2, 0), 2 * at,
            torch.full((T,), 2, **i64), 2, r, scale, want_lse=True)
    assert kvc.device_status() == kvc.KVC_OK
    K = AT.cache_values(nope.view(torch.uint8).numpy(), rope.double().numpy(), 1.0)
    want = torch.from_numpy(K).cuda()
    x = scale * (q1[0].double().numpy() @ K.T)                      # [H, rows]
    B = scale * (np.abs(q1[0].double().numpy()) @ np.abs(K).T).max()
    wlse = torch.from_numpy(x + np.log(2.0)).cuda()
    for t0 in range(0, T, 1000):
        k = at[t0: t0 + 1000]
        # equal weights: their rounding cancels but for the two parts' own (2^-11, 2^-8)
        o = out[t0: t0 + 1000].double()
        eta = torch.where(torch.arange(c, device="cuda") < c - r, 2.0 ** -11, 2.0 ** -8)
        assert bool(torch.all((o - want[k][:, None]).abs() <=
                              (2.0 ** -8 + eta + 2.0 ** -20) * want[k][:, None].abs()))
        err = (lse[t0: t0 + 1000].double() - wlse.T[k]).abs()
        assert float(err.max()) <= (c + 8) * 2.0 ** -23 * B + 2.0 ** -18
