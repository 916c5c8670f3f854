"""What the binding allocates for a call on a given stream comes from that stream's pool: a block
freed on the current stream, with a write to it still queued there, must not come back as the
output (or the zeroed scores) of a call that does not wait for it (GPU)."""

from __future__ import annotations

import pytest
import torch

from kv_token_compressor_b200 import kvc

pytestmark = pytest.mark.gpu

N, C = 8192, 512


def _bf(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _calls():
    s = [_bf(1, N, C, seed=i) for i in range(4)]
    b4 = [torch.zeros((4, C), device="cuda") for _ in range(2)]
    f = kvc.rope_frequencies(64)
    i64 = dict(dtype=torch.int64, device="cuda")
    num = 2048
    lists = (torch.zeros(num, **i64), torch.full((num,), N, **i64), torch.arange(num, **i64))
    iq, iw = _bf(16, 64, 128, seed=5), torch.rand((16, 64), device="cuda")
    keys, nk = _bf(65536, 128, seed=6), 65536
    starts, vis = torch.zeros(16, **i64), torch.full((16,), nk, **i64)
    scores = torch.rand((256, 8192), device="cuda")
    many = torch.full((256,), 8192, **i64)
    return {
        "csa": lambda st: kvc.csa_compress(*s, *b4, stream=st),
        "hca, m = 4": lambda st: kvc.hca_compress(s[0], s[1], b4[0], m=4, stream=st),
        "cache, FP8 part": lambda st: kvc.csa_compress_cache(*s, *b4, 64, f, stream=st)[0],
        "entries": lambda st: kvc.csa_compress_entries(*(x[0] for x in s), *b4, *lists, stream=st),
        "scores": lambda st: kvc.lightning_indexer_scores(iq, iw, keys, starts, vis, nk, stream=st),
        "top-k": lambda st: kvc.indexer_topk(scores, many, 2048, 8192, want_scores=False,
                                             stream=st)[0],
    }


@pytest.mark.parametrize("what", ["csa", "hca, m = 4", "cache, FP8 part", "entries", "scores",
                                  "top-k"])
def test_outputs_made_for_another_stream(what):
    call = _calls()[what]
    want = call(None).clone()
    want.fill_(3)  # (loads the kernels used below)
    want.copy_(call(None))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    late = torch.empty_like(want)
    torch.cuda._sleep(1_000_000_000)  # about half a second on the current stream
    late.fill_(3)
    del late
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert kvc.device_status() == kvc.KVC_OK
