"""The newer operators given a stream of their own while the current one is busy (GPU): what they
allocate must not be a block that queued work still writes."""

from __future__ import annotations

import threading

import pytest
import torch

from kv_token_compressor_b200 import kvc

pytestmark = pytest.mark.gpu


def _args(T=3, H=64, c=512, r=64, n=700, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((T, H, c), generator=g, device="cuda").bfloat16()
    nope = torch.randn((n, c - r), generator=g, device="cuda").to(torch.float8_e4m3fn)
    rope = torch.randn((n, r), generator=g, device="cuda").bfloat16()
    ks = torch.zeros(T, dtype=torch.int64, device="cuda")
    nv = torch.full((T,), n, dtype=torch.int64, device="cuda")
    return dict(q=q, nope=nope, rope=rope, key_start=ks, n_visible=nv, max_visible=n, r=r,
                scale=0.04, want_lse=True)


@pytest.mark.parametrize("what", ["rope", "attention", "lse"])
def test_outputs_made_for_another_stream(what):
    """Freed on the current stream with a write to it still queued, a block must not come back as
    the output of a call on a side stream."""
    H = 64 if what != "lse" else 4096
    a = _args(T=64, H=H, c=512 if what != "lse" else 8, r=64 if what != "lse" else 8, n=70)
    x = a["q"].contiguous()
    pos, f = torch.arange(64, device="cuda"), kvc.rope_frequencies(64)
    given = torch.empty_like(x)

    def call(stream=None):
        if what == "rope":
            return kvc.partial_rope(x, pos, f, 64, stream=stream)
        out, lse = kvc.shared_kv_attention(**a, stream=stream, out=given if what == "lse" else None)
        return out if what == "attention" else lse

    want = call().clone().fill_(7.0)  # (loads the kernels used below)
    want.copy_(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    late = torch.empty_like(want)
    torch.cuda._sleep(1_000_000_000)  # about half a second on the current stream
    late.fill_(7.0)
    del late
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert kvc.device_status() == kvc.KVC_OK


def test_the_default_stream_by_its_handle():
    """stream=0 is the default stream, whatever stream is current; with a split query's workspace."""
    a = _args()
    assert kvc.shared_kv_attention_workspace_bytes(3, 64, 512, 64, 700) > 0
    want = kvc.shared_kv_attention(**a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = kvc.shared_kv_attention(**a, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_calls_from_several_host_threads():
    """Host threads with a stream each, first calls and later ones at once."""
    sets = [_args(T=1 + i, n=300 + 211 * i, seed=i) for i in range(4)]
    pos = [torch.arange(1 + i, device="cuda") for i in range(4)]
    f = kvc.rope_frequencies(64)
    want = [kvc.shared_kv_attention(**a) for a in sets]
    turned = [kvc.partial_rope(a["q"], p, f, 64) for a, p in zip(sets, pos)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(25):
            got = kvc.shared_kv_attention(**sets[i], stream=s)
            y = kvc.partial_rope(sets[i]["q"], pos[i], f, 64, stream=s)
            s.synchronize()
            if not (all(torch.equal(x, w) for x, w in zip(got, want[i])) and
                    torch.equal(y, turned[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and kvc.device_status() == kvc.KVC_OK


def test_captured_on_a_given_stream():
    """Inside a capture the capturing stream may be named: outputs and workspace then belong to the
    graph, and replays with new inputs fill the same tensors."""
    a, b = _args(seed=1), _args(seed=2)
    pos, f = torch.arange(3, device="cuda"), kvc.rope_frequencies(64)

    def step(x, stream=None):
        q = kvc.partial_rope(x["q"], pos, f, 64, stream=stream)
        out, lse = kvc.shared_kv_attention(**{**x, "q": q}, stream=stream)
        return kvc.partial_rope(out, pos, f, 64, inverse=True, stream=stream), lse

    want = [[t.clone() for t in step(x)] for x in (a, b)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(a, torch.cuda.current_stream())
    junk = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(4)]
    for x, w in zip((a, b), want):
        for name in ("q", "nope", "rope"):
            a[name].copy_(x[name])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(got, w))
    assert all(bool(torch.all(j == 7.0)) for j in junk) and kvc.device_status() == kvc.KVC_OK
