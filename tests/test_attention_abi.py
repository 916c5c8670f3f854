"""Refusals of partial_rope and shared_kv_attention(_topk) before anything is launched: no
device is needed and no pointer is dereferenced."""

from __future__ import annotations

import math

import pytest
import torch

from kv_token_compressor_b200 import kvc

A = 0x7F0000000000
B = A + (1 << 40)
MIS = A + 8


@pytest.fixture(scope="module")
def L():
    from kv_token_compressor_b200 import build

    build.build()
    return kvc.lib()


def rope(L, **kw):
    a = dict(x=A, out=A, dt=kvc.KVC_BF16, T=4, H=8, c=512, r=64, pos=A, f=A, layout=0, inverse=0,
             mag=1.0)
    a.update(kw)
    return L.partial_rope(*[a[k] for k in ("x", "out", "dt", "T", "H", "c", "r", "pos", "f",
                                           "layout", "inverse", "mag")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=5), kvc.KVC_ERR_DTYPE),
    (dict(T=-1), kvc.KVC_ERR_SHAPE),
    (dict(H=0), kvc.KVC_ERR_SHAPE),
    (dict(c=500), kvc.KVC_ERR_SHAPE),
    (dict(r=12), kvc.KVC_ERR_SHAPE),
    (dict(r=520), kvc.KVC_ERR_SHAPE),
    (dict(r=-8), kvc.KVC_ERR_SHAPE),
    (dict(layout=2), kvc.KVC_ERR_SHAPE),
    (dict(inverse=2), kvc.KVC_ERR_SHAPE),
    (dict(mag=math.nan), kvc.KVC_ERR_SHAPE),
    (dict(mag=math.inf), kvc.KVC_ERR_SHAPE),
    (dict(T=1 << 50, H=1 << 10), kvc.KVC_ERR_SHAPE),
    (dict(x=None), kvc.KVC_ERR_NULL),
    (dict(out=None), kvc.KVC_ERR_NULL),
    (dict(pos=None), kvc.KVC_ERR_NULL),
    (dict(f=None), kvc.KVC_ERR_NULL),
    (dict(x=MIS), kvc.KVC_ERR_ALIGN),
    (dict(pos=A + 4), kvc.KVC_ERR_ALIGN),
    (dict(f=A + 2), kvc.KVC_ERR_ALIGN),
    (dict(out=A + 16), kvc.KVC_ERR_POINTER),                      # overlaps x, not in place
    (dict(out=A + 4 * 8 * 512 * 2 - 16), kvc.KVC_ERR_POINTER),
    (dict(T=0, x=None, out=None), kvc.KVC_OK),
    (dict(r=0, pos=None, f=None), kvc.KVC_OK),                    # in place: nothing to do
])
def test_partial_rope_rejects_before_launch(L, kw, status):
    assert rope(L, **kw) == status


ORDER = ("q", "T", "H", "c", "r", "nope", "rope", "rows", "s", "ks", "nv", "sel", "wn", "wr",
         "wrows", "ws", "wl", "mw", "sink", "scale", "out", "lse", "wsp", "wsb")


def att(L, topk=False, **kw):
    a = dict(q=A, T=4, H=128, c=512, r=64, nope=A, rope=A, rows=1000, s=1.0, ks=A, nv=A,
             sel=(A, 64) if topk else (900,), wn=A, wr=A, wrows=100, ws=A, wl=A, mw=32, sink=A,
             scale=0.1, out=B, lse=A, wsp=A, wsb=1 << 40)
    a.update(kw)
    flat = []
    for k in ORDER:
        flat += list(a[k]) if k == "sel" else [a[k]]
    fn = L.shared_kv_attention_topk if topk else L.shared_kv_attention
    return fn(*flat, None)


CASES = [
    (dict(T=-1), kvc.KVC_ERR_SHAPE),
    (dict(H=0), kvc.KVC_ERR_SHAPE),
    (dict(c=0), kvc.KVC_ERR_SHAPE),
    (dict(c=508), kvc.KVC_ERR_SHAPE),
    (dict(r=4), kvc.KVC_ERR_SHAPE),
    (dict(r=576), kvc.KVC_ERR_SHAPE),
    (dict(rows=-1), kvc.KVC_ERR_SHAPE),
    (dict(wrows=-1), kvc.KVC_ERR_SHAPE),
    (dict(mw=-1), kvc.KVC_ERR_SHAPE),
    (dict(s=0.0), kvc.KVC_ERR_SHAPE),
    (dict(s=-1.0), kvc.KVC_ERR_SHAPE),
    (dict(s=math.inf), kvc.KVC_ERR_SHAPE),
    (dict(s=math.nan), kvc.KVC_ERR_SHAPE),
    (dict(scale=math.nan), kvc.KVC_ERR_SHAPE),
    (dict(T=1 << 50, H=1 << 10), kvc.KVC_ERR_SHAPE),
    (dict(rows=1 << 60), kvc.KVC_ERR_SHAPE),
    (dict(c=520), kvc.KVC_ERR_UNSUPPORTED),          # nine 64-channel blocks
    (dict(c=512, r=32), kvc.KVC_ERR_UNSUPPORTED),    # 480 and 32 pad to nine blocks
    (dict(mw=1 << 31), kvc.KVC_ERR_UNSUPPORTED),
    (dict(q=None), kvc.KVC_ERR_NULL),
    (dict(nope=None), kvc.KVC_ERR_NULL),
    (dict(rope=None), kvc.KVC_ERR_NULL),
    (dict(ks=None), kvc.KVC_ERR_NULL),
    (dict(nv=None), kvc.KVC_ERR_NULL),
    (dict(wl=None), kvc.KVC_ERR_NULL),
    (dict(wn=None), kvc.KVC_ERR_NULL),
    (dict(wr=None), kvc.KVC_ERR_NULL),
    (dict(out=None), kvc.KVC_ERR_NULL),
    (dict(q=MIS), kvc.KVC_ERR_ALIGN),
    (dict(nope=MIS), kvc.KVC_ERR_ALIGN),
    (dict(rope=MIS), kvc.KVC_ERR_ALIGN),
    (dict(wr=MIS), kvc.KVC_ERR_ALIGN),
    (dict(out=B + 8), kvc.KVC_ERR_ALIGN),
    (dict(ks=A + 4), kvc.KVC_ERR_ALIGN),
    (dict(lse=A + 2), kvc.KVC_ERR_ALIGN),
    (dict(sink=A + 1), kvc.KVC_ERR_ALIGN),
    (dict(out=A), kvc.KVC_ERR_POINTER),              # out on q
    (dict(out=A + 4 * 128 * 512 * 2 - 16), kvc.KVC_ERR_POINTER),
    (dict(T=0, q=None, out=None), kvc.KVC_OK),
]


@pytest.mark.parametrize("topk", [False, True], ids=["dense", "topk"])
@pytest.mark.parametrize("kw,status", CASES)
def test_attention_rejects_before_launch(L, topk, kw, status):
    assert att(L, topk, **kw) == status


def test_attention_rejects_its_own_arguments(L):
    assert att(L, sel=(-1,)) == kvc.KVC_ERR_SHAPE
    assert att(L, sel=(1 << 31,)) == kvc.KVC_ERR_UNSUPPORTED
    assert att(L, True, sel=(A, 0)) == kvc.KVC_ERR_SHAPE
    assert att(L, True, sel=(A, (1 << 20) + 1)) == kvc.KVC_ERR_SHAPE
    assert att(L, True, sel=(None, 64)) == kvc.KVC_ERR_NULL
    assert att(L, True, sel=(A + 2, 64)) == kvc.KVC_ERR_ALIGN


def test_attention_workspace_bytes(L):
    f = L.shared_kv_attention_workspace_bytes
    assert f(-1, 128, 512, 64, 10) == -1 and f(4, 0, 512, 64, 10) == -1
    assert f(4, 128, 512, 32, 10) == -1 and f(4, 128, 512, 64, -1) == -1
    assert f(0, 128, 512, 64, 1000) == 0 and f(4, 128, 512, 64, 0) == 0
    need = f(4, 128, 512, 64, 932)
    assert 0 <= need < 1 << 27
    if need:
        assert att(L, wsb=need - 1) == kvc.KVC_ERR_SHAPE
        assert att(L, wsp=None) == kvc.KVC_ERR_NULL
        assert att(L, wsp=A + 128) == kvc.KVC_ERR_ALIGN


def _z(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt)


def _args(**kw):
    i64, u8, bf = torch.int64, torch.uint8, torch.bfloat16
    a = dict(q=_z(2, 4, 128, dt=bf), nope=_z(9, 64, dt=u8), rope=_z(9, 64, dt=bf),
             key_start=_z(2, dt=i64), n_visible=_z(2, dt=i64), max_visible=9, r=64, scale=1.0,
             window=(_z(5, 64, dt=u8), _z(5, 64, dt=bf), _z(2, dt=i64), _z(2, dt=i64), 4),
             sink=_z(4))
    a.update(kw)
    return a


def _win(i, t):
    w = list(_args()["window"])
    w[i] = t
    return tuple(w)


BINDING = [
    ("q dtype", dict(q=_z(2, 4, 128)), "q must be"),
    ("nope width", dict(nope=_z(9, 32, dt=torch.uint8)), "nope must be"),
    ("nope dtype", dict(nope=_z(9, 64)), "nope must be"),
    ("nope missing", dict(nope=None), "nope must be"),
    ("rope dtype", dict(rope=_z(9, 64)), "rope must be"),
    ("rows differ", dict(rope=_z(8, 64, dt=torch.bfloat16)), "same number of rows"),
    ("window rope", dict(window=_win(1, _z(5, 64))), "window rope must be"),
    ("sink size", dict(sink=_z(3)), "sink holds"),
    ("out shape", dict(out=_z(2, 4, 64, dt=torch.bfloat16)), "out must be"),
    ("lse shape", dict(lse=_z(2, 3)), "out must be"),
    ("consistent", dict(), "CUDA device"),
]


@pytest.mark.parametrize("name,kw,msg", BINDING, ids=[b[0] for b in BINDING])
def test_binding_refuses_tensors_the_library_would_misread(L, name, kw, msg):
    with pytest.raises(ValueError, match=msg):
        kvc.shared_kv_attention(**_args(**kw))


def test_binding_refuses_lists_and_rope_arguments(L):
    a = _args()
    del a["max_visible"]
    for idx in (_z(2, 4, dt=torch.int64), _z(8, dt=torch.int32), _z(3, 4, dt=torch.int32)):
        with pytest.raises(ValueError, match="idx must be"):
            kvc.shared_kv_attention_topk(idx=idx, **a)
    x, pos, f = _z(2, 4, 64), _z(2, dt=torch.int64), _z(16)
    with pytest.raises(ValueError, match="layout"):
        kvc.partial_rope(x, pos, f, 32, layout="pairs")
    with pytest.raises(ValueError, match="inv_freq holds"):
        kvc.partial_rope(x, pos, f, 64)
    with pytest.raises(ValueError, match="index arrays"):
        kvc.partial_rope(x, pos.int(), f, 32, out=x)  # int32 positions
    with pytest.raises(TypeError):
        kvc.partial_rope(x.double(), pos, f, 32)


def test_limits_of_what_the_kernels_hold(L):
    """Sizes and scales that would leave 32-bit counts, shared memory or fp32's range."""
    assert rope(L, c=32776, r=32776, x=None) == kvc.KVC_ERR_UNSUPPORTED
    assert rope(L, c=32776, r=32768, x=None) == kvc.KVC_ERR_NULL  # the shape is accepted
    for topk in (False, True):
        assert att(L, topk, s=1e-39) == kvc.KVC_ERR_UNSUPPORTED       # 1 / fp8_scale overflows
        assert att(L, topk, s=1e-20, scale=1e19) == kvc.KVC_ERR_UNSUPPORTED
        assert att(L, topk, scale=3e38) == kvc.KVC_ERR_UNSUPPORTED    # times log2(e)
        assert att(L, topk, s=1e-38, scale=1e-3, q=None) == kvc.KVC_ERR_NULL
    assert att(L, sel=((1 << 31) - 64,), mw=0, q=None) == kvc.KVC_ERR_NULL
    assert att(L, sel=((1 << 31) - 63,), mw=0, q=None) == kvc.KVC_ERR_UNSUPPORTED
    assert att(L, sel=((1 << 31) - 64,), mw=1, q=None) == kvc.KVC_ERR_UNSUPPORTED


def test_binding_refuses_a_window_without_starts():
    with pytest.raises(ValueError, match="win_start"):
        kvc.shared_kv_attention(**_args(window=_win(2, None)))
