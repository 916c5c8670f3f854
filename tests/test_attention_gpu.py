"""GPU parity of partial_rope and shared_kv_attention(_topk) against the fp64 oracle.

Tolerances, derived before the first run.  One rounding to bf16 costs at most 2^-8 |ref|
(half a step), to fp32 2^-24.
* partial_rope: the reduced angle (|.| <= pi) rounds to fp32 (2^-24 pi) and its sine and cosine
  are within 2 units (2^-23): each turned value is off by at most 2^-21 (|a| + |b|), plus the
  output's own rounding.
* attention: x_s = scale q.K_s is a sum of c products that are exact in fp32, accumulated
  in fp32 in parts: |dx| <= (c + 8) 2^-23 B with B = max_s scale sum_d |q_d K_sd|.  A weight
  exp(x_s - lse) is then off by a factor within 1 +- 4 |dx|; the weights are rounded to 11
  bits (2^-11) where they multiply FP8 values, to 8 bits (2^-8) where they multiply bf16 ones,
  weights below 2^-24 of the largest vanish (at most rows 2^-24).  So
      |out - ref| <= 2^-8 |ref| + (eta + 4 dx + rows 2^-24) sum_s p_s |K_s|,
  eta = 2^-11 or 2^-8 by channel, and |lse - ref| <= dx + 2^-20 (1 + |ref|)."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from kv_token_compressor_b200 import kvc
from oracle import attention as AT

pytestmark = pytest.mark.gpu


def _i64(xs):
    return torch.tensor(list(xs), dtype=torch.int64, device="cuda")


# ------------------------------------------------------------------ partial_rope

ROPE = [  # T, H, c, r, dtype, half
    (1, 1, 8, 8, torch.bfloat16, False),
    (1, 1, 8, 8, torch.bfloat16, True),
    (3, 128, 512, 64, torch.bfloat16, False),
    (3, 128, 512, 64, torch.bfloat16, True),
    (1000, 1, 64, 24, torch.float32, False),
    (1000, 1, 64, 24, torch.bfloat16, True),
    (37, 5, 200, 200, torch.float32, True),
    (257, 7, 72, 40, torch.bfloat16, False),
    (5, 300, 136, 0, torch.bfloat16, False),
    (2, 3, 4096, 4096, torch.float32, False),
]


@pytest.mark.parametrize("T,H,c,r,dt,half", ROPE)
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_partial_rope(T, H, c, r, dt, half, inverse, in_place):
    g = torch.Generator().manual_seed(T + c + r)
    x = torch.randn((T, H, c), generator=g).to(dt)
    pos = torch.randint(0, 1 << 21, (T,), generator=g)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = -5, (1 << 40) + 1
    f = kvc.rope_frequencies(max(r, 8))[: r // 2].contiguous()
    mag = 1.25
    xd = x.cuda()
    out = xd if in_place else torch.empty_like(xd)
    kvc.partial_rope(xd, pos.cuda(), f, r, layout="half" if half else "interleaved",
                     inverse=inverse, magnitude=mag, out=out)
    assert kvc.device_status() == kvc.KVC_OK
    x64 = x.double().numpy()
    ref = AT.partial_rope(x64, pos.numpy(), f.double().cpu().numpy(), r, half, inverse, mag)
    got = out.double().cpu().numpy()
    assert np.array_equal(got[..., : c - r], x64[..., : c - r])
    step = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    both = np.abs(AT.partial_rope(np.abs(x64), 0 * pos.numpy(), f.double().cpu().numpy(), r, half))
    other = both.copy()  # |a| + |b| of every value's pair
    if r:
        p = both[..., c - r:]
        s = (p[..., : r // 2] + p[..., r // 2:] if half else p[..., 0::2] + p[..., 1::2])
        other[..., c - r:] = np.concatenate([s, s], -1) if half else np.repeat(s, 2, -1)
    bound = step * np.abs(ref) + mag * 2.0 ** -21 * other
    bound[..., : c - r] = 0
    over = int(np.count_nonzero(~(np.abs(got - ref) <= bound)))
    assert over == 0, f"{over} values beyond the bound"
    if not in_place:
        assert torch.equal(xd.cpu(), x)


def test_partial_rope_inverse_is_the_gradient():
    """Against the definition's differences: <R^T g, dx> = d<g, R x> along dx, fp32."""
    T, H, c, r = 4, 3, 48, 32
    g = torch.Generator().manual_seed(3)
    x, dx, gr = (torch.randn((T, H, c), generator=g).cuda() for _ in range(3))
    pos, f = _i64([0, 3, 77, 100000]), kvc.rope_frequencies(r)

    def fwd(v):
        return kvc.partial_rope(v, pos, f, r, magnitude=0.9, out=torch.empty_like(v)).double()

    num = (gr.double() * (fwd(x + dx) - fwd(x))).sum() - (gr[..., : c - r].double() *
                                                          dx[..., : c - r].double()).sum()
    back = kvc.partial_rope(gr, pos, f, r, inverse=True, magnitude=0.9, out=torch.empty_like(gr))
    ana = (back[..., c - r:].double() * dx[..., c - r:].double()).sum()
    # fp32 values of size below 6 through 384 terms, each within 2^-21 of its size
    assert abs(float(num - ana)) <= 384 * 36 * 2.0 ** -20


# ------------------------------------------------------------------ attention

def _cache(rows, cn, r, fp8_scale, rng, big=1.0):
    nope = torch.from_numpy(rng.standard_normal((rows, cn)).astype(np.float32)) * big
    nope = (nope * fp8_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    rope = torch.from_numpy(rng.standard_normal((rows, r)).astype(np.float32) * big)
    return nope, rope.to(torch.bfloat16)


class Problem:
    """Host and device copies of one attention problem."""

    def __init__(self, T, H, c, r, starts, lens, seed, window=None, sink=False, idx=None, rows=None,
                 fp8_scale=24.0, qs=2.0, scale=None):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.c, self.r, self.fp8_scale = T, H, c, r, fp8_scale
        self.scale = 1.0 / math.sqrt(c) if scale is None else scale
        self.q = torch.from_numpy((qs * rng.standard_normal((T, H, c))).astype(np.float32)).bfloat16()
        rows = max([s + n for s, n in zip(starts, lens)] + [1]) if rows is None else rows
        self.nope, self.rope = _cache(rows, c - r, r, fp8_scale, rng)
        self.starts, self.lens, self.idx = list(starts), list(lens), idx
        self.win = None
        if window is not None:
            wstarts, wlens, wmax = window
            wrows = max([s + n for s, n in zip(wstarts, wlens)] + [1])
            self.win = [*_cache(wrows, c - r, r, fp8_scale, rng), list(wstarts), list(wlens), wmax]
        self.sink = (torch.from_numpy(rng.standard_normal(H).astype(np.float32)) * 2) if sink else None

    def args(self):
        w = self.win
        win = None if w is None else (w[0].cuda(), w[1].cuda(), _i64(w[2]), _i64(w[3]), w[4])
        a = dict(q=self.q.cuda(), nope=self.nope.cuda(), rope=self.rope.cuda(),
                 key_start=_i64(self.starts), n_visible=_i64(self.lens), r=self.r,
                 scale=self.scale, fp8_scale=self.fp8_scale, window=win,
                 sink=None if self.sink is None else self.sink.cuda(), want_lse=True)
        if self.idx is None:
            a["max_visible"] = max(self.lens + [1])
        else:
            a["idx"] = torch.tensor(self.idx, dtype=torch.int32, device="cuda")
        return a

    def run(self, **kw):
        fn = kvc.shared_kv_attention if self.idx is None else kvc.shared_kv_attention_topk
        return fn(**{**self.args(), **kw})

    def rows(self, t):
        n, s = self.lens[t], self.starts[t]
        if self.idx is None:
            at = np.arange(s, s + n)
        else:
            at = np.array([s + i for i in self.idx[t][: min(len(self.idx[t]), n)] if 0 <= i < n],
                          dtype=np.int64)
        K = AT.cache_values(self.nope.numpy()[at], self.rope.double().numpy()[at], self.fp8_scale)
        if self.win is not None:
            w = slice(self.win[2][t], self.win[2][t] + self.win[3][t])
            K = np.concatenate([K, AT.cache_values(self.win[0].numpy()[w],
                                                   self.win[1].double().numpy()[w], self.fp8_scale)])
        return K

    def check(self, out, lse, queries=None):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        sink = None if self.sink is None else self.sink.double().numpy()
        eta = np.where(np.arange(self.c) < self.c - self.r, 2.0 ** -11, 2.0 ** -8)
        for t in range(self.T) if queries is None else queries:
            K = self.rows(t)
            ref, rlse, mag, top = AT.attend(self.q[t].double().numpy(), K, self.scale, sink)
            dx = ((self.c + 8) * 2.0 ** -23 * top)[:, None]
            bound = 2.0 ** -8 * np.abs(ref) + (eta + 4 * dx + len(K) * 2.0 ** -24) * mag + 1e-30
            bad = np.argwhere(~(np.abs(out[t] - ref) <= bound))
            assert bad.size == 0, (t, len(bad), bad[:3], out[t][tuple(bad[0])], ref[tuple(bad[0])])
            fin = np.isfinite(rlse)
            assert np.array_equal(lse[t][~fin], rlse[~fin])
            err = np.abs(lse[t][fin] - rlse[fin])
            assert np.all(err <= dx[fin, 0] + 2.0 ** -20 * (1 + np.abs(rlse[fin]))), (t, err.max())


def _lists(rng, lens, k, holes=0.0):
    idx = np.full((len(lens), k), -1, dtype=np.int64)
    for t, n in enumerate(lens):
        m = min(n, k)
        idx[t, :m] = rng.permutation(n)[:m]
        idx[t, :m][rng.random(m) < holes] = -1
    return idx


SHAPES = [  # H, c, r
    (128, 512, 64), (64, 512, 64), (1, 512, 64), (16, 512, 0), (128, 512, 512), (24, 256, 32),
    (8, 128, 64), (128, 64, 64), (5, 8, 0), (3, 8, 8), (100, 448, 8), (130, 72, 16), (257, 96, 24),
    (128, 200, 72), (40, 512, 128),
]


@pytest.mark.parametrize("H,c,r", SHAPES)
@pytest.mark.parametrize("listed", [False, True])
def test_attention_shapes(H, c, r, listed):
    rng = np.random.default_rng(c + H)
    lens = [1, 63, 64, 65, 200, 0, 129]
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]]).tolist()
    idx = _lists(rng, lens, 130) if listed else None
    p = Problem(7, H, c, r, starts, lens, seed=H, idx=idx, sink=H % 2 == 0)
    out, lse = p.run()
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse)


@pytest.mark.parametrize("T", [1, 2, 3, 20, 80, 200])
@pytest.mark.parametrize("n", [1, 40, 700, 3000])
def test_attention_lengths_and_batches(T, n):
    """From one short row to splits of long ones; every query its own length, the first the
    longest, some empty; window and sink beside."""
    if T * n > 100000:
        lens = [n] + [(t * 37) % 90 for t in range(T - 1)]
    else:
        lens = [n] + [(t * 7919) % (n + 1) for t in range(T - 1)]
    starts = [(t * 13) % 50 for t in range(T)]
    wl = [(t * 3) % 6 for t in range(T)]
    p = Problem(T, 32, 512, 64, starts, lens, seed=T + n, window=([t for t in range(T)], wl, 5),
                sink=True)
    out, lse = p.run()
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse, range(0, T, max(1, T // 12)))


@pytest.mark.parametrize("k", [1, 5, 64, 100, 512, 1024, 2048])
@pytest.mark.parametrize("T", [1, 9])
def test_listed_sizes(k, T):
    rng = np.random.default_rng(k)
    lens = [1500 - 100 * t for t in range(T)]
    p = Problem(T, 64, 512, 64, [7] * T, lens, seed=k, idx=_lists(rng, lens, k, holes=0.1),
                window=([0] * T, [128] * T, 128))
    out, lse = p.run()
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse)


def test_queries_without_rows():
    """No row at all: zero output, lse -inf (or the sink's logit); an all-(-1) list likewise."""
    for sink in (False, True):
        p = Problem(3, 20, 512, 64, [0, 5, 5], [0, 10, 0], seed=1, sink=sink,
                    window=([0, 0, 0], [0, 0, 0], 7))
        out, lse = p.run()
        p.check(out, lse)
        assert torch.count_nonzero(out[0]).item() == 0
        idx = np.full((2, 70), -1)
        p = Problem(2, 20, 512, 64, [0, 5], [100, 50], seed=2, sink=sink, idx=idx)
        out, lse = p.run()
        p.check(out, lse)
        assert torch.count_nonzero(out).item() == 0
        # nothing anywhere: a cache of no rows
        z = torch.zeros((0, 448), dtype=torch.uint8, device="cuda")
        zr = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
        out, lse = kvc.shared_kv_attention(torch.ones((2, 4, 512), dtype=torch.bfloat16, device="cuda"),
                                           z, zr, _i64([0, 0]), _i64([0, 0]), 0, 64, 1.0,
                                           want_lse=True)
        assert torch.count_nonzero(out).item() == 0 and bool(torch.all(lse == -math.inf))
    assert kvc.device_status() == kvc.KVC_OK


def test_sinks_large_small_and_absent():
    p = Problem(2, 5, 512, 64, [0, 0], [100, 3], seed=3, sink=True)
    p.sink = torch.tensor([-math.inf, -80.0, 0.0, 30.0, 200.0])
    out, lse = p.run()
    p.check(out, lse)
    p.lens = [0, 0]
    out, lse = p.run(max_visible=5)
    assert torch.equal(lse.cpu(), p.sink.expand(2, 5)) and torch.count_nonzero(out).item() == 0


def test_list_order_repeats_and_bad_entries():
    """An entry listed twice counts twice; -1 lists nothing anywhere in the list; entries
    outside the visible ones are left out and reported."""
    idx = [[5, 5, -1, 3, 0, 9, -1, 5, 8, 1]]
    p = Problem(1, 16, 512, 64, [2], [10], seed=4, idx=idx)
    out, lse = p.run()
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse)
    for bad in (10, -2, 1 << 30, -(1 << 31)):
        p.idx = [[5, 5, bad, 3, 0, 9, -1, 5, 8, 1]]
        out, lse = p.run()
        assert kvc.device_status() == kvc.KVC_ERR_INDEX
        assert kvc.device_status() == kvc.KVC_OK
        p.check(out, lse)
    # places past min(k, n_visible) are not read
    p = Problem(1, 16, 512, 64, [0], [3], seed=5, idx=[[2, 0, 1, 77, -9]])
    out, lse = p.run()
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse)


@pytest.mark.parametrize("T", [5, 300])
def test_bad_queries_are_skipped_and_reported(T):
    lens = [50] * T
    p = Problem(T, 16, 512, 64, [0] * T, lens, seed=6, window=([0] * T, [4] * T, 4), rows=60)
    a = p.args()
    ks, nv = [0] * T, [50] * T
    ws, wl = [0] * T, [4] * T
    ks[0] = 11           # past the cache
    nv[1] = -1
    ws[2] = 1            # past the window rows (4 of them)
    wl[3] = 5            # above max_win
    out = torch.full((T, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 16), 7.0, device="cuda")
    win = (a["window"][0], a["window"][1], _i64(ws), _i64(wl), 4)
    kvc.shared_kv_attention(**{**a, "key_start": _i64(ks), "n_visible": _i64(nv), "window": win,
                               "out": out, "lse": lse})
    assert kvc.device_status() == kvc.KVC_ERR_INDEX
    assert bool(torch.all(out[:4] == 7.0)) and bool(torch.all(lse[:4] == 7.0))
    p.check(out, lse, [4, T - 1])
    # n_visible above max_visible
    out.fill_(7.0)
    kvc.shared_kv_attention(**{**a, "max_visible": 49, "out": out, "lse": lse})
    assert kvc.device_status() == kvc.KVC_ERR_INDEX
    assert bool(torch.all(out == 7.0))


def test_rows_that_are_not_attended_may_hold_anything():
    """NaN bytes, NaN and infinities in rows outside the lists, windows and visible ranges."""
    rng = np.random.default_rng(8)
    lens = [70, 33]
    p = Problem(2, 128, 512, 64, [10, 90], lens, seed=8, rows=200, window=([3, 9], [5, 6], 16))
    used = np.zeros(200, bool)
    used[10:80] = used[90:123] = True
    p.nope[~used] = 0x7F
    p.rope[~used] = math.nan
    wused = np.zeros(15, bool)
    wused[3:8] = wused[9:15] = True
    p.win[0][~wused], p.win[1][~wused] = 0xFF, math.inf
    out, lse = p.run()
    p.check(out, lse)
    p.idx = _lists(rng, lens, 40)
    live = np.zeros(200, bool)
    for t in range(2):
        live[p.starts[t] + p.idx[t][p.idx[t] >= 0]] = True
    p.nope[~live], p.rope[~live] = 0xFF, -math.inf
    out, lse = p.run()
    p.check(out, lse)
    assert kvc.device_status() == kvc.KVC_OK


def test_nan_in_an_attended_row_reaches_only_its_query():
    p = Problem(2, 16, 512, 64, [0, 40], [40, 40], seed=9)
    p.nope[7, 100] = 0x7F
    out, lse = p.run()
    assert bool(torch.all(torch.isnan(out[0]))) and bool(torch.all(torch.isnan(lse[0])))
    p.check(out, lse, [1])


@pytest.mark.parametrize("qs,scale,fp8", [(1e-3, 1.0, 1.0), (50.0, 0.5, 24.0), (1.0, 0.0, 3.0),
                                          (1.0, -0.2, 0.37), (1e18, 1e-18, 100.0),
                                          (1e-18, 1e18, 448.0)])
def test_ranges_of_logits_and_scales(qs, scale, fp8):
    """Flat, peaked (one row takes all), negative and zero scales; queries near the ends of the
    exponent range; the maximum arriving late (rows sorted by score)."""
    p = Problem(2, 64, 512, 64, [0, 0], [300, 200], seed=10, qs=qs, scale=scale, fp8_scale=fp8)
    out, lse = p.run()
    p.check(out, lse)
    x = p.q[0, 0].double().numpy() @ p.rows(0).T * scale
    order = np.argsort(x)
    p.nope[:300], p.rope[:300] = p.nope[:300][order], p.rope[:300][order]
    out, lse = p.run()
    p.check(out, lse)


def test_wide_values_in_the_bf16_part():
    """bf16 channels keep their whole exponent range (values FP16 could not hold)."""
    for mag in (1e6, 1e-8):
        p = Problem(1, 16, 512, 64, [0], [150], seed=11, scale=1e-3 / mag)
        p.rope.mul_(mag)
        out, lse = p.run()
        p.check(out, lse)


def test_against_differences_of_lse():
    """d lse / d q = scale * out: the two outputs agree through a central difference."""
    p = Problem(1, 4, 128, 64, [0], [90], seed=12)
    out, lse = p.run()
    d = torch.zeros_like(p.q)
    d[0, :, 100] = 0.25
    q0 = p.q.clone()
    p.q = (q0.float() + d.float()).bfloat16()
    up, q_up = p.run()[1], p.q.double()
    p.q = (q0.float() - d.float()).bfloat16()
    dn, q_dn = p.run()[1], p.q.double()
    step = (q_up - q_dn)[0, :, 100]
    slope = (up - dn).double().cpu()[0] / step
    want = p.scale * out[0, :, 100].double().cpu()
    # third-order term: step^2 / 24 * scale^3 * |K|^3 bound (|K| <= 4), plus output rounding
    tol = float(step.max()) ** 2 * p.scale ** 3 * 64 + 2.0 ** -8 * want.abs() + 1e-4
    assert bool(torch.all((slope - want).abs() <= tol))


def test_same_result_every_time_and_with_a_reused_workspace():
    rng = np.random.default_rng(13)
    lens = [2500, 100, 2049]
    p = Problem(3, 128, 512, 64, [0, 0, 5], lens, seed=13, sink=True)
    a = p.args()
    n = kvc.shared_kv_attention_workspace_bytes(3, 128, 512, 64, 2500)
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
    out, lse = kvc.shared_kv_attention(**a, workspace=ws)
    p.check(out, lse)
    first = out.clone(), lse.clone()
    for _ in range(20):
        out, lse = kvc.shared_kv_attention(**a, workspace=ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    del rng


def test_streams_and_captured_graphs():
    """On a side stream, and captured and replayed with new inputs in the same buffers; two
    graphs with a workspace each replayed at once."""
    ps = [Problem(2, 64, 512, 64, [0, 0], [700, 650], seed=s, sink=True) for s in (14, 15)]
    s = torch.cuda.Stream()
    args = [p.args() for p in ps]
    torch.cuda.synchronize()
    out, lse = kvc.shared_kv_attention(**args[0], stream=s)
    s.synchronize()
    ps[0].check(out, lse)
    n = kvc.shared_kv_attention_workspace_bytes(2, 64, 512, 64, 700)
    graphs = []
    for a in args:
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        o, l = torch.empty_like(a["q"]), torch.empty((2, 64), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvc.shared_kv_attention(**a, workspace=ws, out=o, lse=l)
        graphs.append((g, o, l, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for p, (g, o, l, ws) in zip(ps, graphs):
        p.check(o, l)
    # new inputs in the first graph's buffers
    new = Problem(2, 64, 512, 64, [0, 0], [700, 650], seed=16, sink=True)
    for name in ("q", "nope", "rope", "sink"):
        args[0][name].copy_(getattr(new, name))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    new.check(graphs[0][1], graphs[0][2])
    assert kvc.device_status() == kvc.KVC_OK


def test_offsets_past_32_bits():
    """Rows beyond 2^32 bytes of the FP8 array (5 GB) are read where they are."""
    rows = 10_500_000
    nope = torch.zeros((rows, 448), dtype=torch.uint8, device="cuda")
    rope = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    p = Problem(1, 32, 512, 64, [0], [300], seed=17)
    at = rows - 300
    nope[at:], rope[at:] = p.nope.cuda(), p.rope.cuda()
    a = p.args()
    a.update(nope=nope, rope=rope, key_start=_i64([at]))
    out, lse = kvc.shared_kv_attention(**a)
    p.check(out, lse)
    idx = torch.randperm(rows, device="cuda")[:64].int()[None]
    idx[0, :50] = torch.arange(rows - 50, rows, device="cuda")
    del a["max_visible"]
    a.update(key_start=_i64([0]), n_visible=_i64([rows]), idx=idx)
    out, lse = kvc.shared_kv_attention_topk(**a)
    sel = idx[0].long()
    p.nope, p.rope = nope[sel].cpu(), rope[sel].cpu()
    p.starts, p.lens = [0], [64]
    p.check(out, lse)
    assert kvc.device_status() == kvc.KVC_OK


def test_sync_check_reports_from_the_call():
    p = Problem(1, 8, 128, 64, [0], [9], seed=18, rows=9)
    a = p.args()
    a["key_start"] = _i64([1])
    kvc.set_sync_check(True)
    try:
        with pytest.raises(kvc.KvcError) as e:
            kvc.shared_kv_attention(**a)
        assert e.value.status == kvc.KVC_ERR_INDEX
    finally:
        kvc.set_sync_check(False)
    assert kvc.device_status() == kvc.KVC_OK


def test_many_concurrent_calls_on_streams():
    """Calls whose work overlaps, a workspace each (the binding's own)."""
    ps = [Problem(4, 128, 512, 64, [0] * 4, [900, 10, 400, 0], seed=20 + i, sink=True)
          for i in range(4)]
    args = [p.args() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = [kvc.shared_kv_attention(**a, stream=s) for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    for p, (o, l) in zip(ps, outs):
        p.check(o, l)


def test_decode_step_together():
    """The operators as a decode step runs them: compress into the cache, score and select
    with the indexer, rotate the queries, attend, rotate the output back."""
    rng = np.random.default_rng(30)
    n, c, r, m, H, k = 2048, 512, 64, 4, 64, 128
    ne, T = n // m, 3

    def stream(width):
        return torch.from_numpy(rng.standard_normal((1, n, width)).astype(np.float32)).cuda().bfloat16()

    bias = [torch.zeros((m, c), device="cuda") for _ in range(2)]
    f = kvc.rope_frequencies(r, factor=4.0)
    nope, rope = kvc.csa_compress_cache(stream(c), stream(c), stream(c), stream(c), *bias, r, f,
                                        fp8_scale=16.0)
    nope, rope = nope.view(ne, c - r), rope.view(ne, r)
    kb = [torch.zeros((m, 128), device="cuda") for _ in range(2)]
    keys = kvc.csa_compress(stream(128), stream(128), stream(128), stream(128), *kb).view(ne, 128)
    pos = _i64([2047, 1033, 130])
    nv = [ne, 258, 32]
    iq = torch.from_numpy(rng.standard_normal((T, 64, 128)).astype(np.float32)).cuda().bfloat16()
    iw = torch.from_numpy(rng.random((T, 64)).astype(np.float32)).cuda()
    scores = kvc.lightning_indexer_scores(iq, iw, keys, _i64([0] * T), _i64(nv), ne)
    idx, _ = kvc.indexer_topk(scores, _i64(nv), k, ne, want_scores=False)
    q0 = torch.from_numpy(2 * rng.standard_normal((T, H, c)).astype(np.float32)).cuda().bfloat16()
    q = kvc.partial_rope(q0, pos, f, r)
    wn, wr = nope[-40:].contiguous(), rope[-40:].contiguous()
    win = (wn, wr, _i64([0, 1, 2]), _i64([30, 39, 1]), 64)
    sink = torch.zeros(H, device="cuda")
    out, lse = kvc.shared_kv_attention_topk(q, nope, rope, _i64([0] * T), _i64(nv), idx, r,
                                            1 / math.sqrt(c), fp8_scale=16.0, window=win, sink=sink,
                                            want_lse=True)
    back = kvc.partial_rope(out, pos, f, r, inverse=True)
    assert kvc.device_status() == kvc.KVC_OK
    p = Problem.__new__(Problem)
    p.T, p.H, p.c, p.r, p.fp8_scale, p.scale = T, H, c, r, 16.0, 1 / math.sqrt(c)
    p.q, p.nope, p.rope, p.sink = q.cpu(), nope.cpu(), rope.cpu(), sink.cpu()
    p.starts, p.lens, p.idx = [0] * T, nv, idx.cpu().numpy().astype(np.int64)
    p.win = [wn.cpu(), wr.cpu(), [0, 1, 2], [30, 39, 1], 64]
    p.check(out, lse)
    assert len(set(p.idx[2][:32].tolist())) == 32 and bool(np.all(p.idx[2][32:] == -1))
    ref = AT.partial_rope(out.double().cpu().numpy(), pos.cpu().numpy(),
                          f.double().cpu().numpy(), r, inverse=True)
    got = back.double().cpu().numpy()
    lim = np.abs(out.double().cpu().numpy()).max()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * lim)


@pytest.mark.parametrize("T,H,n", [(1, 130, 9000), (1, 7, 20000), (2, 65, 5000), (3, 1, 12000),
                                   (40, 66, 500), (100, 128, 300), (149, 64, 190), (40, 66, 2000),
                                   (100, 128, 1500), (149, 64, 900), (1, 64, 640)])
def test_split_queries_and_the_bounds_of_the_workspace(T, H, n):
    """Queries in two to more than a hundred parts, odd heads, several head groups; a workspace
    of exactly the stated bytes, full of NaN patterns, between guards."""
    lens = [n - (t * 977) % n for t in range(T)]
    p = Problem(T, H, 512, 64, [3] * T, lens, seed=T + H, sink=True,
                window=([0] * T, [t % 9 for t in range(T)], 8))
    need = kvc.shared_kv_attention_workspace_bytes(T, H, 512, 64, n + 8)
    assert need > 0 or n <= 500  # (0: short queries of a fairly full machine go whole)
    buf = torch.full((need + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = p.run(workspace=buf[4096: 4096 + need])
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse, range(0, T, max(1, T // 8)))
    assert bool(torch.all(buf[:4096] == 0xFF)) and bool(torch.all(buf[4096 + need:] == 0xFF))
    again, lse2 = p.run(workspace=buf[4096: 4096 + need])
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("T", [591, 592, 1300])
def test_many_queries_on_both_sides_of_whole_query_scheduling(T, listed):
    """Two head groups each: 1182, 1184 and 2600 items in turn on 148 CTAs, a full last round or
    not; empty queries and windows among them, outputs between guards."""
    rng = np.random.default_rng(T)
    lens = [(t * 31) % 140 for t in range(T)]
    idx = _lists(rng, lens, 70, holes=0.1) if listed else None
    wl = [(t * 5) % 7 for t in range(T)]
    p = Problem(T, 70, 128, 64, [(t * 3) % 40 for t in range(T)], lens, seed=T, idx=idx, sink=True,
                window=([t for t in range(T)], wl, 6))
    buf = torch.full((T * 70 * 128 + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((T * 70 + 512,), 7.0, device="cuda")
    out, lse = buf[2048: -2048].view(T, 70, 128), lbuf[256: -256].view(T, 70)
    p.run(out=out, lse=lse)
    assert kvc.device_status() == kvc.KVC_OK
    p.check(out, lse, [*range(0, T, 37), T - 1])
    for g in (buf[:2048], buf[-2048:], lbuf[:256], lbuf[-256:]):
        assert bool(torch.all(g == 7.0))


def test_partial_rope_many_pairs():
    """Up to 2^14 pairs a token, whose sines and cosines take 128 KB of shared memory."""
    g = torch.Generator().manual_seed(5)
    for c, r, half in ((32776, 32768, False), (16384, 16384, True), (4104, 4096, True)):
        x = torch.randn((3, 2, c), generator=g)
        pos, f = torch.tensor([0, 5, 70000]), kvc.rope_frequencies(r)
        got = kvc.partial_rope(x.cuda(), pos.cuda(), f, r, layout="half" if half else "interleaved")
        ref = AT.partial_rope(x.double().numpy(), pos.numpy(), f.double().cpu().numpy(), r, half)
        # |a| + |b| <= 12 for these; each value within 2^-21 of it and its own rounding
        assert float(x.abs().max()) <= 6
        err = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(err <= 12 * 2.0 ** -21 + 2.0 ** -24 * np.abs(ref))
    assert kvc.device_status() == kvc.KVC_OK


@pytest.mark.parametrize("T,every,most", [(3000, 400, 100), (3000, 2999, 200), (1000, 7, 1),
                                          (1100, 60, 500), (2000, 5000, 64)])
def test_long_runs_of_empty_queries(T, every, most):
    """Padded batches: hundreds of queries without rows between those that have some, and at
    the end."""
    lens = [1 + (t * 17) % most if t % every == 0 else 0 for t in range(T)]
    p = Problem(T, 20, 64, 64, [0] * T, lens, seed=T + every, sink=True)
    out, lse = p.run(max_visible=most)
    assert kvc.device_status() == kvc.KVC_OK
    used = [t for t in range(T) if lens[t]]
    p.check(out, lse, [*used, *range(1, T, 97)])
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert torch.count_nonzero(out[empty]).item() == 0
    assert torch.equal(lse[empty], p.sink.cuda().expand(int(empty.sum()), 20))
