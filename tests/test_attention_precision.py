"""Shared-KV attention on entries that cancel: what is left is the kernel's own error.

On random entries the output's rounding to bf16 and the worst case of the scores' sums hide both
the rounding of the weights and a single row among thousands.  Here the scores come from 64
channels alone; in all others (the free ones, where the queries are 0) every row's sign opposes the
sum of the weightier rows, so that sum_s p_s K_sd is next to 0 and its rounding too.  All heads of
a query have the same q, hence the same answer.

Tolerances, derived before the first run (w_s: the weight that multiplies row s).
* Rounded weights: |dw / w| <= eta, 2^-11 (fp16, FP8 channels) or 2^-8 (bf16 channels), so over the
  free channels, where the signs are as good as random, the error's root mean square is at most
  eta S, S = sqrt(mean_d sum_s p_s^2 K_sd^2).  For weights whose mantissas m are spread evenly over
  an octave it is eta S sqrt(E[1 / m^2] / 3) = 0.425 eta S.
* Scores: 4 MMAs of 16 products, each with an error of at most 17 * 2^-23 of the largest partial
  sum, below B = max_s |scale| sum_d |q_d K_sd|: dx = 2 * 17 * 2^-23 B as a root of squares, and
  2^-20 for the exponential and the multiplications.
* Output sums: n / 16 MMAs and 8 joins, each 17 * 2^-23 of a partial sum that is S in size.
So each query's rms error is at most 1.5 (eta + dx + 2^-20 + sqrt(n / 16 + 8) 17 * 2^-23) S +
2^-8 rms(ref) (1.5: the sampling of 300 channels or more), and over all queries in which 16 rows or
more count (as (sum p)^2 / sum p^2), if these are 100 together, at most 0.6 instead of 1.5: one bit
less in the weights gives 0.85.  lse: 64 products and the sum of the weights, |error| <= 72 * 2^-23 B +
2^-20 (1 + |lse|).
* Flat scores (scale 0): every weight is 2^7, exact in every type, so
  |out - ref| <= 2^-8 |ref| + 2^-22 A + (n / 16 + 8) 17 * 2^-23 * 2 A, A the largest |partial sum|
  / n, and |lse - ln n| <= 2^-20 (1 + ln n): a row of n shows as 1 / n."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from kv_token_compressor_b200 import kvc
from oracle import attention as AT

FP8 = 16.0  # fp8_scale
ACC = 17 * 2.0 ** -23


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16()


def _e4m3(x):
    return torch.from_numpy(np.ascontiguousarray(x * FP8, np.float32)).to(torch.float8_e4m3fn)


def _bits(x, n):
    """x rounded to n significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, n)), e - n)


class Cancelling:
    """T queries of H equal heads.  lens: visible entries; wins: window rows; listed: through a
    shuffled list with holes, a tenth of the entries unlisted.  score: "fp8" or "bf16", the 64
    channels the scores come from; None: flat scores (scale 0)."""

    def __init__(self, H, c, r, lens, seed, wins=None, listed=False, score="bf16", sink=False):
        rng = np.random.default_rng(seed)
        self.H, self.c, self.r, self.lens, self.T = H, c, r, list(lens), len(lens)
        self.wins = list(wins) if wins is not None else None
        self.scale = 0.0 if score is None else 0.125
        at = {"fp8": slice(0, 64), "bf16": slice(c - 64, c), None: slice(0, 0)}[score]
        self.free = np.ones(c, bool)
        self.free[at] = False
        self.starts = np.concatenate([[0], np.cumsum(self.lens)[:-1]]).tolist()
        wins = self.wins or [0] * self.T
        self.wstarts = np.concatenate([[0], np.cumsum(wins)[:-1]]).tolist()
        cache = rng.standard_normal((sum(self.lens) + 1, c))
        window = rng.standard_normal((sum(wins) + 1, c))
        q = np.zeros((self.T, c))
        q[:, at] = rng.standard_normal((self.T, at.stop - at.start))
        self.q = _bf16(q)
        self.sink = rng.standard_normal(H).astype(np.float32) if sink else None
        self.idx = None
        if listed:
            k = max(self.lens) + 3
            self.idx = np.full((self.T, k), -1, np.int64)
            for t, n in enumerate(self.lens):
                self.idx[t, :n] = rng.permutation(n)
                self.idx[t, :n][rng.random(n) < 0.1] = -1
        self.rows, self.p, self.x = [], [], []
        for t in range(self.T):
            own = np.arange(self.lens[t])
            if listed:
                own = self.idx[t, : self.lens[t]]
                own = own[own >= 0]
            own = own + self.starts[t]
            w = np.arange(wins[t]) + self.wstarts[t]
            K = self.stored(np.concatenate([cache[own], window[w]]))
            x = self.scale * (K @ self.q[t].double().numpy())
            order = np.argsort(-x, kind="stable")
            size = np.abs(self.stored(rng.uniform(0.5, 2.0, K.shape)))
            e = np.exp(x - (x.max() if len(x) else 0.0))
            run = rng.choice([-1e-300, 1e-300], c)[self.free]
            free = size[:, self.free]
            for s in order:
                free[s] = np.copysign(free[s], -run)
                run += e[s] * free[s]
            K[:, self.free] = free
            cache[own], window[w] = K[: len(own)], K[len(own):]
            self.rows.append(K)
            self.x.append(x)
        self.nope, self.rope = self.split(cache)
        self.wnope, self.wrope = self.split(window)

    def split(self, v):
        cn = self.c - self.r
        return _e4m3(v[:, :cn]).view(torch.uint8), _bf16(v[:, cn:])

    def stored(self, v):
        """v as the cache layout holds it, fp64."""
        nope, rope = self.split(v)
        return AT.cache_values(nope.numpy(), rope.double().numpy(), FP8)

    def run(self, **kw):
        def i64(v):
            return torch.tensor(v, dtype=torch.int64, device="cuda")

        win = None
        if self.wins is not None:
            win = (self.wnope.cuda(), self.wrope.cuda(), i64(self.wstarts), i64(self.wins),
                   max(self.wins))
        q = self.q[:, None, :].expand(self.T, self.H, self.c).contiguous().cuda()
        sink = None if self.sink is None else torch.from_numpy(self.sink).cuda()
        a = dict(q=q, nope=self.nope.cuda(), rope=self.rope.cuda(), key_start=i64(self.starts),
                 n_visible=i64(self.lens), r=self.r, scale=self.scale, fp8_scale=FP8, window=win,
                 sink=sink, want_lse=True, **kw)
        if self.idx is None:
            out, lse = kvc.shared_kv_attention(max_visible=max(self.lens), **a)
        else:
            idx = torch.tensor(self.idx, dtype=torch.int32, device="cuda")
            out, lse = kvc.shared_kv_attention_topk(idx=idx, **a)
        assert kvc.device_status() == kvc.KVC_OK
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def simulate(self, fp8_bits=11, bf16_bits=8, rows=None, keep_lse=False):
        """What the kernel computes, on the host, with weights of so many bits; rows(t, indices)
        gives the rows that it takes."""
        out, lse = np.zeros((self.T, self.H, self.c)), np.zeros((self.T, self.H))
        for t in range(self.T):
            at = np.arange(len(self.rows[t]))
            mine = at if rows is None else rows(t, at)
            K, x = self.rows[t][mine], self.x[t][mine]
            ref = x.max() if len(x) else 0.0
            w = np.exp(x - ref)
            wide = np.arange(self.c) < self.c - self.r
            num = np.where(wide, _bits(w, fp8_bits) @ K, _bits(w, bf16_bits) @ K)
            for h in range(self.H):
                den = w.sum() + (math.exp(self.sink[h] - ref) if self.sink is not None else 0.0)
                out[t, h] = _bf16(num / den if den else num).double().numpy()
                lse[t, h] = np.float32(ref + math.log(den)) if den else -math.inf
            if keep_lse:
                lse[t] = [self.lse_of(t, h) for h in range(self.H)]
        return out, lse

    def lse_of(self, t, h):
        x = self.x[t] if self.sink is None else np.append(self.x[t], self.sink[h])
        return -math.inf if not len(x) else x.max() + math.log(np.exp(x - x.max()).sum())

    def check(self, out, lse):
        """Every query against the bounds above; returns the largest share of its bound that a
        query's error took."""
        wide = np.arange(self.c) < self.c - self.r
        q64, worst = np.abs(self.q.double().numpy()), 0.0
        pool = {True: [0.0, 0.0, 0.0], False: [0.0, 0.0, 0.0]}
        for t in range(self.T):
            K, x = self.rows[t], self.x[t]
            n = len(K)
            B = self.scale * np.max(np.abs(K) @ q64[t], initial=0.0)
            for h in range(self.H):
                L = self.lse_of(t, h)
                if n == 0 and self.sink is None:
                    assert lse[t, h] == L and not out[t, h].any()
                    continue
                assert abs(lse[t, h] - L) <= 72 * 2.0 ** -23 * B + 2.0 ** -20 * (1 + abs(L)), (t, h)
                p = np.exp(x - L)
                ref = p @ K
                err = out[t, h] - ref
                if self.scale == 0.0:
                    A = np.abs(np.cumsum(K, 0) * p[:1]).max(0, initial=0.0)
                    bound = 2.0 ** -8 * np.abs(ref) + A * (2.0 ** -22 + (n / 16 + 8) * 2 * ACC) + 1e-30
                    assert np.all(np.abs(err) <= bound), (t, h, np.max(np.abs(err) / bound))
                    continue
                extra = 2 * ACC * B + 2.0 ** -20 + math.sqrt(n / 16 + 8) * ACC
                for fp8, eta in ((True, 2.0 ** -11), (False, 2.0 ** -8)):
                    d = self.free & (wide == fp8)
                    if d.sum() < 300 or n == 0:
                        continue
                    S2 = np.mean((p * p) @ (K[:, d] ** 2))
                    rms = math.sqrt(np.mean(err[d] ** 2))
                    base = (eta + extra) * math.sqrt(S2)
                    rounding = 2.0 ** -8 * math.sqrt(np.mean(ref[d] ** 2))
                    share = rms / (1.5 * base + rounding)
                    assert share <= 1, (t, h, fp8, share)
                    worst = max(worst, share)
                    count = p.sum() ** 2 / (p * p).sum()
                    if h == 0 and count >= 16:
                        g = pool[fp8]
                        g[0] += max(rms - rounding, 0.0) ** 2 / S2
                        g[1] += (eta + extra) ** 2
                        g[2] += count
        for fp8, (e2, b2, count) in pool.items():
            if count >= 100:
                share = math.sqrt(e2 / b2) / 0.6
                assert share <= 1, ("all queries", fp8, share)
        return worst


# H, c, r, score channels: free channels FP8 (448, 448, 512 - 64) or bf16 (448)
KINDS = [(64, 512, 64, "bf16"), (5, 512, 0, "fp8"), (70, 512, 512, "bf16")]
LENS = [[1], [2, 63], [64, 65, 0, 129], [300], [700, 1, 640], [1500], [3000, 200], [8193],
        [190] * 40, [70 + 3 * t for t in range(160)]]


def _case(kind, lens, listed, window, flat, seed=0):
    H, c, r, score = kind
    if sum(lens) > 10000:
        H = min(H, 5)
    wins = [(7 * t + 5) % 67 for t in range(len(lens))] if window else None
    return Cancelling(H, c, r, lens, seed=seed + sum(lens) + c + r, wins=wins, listed=listed,
                      score=None if flat else score, sink=window)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=["mixed", "fp8", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("listed,window", [(False, False), (True, True)])
@pytest.mark.parametrize("flat", [False, True], ids=["scores", "flat"])
def test_cancelling_entries(kind, lens, listed, window, flat):
    p = _case(kind, lens, listed, window, flat)
    out, lse = p.run()
    if p.sink is None:  # equal heads of a group of 64 (groups are cut into parts apart)
        for h in range(p.H):
            assert np.array_equal(out[:, h], out[:, h // 64 * 64])
    p.check(out, lse)


# ------------------------------------------------------------------ the checks themselves (CPU)

@pytest.mark.parametrize("kind", KINDS, ids=["mixed", "fp8", "bf16"])
@pytest.mark.parametrize("lens", LENS[:8], ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("flat", [False, True], ids=["scores", "flat"])
def test_the_stated_arithmetic_passes(kind, lens, flat):
    p = _case((3, *kind[1:]), lens, True, True, flat)
    p.check(*p.simulate())


@pytest.mark.parametrize("lens", [[700, 1, 640], [1500], [3000, 200], [190] * 40],
                         ids=lambda v: f"{len(v)}x{max(v)}")
@pytest.mark.parametrize("kind,bits", [(KINDS[0], dict(fp8_bits=10)), (KINDS[0], dict(fp8_bits=8)),
                                       (KINDS[1], dict(fp8_bits=10)), (KINDS[2], dict(bf16_bits=7)),
                                       (KINDS[2], dict(bf16_bits=5))])
def test_weights_of_fewer_bits_are_found(kind, bits, lens):
    p = _case((2, *kind[1:]), lens, False, False, False)
    p.check(*p.simulate())
    with pytest.raises(AssertionError):
        p.check(*p.simulate(**bits))


ROWS = {
    "last row lost": lambda t, at: at[:-1],
    "first row lost": lambda t, at: at[1:],
    "first row of the second tile lost": lambda t, at: np.delete(at, 64),
    "row at a part's end taken twice": lambda t, at: np.insert(at, 128, 127),
    "neighbour taken for a row": lambda t, at: np.where(at == 200, 201, at),
}


@pytest.mark.parametrize("what", ROWS)
@pytest.mark.parametrize("kind", KINDS, ids=["mixed", "fp8", "bf16"])
@pytest.mark.parametrize("n", [300, 3000])
@pytest.mark.parametrize("keep_lse", [False, True])
def test_a_lost_or_repeated_row_is_found(what, kind, n, keep_lse):
    """With flat scores whatever the types; with the right lse beside the wrong output too."""
    p = _case((2, *kind[1:]), [n], False, True, True)
    p.check(*p.simulate())
    with pytest.raises(AssertionError):
        p.check(*p.simulate(rows=ROWS[what], keep_lse=keep_lse))
