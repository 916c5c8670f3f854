"""What is measured of the attention-side operators: rotary positions on part of a head, and
shared-KV attention over the compressed cache (every visible entry, or an indexer's list).

A case is a dict of plain values.  prepare() makes the inputs on the GPU, run() makes one
pass (in plain torch operations, or the library's calls where `own` is true), work() counts
what the pass cannot do without, exact() is the definition in 64 bits.

Formulas.  A cache row s holds one entry, key and value of every head at once: its first
c - r channels are E4M3 bytes (value = byte / fp8_scale), its last r channels bf16.  Query t
of head h attends the rows of its list (indexer entries, or all n_t visible entries) followed
by its window's rows:
    x_s = scale * q[t, h] . K_s        p_s = exp(x_s) / (exp(sink_h) + sum_s exp(x_s))
    out[t, h] = sum_s p_s K_s          lse[t, h] = log(exp(sink_h) + sum_s exp(x_s))
Rotary positions: pair j of the last r channels is rotated by pos_t * inv_freq[j].
"""

from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    rope = dict(op="rope", dtype="bf16", layout="interleaved", inverse=False, in_place=True, c=512, r=64)
    att = dict(c=512, r=64, window=0, sink=False, shared=False, ragged=0)
    return [
        # one token's query heads, rotated in place before its attention: launch latency
        dict(rope, name="rope one token", T=1, H=64),
        # a decode batch's queries
        dict(rope, name="rope decode batch", T=128, H=128),
        # a prefill chunk's queries: pure bandwidth on 128-byte pieces of 1 KB rows
        dict(rope, name="rope prefill chunk", T=4096, H=128),
        # gradients (or outputs) turned back, fp32, half layout, odd sizes, into a new tensor
        dict(rope, name="rope back fp32 odd", T=777, H=24, c=192, r=80, dtype="f32", layout="half",
             inverse=True, in_place=False),
        # one sequence's decode step over the indexer's list and its local window
        dict(att, name="topk one token", op="topk", T=1, H=64, k=512, n=16384, window=128, sink=True),
        # a decode batch of long sequences: list, window and sink
        dict(att, name="topk decode batch", op="topk", T=128, H=128, k=1024, n=8192, window=128,
             sink=True, ragged=5000),
        # odd everything: few heads, narrow entries, a list length that fills no tile
        dict(att, name="topk odd", op="topk", T=37, H=24, c=256, r=32, k=777, n=3001, ragged=3001),
        # a prefill chunk: consecutive queries of one sequence, each with its own list
        dict(att, name="topk prefill chunk", op="topk", T=1024, H=128, k=1024, n=4096, window=128,
             sink=True, shared=True, ragged=256),
        # one sequence's decode step over all its heavily compressed entries
        dict(att, name="dense one token", op="dense", T=1, H=128, n=8192, window=128, sink=True),
        # a decode batch with sequences of different lengths
        dict(att, name="dense decode batch", op="dense", T=64, H=128, n=8192, window=128, sink=True,
             ragged=7000),
        # a prefill chunk: the visible prefix grows along the chunk
        dict(att, name="dense prefill chunk", op="dense", T=1024, H=128, n=512, window=128, sink=True,
             shared=True, ragged=8),
        # entries kept wholly in bf16 (no FP8 part), few heads
        dict(att, name="dense bf16 entries", op="dense", T=16, H=16, c=128, r=128, n=2000, ragged=1999),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "topk", "topk", "dense", "dense"])
    if op == "rope":
        c = 8 * rng.randint(1, 64)
        r = 8 * rng.randint(1, c // 8)
        H = rng.randint(1, 128)
        T = _log_int(rng, 1, 4096)
        return dict(op=op, T=T, H=H, c=c, r=r, dtype=rng.choice(["bf16", "f32"]),
                    layout=rng.choice(["interleaved", "half"]), inverse=rng.random() < 0.5,
                    in_place=rng.random() < 0.5)
    if rng.random() < 0.5:
        c, r = 512, 64
    else:
        while True:
            c = 8 * rng.randint(2, 64)
            r = rng.choice([0, c, 8 * rng.randint(0, c // 8)])
            if -(-(c - r) // 64) + -(-r // 64) <= 8:
                break
    H = rng.choice([1, 8, 16, 24, 64, 128, rng.randint(1, 128)])
    window = rng.choice([0, 0, 128, rng.randint(1, 128)])
    case = dict(op=op, H=H, c=c, r=r, window=window, sink=rng.random() < 0.5,
                shared=rng.random() < 0.5)
    if op == "topk":
        k = _log_int(rng, 1, 1024)
        n = _log_int(rng, 1, 8192)
        T = _log_int(rng, 1, 128)
        return dict(case, T=T, k=k, n=n, ragged=rng.randint(0, n))
    n = _log_int(rng, 1, 8192)
    T = _log_int(rng, 1, 64)
    return dict(case, T=T, n=n, ragged=rng.randint(0, n))


def _lengths(case):
    """Visible entries of each query: n less something below or at `ragged`, known from the
    case alone (a shared sequence: growing along the chunk)."""
    T, n, g = case["T"], case["n"], case["ragged"]
    if case["shared"]:
        return [n - g + (g * t) // max(T - 1, 1) for t in range(T)]
    return [n - (t * 7919) % (g + 1) for t in range(T)]


def _windows(case):
    """Window rows of each query (a sequence's first tokens have fewer)."""
    w = case["window"]
    return [w if t % 5 else max(w - t // 5, 0) for t in range(case["T"])]


def _cache(rows, cn, r, fp8_scale, gen):
    x = torch.randn((rows, cn), generator=gen, device="cuda", dtype=torch.bfloat16) * fp8_scale
    nope = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    rope = torch.randn((rows, r), generator=gen, device="cuda", dtype=torch.bfloat16)
    return nope, rope


def _ints(xs):
    return torch.tensor(xs, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, H, c, r = case["T"], case["H"], case["c"], case["r"]
    s = dict(case)
    if case["op"] == "rope":
        s["x"] = torch.randn((T, H, c), generator=gen, device="cuda").to(DT[case["dtype"]])
        start = torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda")
        s["pos"] = start + torch.arange(T, device="cuda")
        j = torch.arange(r // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * j / r)).float()
        s["out"] = s["x"] if case["in_place"] else torch.empty_like(s["x"])
        return s
    cn, n = c - r, case["n"]
    lens, wins = _lengths(case), _windows(case)
    seqs = 1 if case["shared"] else T
    s["fp8_scale"] = 24.0
    s["scale"] = 1.0 / math.sqrt(c)
    s["q"] = (2.0 * torch.randn((T, H, c), generator=gen, device="cuda")).to(torch.bfloat16)
    s["nope"], s["rope"] = _cache(seqs * n, cn, r, s["fp8_scale"], gen)
    s["key_start"] = _ints([0 if case["shared"] else t * n for t in range(T)])
    s["n_visible"] = _ints(lens)
    s["max_visible"] = n
    s["win"] = None
    if case["window"]:
        w = case["window"]
        rows = T + w if case["shared"] else T * w
        wn, wr = _cache(rows, cn, r, s["fp8_scale"], gen)
        s["win"] = (wn, wr, _ints([t if case["shared"] else t * w for t in range(T)]), _ints(wins), w)
    s["sink"] = torch.randn((H,), generator=gen, device="cuda") if case["sink"] else None
    if case["op"] == "topk":
        # the indexer's list: distinct visible entries in no order of position, -1 past them
        k = case["k"]
        u = torch.rand((T, n), generator=gen, device="cuda")
        u = torch.where(torch.arange(n, device="cuda") < s["n_visible"][:, None], u, 2.0)
        v, order = u.sort(dim=1)
        idx = torch.where(v < 1.5, order, -1)[:, :k].to(torch.int32)
        pad = torch.full((T, k - idx.shape[1]), -1, dtype=torch.int32, device="cuda")
        s["idx"] = torch.cat([idx, pad], 1).contiguous()
    return s


def _rotate(s, dt):
    """x with its last r channels rotated, in `dt` arithmetic (angles in 64 bits)."""
    r = s["r"]
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    if s["inverse"]:
        ang = -ang
    cs, sn = ang.cos().to(dt)[:, None, :], ang.sin().to(dt)[:, None, :]
    x = s["x"][..., s["x"].shape[-1] - r:].to(dt)
    if s["layout"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2:]
        return torch.cat([a * cs - b * sn, a * sn + b * cs], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)


def _rows(nope, rope, at, fp8_scale):
    """Rows `at` of a cache as fp32 values."""
    parts = [nope[at].view(torch.float8_e4m3fn).float() / fp8_scale, rope[at].float()]
    return torch.cat(parts, -1)


def _plain_attention(s):
    n_vis = s["n_visible"][:, None]
    if s["op"] == "topk":
        idx = s["idx"].long()
        live = idx >= 0
    else:
        idx = torch.arange(s["max_visible"], device="cuda").expand(s["T"], -1)
        live = idx < n_vis
    at = torch.where(live, s["key_start"][:, None] + idx, 0)
    K = _rows(s["nope"], s["rope"], at, s["fp8_scale"])
    if s["win"] is not None:
        wn, wr, start, wlen, w = s["win"]
        j = torch.arange(w, device="cuda").expand(s["T"], -1)
        wlive = j < wlen[:, None]
        K = torch.cat([K, _rows(wn, wr, torch.where(wlive, start[:, None] + j, 0), s["fp8_scale"])], 1)
        live = torch.cat([live, wlive], 1)
    x = torch.matmul(s["q"].float(), K.transpose(1, 2)) * s["scale"]
    x = torch.where(live[:, None, :], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    sink = s["sink"]
    if sink is not None:
        top = torch.maximum(top, sink[None, :, None])
    ref = torch.where(top == -math.inf, 0.0, top)
    p = (x - ref).exp()
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + (sink[None, :, None] - ref).exp()
    out = torch.matmul(p, K) / torch.where(total > 0, total, 1.0)
    return [out.to(torch.bfloat16), (total.log() + ref)[..., 0]]


def run(state):
    s = state
    if own:
        from kv_token_compressor_b200 import kvc

        if s["op"] == "rope":
            return kvc.partial_rope(s["x"], s["pos"], s["inv_freq"], s["r"], layout=s["layout"],
                                    inverse=s["inverse"], out=s["out"])
        if s["op"] == "topk":
            return kvc.shared_kv_attention_topk(
                s["q"], s["nope"], s["rope"], s["key_start"], s["n_visible"], s["idx"], s["r"],
                s["scale"], fp8_scale=s["fp8_scale"], window=s["win"], sink=s["sink"], want_lse=True)
        return kvc.shared_kv_attention(
            s["q"], s["nope"], s["rope"], s["key_start"], s["n_visible"], s["max_visible"], s["r"],
            s["scale"], fp8_scale=s["fp8_scale"], window=s["win"], sink=s["sink"], want_lse=True)
    if s["op"] == "rope":
        turned = _rotate(s, torch.float32)
        if not s["in_place"]:
            s["out"].copy_(s["x"])
        s["out"][..., s["c"] - s["r"]:] = turned.to(s["x"].dtype)
        return s["out"]
    return _plain_attention(s)


def work(case):
    T, H, c, r = case["T"], case["H"], case["c"], case["r"]
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        width = r if case["in_place"] else c
        return {"bytes": 2 * T * H * width * size + 8 * T + 2 * r, "flops": 3 * T * H * r}
    lens, wins = _lengths(case), _windows(case)
    if case["op"] == "topk":
        lens = [min(n, case["k"]) for n in lens]
    seen = sum(lens) + sum(wins)
    if case["op"] == "topk":
        # a shared sequence's entries: no more than it has
        rows = min(sum(lens), case["n"]) if case["shared"] else sum(lens)
        lists = 4 * sum(lens)
    else:
        rows, lists = (max(lens) if case["shared"] else sum(lens)), 0
    rows += min(sum(wins), T + case["window"]) if case["shared"] else sum(wins)
    return {"bytes": rows * (c + r) + 4 * T * H * c + 4 * T * H + 16 * T + lists,
            "flops": 4 * H * c * seen}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        x = s["x"].double()
        c, r = case["c"], case["r"]
        sign = -1.0 if case["inverse"] else 1.0
        turn = torch.exp(1j * sign * s["pos"].double()[:, None, None] * s["inv_freq"].double())
        if case["layout"] == "half":
            z = torch.complex(x[..., c - r: c - r // 2], x[..., c - r // 2:]) * turn
            return torch.cat([x[..., : c - r], z.real, z.imag], -1)
        z = torch.view_as_complex(x[..., c - r:].reshape(*x.shape[:2], r // 2, 2)) * turn
        return torch.cat([x[..., : c - r], torch.view_as_real(z).flatten(-2)], -1)
    T, H, c = case["T"], case["H"], case["c"]
    lens, wins = _lengths(case), _windows(case)
    out = torch.zeros((T, H, c), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    for t in range(T):
        first = 0 if case["shared"] else t * case["n"]
        if case["op"] == "topk":
            rows = first + s["idx"][t, : min(lens[t], case["k"])].long()
        else:
            rows = slice(first, first + lens[t])
        kn, kr = s["nope"][rows], s["rope"][rows]
        if s["win"] is not None:
            w0 = t if case["shared"] else t * case["window"]
            kn = torch.cat([kn, s["win"][0][w0: w0 + wins[t]]])
            kr = torch.cat([kr, s["win"][1][w0: w0 + wins[t]]])
        K = torch.cat([kn.view(torch.float8_e4m3fn).double() / s["fp8_scale"], kr.double()], 1)
        x = (s["q"][t].double() @ K.T) * s["scale"]
        if s["sink"] is not None:
            x = torch.cat([x, s["sink"].double()[:, None]], 1)
        if x.shape[1] == 0:
            continue
        lse[t] = torch.logsumexp(x, 1)
        out[t] = (x - lse[t][:, None]).exp()[:, : K.shape[0]] @ K
    return [out, lse]
