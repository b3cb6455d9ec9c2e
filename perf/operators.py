"""Cases of the attention operators around the linear layer: rotary positions, a paged cache that is
quantised as it is written and read back, the attention of new tokens over that cache, and the causal
attention of whole prompts.

`run` computes a case in plain torch operations (own = False) or through the package's calls (own = True) on
what `prepare` made; `exact` computes the same values in 64 bits, apart from both.

One description of a batch serves every call: `cu` [B + 1] (row offsets of the sequences' new tokens),
`kv_len` [B] (tokens cached, the new ones included) and `table` [B, pages per sequence] (page numbers;
-1: the page was dropped).  New token i of sequence b has position kv_len[b] - n_b + i.

The cache: per (page, KV head, token) a row of d codes of `bits` bits (4: channel 2j in the low nibble of byte
j), and (scale, minimum) in FP16; a code c stands for scale * c + minimum.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # q and k heads of one decode step of 64 sequences (32 query and 8 KV heads)
        dict(name="rotary_step", op="rotary", T=64, H=40, d=128, rot=128, interleaved=False, top=8192, stretch=1.0, shape=1),
        # a long prompt's rows, half of each head rotated, positions near a million (frequencies stretched 8x)
        dict(name="rotary_far", op="rotary", T=8191, H=40, d=128, rot=64, interleaved=True, top=1000000, stretch=8.0, shape=2),
        # one new token for each of 64 sequences: rotate q and k, write the cache, read the new rows back
        dict(name="cache_step", op="cache", B=64, new_lo=1, new_hi=1, len_lo=100, len_hi=8000, Hq=32, Hkv=8, d=128, bits=4,
             page=64, rot=128, interleaved=False, shape=3),
        # prompts of different lengths entering an empty cache
        dict(name="cache_prompts", op="cache", B=9, new_lo=500, new_hi=3001, len_lo=0, len_hi=0, Hq=32, Hkv=8, d=128, bits=4,
             page=64, rot=128, interleaved=False, shape=4),
        # reading whole sequences back (to move them, or to check them), 8 bits, small heads, short pages
        dict(name="cache_read_8bit", op="read", B=13, new_lo=700, new_hi=5000, len_lo=0, len_hi=0, Hq=8, Hkv=8, d=64, bits=8,
             page=16, rot=0, interleaved=False, shape=5),
        # a single sequence answering: latency counts
        dict(name="paged_one", op="paged", B=1, new_lo=1, new_hi=1, len_lo=1776, len_hi=1776, Hq=32, Hkv=8, d=128, bits=4,
             page=64, dropped=0.0, shape=6),
        # a full decode batch with ragged contexts
        dict(name="paged_batch", op="paged", B=64, new_lo=1, new_hi=1, len_lo=300, len_hi=8191, Hq=32, Hkv=8, d=128, bits=4,
             page=64, dropped=0.0, shape=7),
        # few sequences with very long contexts, 8 bits: the work has to be split along the context
        dict(name="paged_far_8bit", op="paged", B=2, new_lo=1, new_hi=1, len_lo=100000, len_hi=131000, Hq=64, Hkv=8, d=128,
             bits=8, page=128, dropped=0.0, shape=8),
        # pieces of long prompts over what is already cached
        dict(name="paged_chunks", op="paged", B=3, new_lo=450, new_hi=600, len_lo=2000, len_hi=16000, Hq=32, Hkv=8, d=128,
             bits=4, page=64, dropped=0.0, shape=9),
        # decode steps and short chunks in one call, small heads, groups of 7, some pages dropped
        dict(name="paged_mixed_8bit", op="paged", B=21, new_lo=1, new_hi=90, len_lo=0, len_hi=3500, Hq=28, Hkv=4, d=64, bits=8,
             page=16, dropped=0.1, shape=10),
        # one long prompt
        dict(name="prompt_long", op="prompt", B=1, new_lo=8192, new_hi=8192, Hq=32, Hkv=8, d=128, shape=11),
        # packed prompts of different lengths, a KV head for each query head
        dict(name="prompt_packed", op="prompt", B=17, new_lo=1, new_hi=1800, Hq=16, Hkv=16, d=128, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "cache", "read", "paged", "paged", "paged", "prompt", "prompt"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    bits, page = rng.choice([4, 4, 8]), rng.choice([16, 32, 64, 128])
    rot, inter = rng.choice([d, d, d // 2, d // 4]), rng.random() < 0.5
    shape = rng.randrange(1 << 30)
    if op == "rotary":
        return dict(op=op, T=_log(rng, 1, 8000), H=Hq + Hkv, d=d, rot=rot, interleaved=inter, top=_log(rng, 1000, 1000000),
                    stretch=rng.choice([1.0, 4.0, 8.0]), shape=shape)
    if op in ("cache", "read"):
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 10000 // B))
        return dict(op=op, B=B, new_lo=rng.randint(1, hi), new_hi=hi, len_lo=0, len_hi=rng.randint(0, 3000), Hq=min(Hq, 32), Hkv=Hkv,
                    d=d, bits=bits, page=page, rot=rot if op == "cache" else 0, interleaved=inter, shape=shape)
    if op == "paged":
        if rng.random() < 0.5:
            B, hi = _log(rng, 1, 64), 1
        else:
            B = _log(rng, 1, 12)
            hi = _log(rng, 2, 1500 // B)
        top = _log(rng, 16, min(60000, 300000 // B, max(16, 60000000 // (B * Hq * hi))))
        return dict(op=op, B=B, new_lo=rng.randint(1, hi), new_hi=hi, len_lo=rng.randint(0, top), len_hi=top, Hq=Hq, Hkv=Hkv, d=d,
                    bits=bits, page=page, dropped=rng.choice([0.0, 0.0, 0.2]), shape=shape)
    B = _log(rng, 1, 24)
    hi = _log(rng, 1, int(math.sqrt(600000000 / (B * Hq))))
    return dict(op=op, B=B, new_lo=rng.randint(1, hi), new_hi=hi, Hq=Hq, Hkv=Hkv, d=d, shape=shape)


def _lens(case):
    """The sequences' new tokens and cached tokens (the new ones included)."""
    r = random.Random(case["shape"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    old = [r.randint(case.get("len_lo", 0), case.get("len_hi", 0)) for _ in range(case["B"])]
    return new, [n + o for n, o in zip(new, old)]


def _pages(case):
    """Page numbers [B][pages per sequence]: a shuffled pool, a share of the full pages dropped."""
    r = random.Random(case["shape"] + 1)
    _, kv = _lens(case)
    per = [-(-n // case["page"]) for n in kv]
    order = list(range(sum(per)))
    r.shuffle(order)
    rows, at = [], 0
    for p in per:
        ids = order[at:at + p]
        at += p
        ids = [-1 if j < p - 1 and r.random() < case.get("dropped", 0.0) else x for j, x in enumerate(ids)]
        rows.append(ids + [-1] * (max(per) - p))
    return rows, sum(per)


# ----------------------------------------------------------------- inputs ----
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) % (1 << 31))


def _heads(g, T, H, d, outliers):
    """FP16 [T, H, d], normal; keys have a few channels 25 times as large."""
    x = torch.randn(T, H, d, generator=g, device=DEV)
    if outliers:
        x[:, :, torch.randperm(d, generator=g, device=DEV)[: max(1, round(0.02 * d))]] *= 25
    return x.half()


def _round_down(x):
    """FP16 of non-negative x in FP32, rounded towards zero."""
    h = x.half()
    return torch.where(h.float() > x, (h.view(torch.int16) - 1).view(torch.float16), h)


def _codes(x, bits):
    """x FP16 [..., d] -> codes uint8 [..., d], (scale, minimum) FP16 [..., 2]."""
    top = float(2 ** bits - 1)
    x = x.float()
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = _round_down((mx - mn) / top).float()
    c = torch.where(s > 0, ((x - mn) / torch.where(s > 0, s, 1.0)).round().clamp(max=top), torch.zeros_like(x))
    return c.to(torch.uint8), torch.cat([s, mn], -1).half()


def _pack(c, bits):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous() if bits == 4 else c


def _values(rows, par, bits):
    """Packed rows and (scale, minimum) -> the values they stand for, FP32 [..., d]."""
    c = torch.stack([rows & 15, rows >> 4], -1).flatten(-2) if bits == 4 else rows
    par = par.float()
    return c.float() * par[..., :1] + par[..., 1:]


def _freq(case):
    """Rotation angle per position of each pair of channels, in radians (64 bits)."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
    return 500000.0 ** (-2.0 * i / case["rot"]) / case.get("stretch", 1.0)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    d = case["d"]
    if case["op"] == "rotary":
        s["x"] = _heads(g, case["T"], case["H"], d, False)
        s["pos"] = torch.randint(0, case["top"], (case["T"],), generator=g, device=DEV, dtype=torch.int32)
        s["freq"] = _freq(case)
        return s
    new, kv = _lens(case)
    T, Hq, Hkv = sum(new), case["Hq"], case["Hkv"]
    s["cu"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    s["T"], s["most_new"], s["most_kv"] = T, max(new), max(kv)
    if case["op"] == "prompt":
        # the fused projection's output: q, k and v are column ranges of one matrix
        s["qkv"] = torch.cat([_heads(g, T, Hq, d, False), _heads(g, T, Hkv, d, True) / 3, _heads(g, T, Hkv, d, False)], 1)
        return s
    rows, pages = _pages(case)
    s["table"] = torch.tensor(rows, dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    bits, page = case["bits"], case["page"]
    if case["op"] == "cache":
        s["qkv"] = torch.cat([_heads(g, T, Hq, d, False), _heads(g, T, Hkv, d, True), _heads(g, T, Hkv, d, False)], 1)
        s["freq"] = _freq(case)
        for n in "kv":
            s[n + "_codes"] = torch.zeros(pages, Hkv, page, d * bits // 8, dtype=torch.uint8, device=DEV)
            s[n + "_par"] = torch.zeros(pages, Hkv, page, 2, dtype=torch.float16, device=DEV)
        return s
    for n in "kv":
        s[n + "_codes"] = torch.empty(pages, Hkv, page, d * bits // 8, dtype=torch.uint8, device=DEV)
        s[n + "_par"] = torch.empty(pages, Hkv, page, 2, dtype=torch.float16, device=DEV)
        for at in range(0, pages, 4096):
            x = _heads(g, min(4096, pages - at) * page, Hkv, d, n == "k").unflatten(0, (-1, page)).transpose(1, 2)
            c, p = _codes(x / 3 if n == "k" else x, bits)
            s[n + "_codes"][at:at + 4096], s[n + "_par"][at:at + 4096] = _pack(c, bits), p
    if case["op"] == "paged":
        s["q"] = _heads(g, T, Hq, d, False)
    return s


# -------------------------------------------------------------- own calls ----
def _own(s):
    import w4a8_integer_gemm_b200 as lib
    case = s["case"]
    if case["op"] == "rotary":
        return lib.qattn_rotary(s["x"], s["pos"], lib.Rotary(s["freq"], case["interleaved"]))
    if case["op"] == "prompt":
        q, k, v = s["qkv"].split([case["Hq"], case["Hkv"], case["Hkv"]], 1)
        return lib.qattn_prompt_attention(q, k, v, s["cu"])
    cache = lib.PagedKVCache(s["k_codes"], s["v_codes"], s["k_par"], s["v_par"], case["bits"])
    if case["op"] == "paged":
        return lib.qattn_paged_attention(s["q"], cache, s["table"], s["cu"], s["kv_len"], max_new=s["most_new"])
    out = {}
    if case["op"] == "cache":
        q, k, v = s["qkv"].split([case["Hq"], case["Hkv"], case["Hkv"]], 1)
        out["q"] = lib.qattn_cache_append(k, v, cache, s["table"], s["cu"], s["kv_len"],
                                          rotary=lib.Rotary(s["freq"], case["interleaved"]), q=q)
    out["k"], out["v"] = lib.qattn_cache_read(cache, s["table"], s["cu"], s["kv_len"], s["T"])
    return out


# ------------------------------------------------------------- plain form ----
def _to_half(x):
    """FP64 -> FP16 in one rounding (half to even)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -14))) - 10)
    return ((x / step).round() * step).half()


def _rotate(x, pos, freq, interleaved):
    """The first 2 * len(freq) channels of x [T, H, d] rotated, in 64 bits, rounded once."""
    n = freq.numel()
    a = pos.double()[:, None, None] * freq
    cos, sin = a.cos(), a.sin()
    r = x[..., :2 * n].double()
    x1, x2 = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :n], r[..., n:])
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([_to_half(y), x[..., 2 * n:]], -1)


def _places(s):
    """Of every new token: its position, its page and its place in the page."""
    t = torch.arange(s["T"], device=DEV)
    seq = torch.bucketize(t, s["cu"][1:].long(), right=True)
    pos = (s["kv_len"][seq] - s["cu"][seq + 1] + t).long()
    return pos, s["table"][seq, pos // s["case"]["page"]].long(), pos % s["case"]["page"]


def _weights(scores, seen):
    """Softmax over the seen keys; a row that sees none gets zeros."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top.masked_fill(top == -math.inf, 0.0)).exp_()
    return p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30))


def _plain_attention(q, k, v, seen):
    """q [B, n, Hq, d], k and v [B, L, Hkv, d], seen [B, n, L] -> [B, n, Hq, d], FP32."""
    B, n, Hq, d = q.shape
    Hkv = k.shape[2]
    q = q.float().transpose(1, 2).unflatten(1, (Hkv, Hq // Hkv))
    w = _weights(q @ k.permute(0, 2, 3, 1).unsqueeze(2) * d ** -0.5, seen[:, None, None])
    return (w @ v.transpose(1, 2).unsqueeze(2)).flatten(1, 2).transpose(1, 2)


def _padded(s, x):
    """Rows of the packed x [T, ...] as [B, most_new, ...], and where each packed row went."""
    i = torch.arange(s["most_new"], device=DEV)
    at = (s["cu"][:-1, None].long() + i).clamp(max=s["T"] - 1)
    t = torch.arange(s["T"], device=DEV)
    seq = torch.bucketize(t, s["cu"][1:].long(), right=True)
    return x[at], seq, t - s["cu"][seq].long()


def _plain(s):
    case = s["case"]
    if case["op"] == "rotary":
        return _rotate(s["x"], s["pos"], s["freq"], case["interleaved"])
    if case["op"] == "prompt":
        x, seq, i = _padded(s, s["qkv"])
        q, k, v = x.split([case["Hq"], case["Hkv"], case["Hkv"]], 2)
        n = torch.arange(s["most_new"], device=DEV)
        seen = (n[None, :] <= n[:, None])[None].expand(case["B"], -1, -1)
        return _plain_attention(q, k.float(), v.float(), seen)[seq, i].half()
    if case["op"] == "paged":
        q, seq, i = _padded(s, s["q"])
        j = torch.arange(s["most_kv"], device=DEV)
        page = s["table"][:, j // case["page"]].long()
        there = (j < s["kv_len"][:, None]) & (page >= 0)
        k, v = (_values(s[n + "_codes"][page.clamp(min=0), :, j % case["page"]], s[n + "_par"][page.clamp(min=0), :, j % case["page"]], case["bits"])
                for n in "kv")
        first = s["kv_len"] - (s["cu"][1:] - s["cu"][:-1])
        n = torch.arange(s["most_new"], device=DEV)
        seen = there[:, None] & (j <= first[:, None, None] + n[:, None])
        return _plain_attention(q, k, v, seen)[seq, i].half()
    pos, page, place = _places(s)
    out = {}
    if case["op"] == "cache":
        q, k, v = s["qkv"].split([case["Hq"], case["Hkv"], case["Hkv"]], 1)
        out["q"] = _rotate(q, pos, s["freq"], case["interleaved"])
        for n, x in (("k", _rotate(k, pos, s["freq"], case["interleaved"])), ("v", v)):
            c, p = _codes(x, case["bits"])
            s[n + "_codes"][page, :, place], s[n + "_par"][page, :, place] = _pack(c, case["bits"]), p
    for n in "kv":
        out[n] = _values(s[n + "_codes"][page, :, place], s[n + "_par"][page, :, place], case["bits"]).half()
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits ----
def _turned(x, pos, case):
    """Rotation as a product of complex numbers, per pair of channels."""
    n = case["rot"] // 2
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["interleaved"] else (slice(0, n), slice(n, 2 * n))
    y = x.double().clone()
    a = torch.outer(pos.double(), _freq(case))[:, None, :]
    z = torch.complex(y[..., one].clone(), y[..., two].clone()) * torch.polar(torch.ones_like(a), a)
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _nearest_half(x):
    """FP16 nearest to FP64 x, through numpy, which rounds once."""
    return torch.from_numpy(x.cpu().numpy().astype(np.float16)).to(x.device)


def _kept(x, bits):
    """What the cache holds of x FP16 [T, H, d], in 64 bits."""
    x = x.double()
    lo = x.min(-1, keepdim=True).values
    step = (x.max(-1, keepdim=True).values - lo) / (2 ** bits - 1)
    unit = torch.exp2(torch.floor(torch.log2(step.clamp(min=2.0 ** -14))) - 10)
    step = torch.floor(step / unit) * unit
    c = torch.round((x - lo) / torch.where(step == 0, torch.ones_like(step), step))
    return lo + torch.minimum(c, torch.full_like(c, 2 ** bits - 1)) * step


def _unpacked(rows, par, bits):
    r = rows.to(torch.int32)
    c = torch.empty(*r.shape[:-1], r.shape[-1] * 8 // bits, dtype=torch.float64, device=DEV)
    if bits == 4:
        c[..., 0::2], c[..., 1::2] = (r % 16).double(), torch.div(r, 16, rounding_mode="floor").double()
    else:
        c[:] = r.double()
    return c * par[..., 0:1].double() + par[..., 1:2].double()


def _attend(q, k, v, hidden):
    """One sequence: q [n, Hq, d], k and v [L, Hkv, d], hidden [n, L], all in 64 bits, in pieces of rows."""
    out = torch.zeros_like(q)
    G = q.shape[1] // k.shape[1]
    piece = max(1, int(2e8) // max(1, k.shape[0]))
    for h in range(q.shape[1]):
        for at in range(0, q.shape[0], piece):
            e = slice(at, at + piece)
            z = torch.einsum("nd,ld->nl", q[e, h], k[:, h // G]) / math.sqrt(q.shape[2])
            z[hidden[e]] = -math.inf
            w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            out[e, h] = w @ v[:, h // G]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _turned(s["x"], s["pos"], case)
    new, kv = _lens(case)
    start = [0] + [int(x) for x in np.cumsum(new)]
    if case["op"] == "prompt":
        out = []
        for b, n in enumerate(new):
            q, k, v = s["qkv"][start[b]:start[b + 1]].double().split([case["Hq"], case["Hkv"], case["Hkv"]], 1)
            out.append(_attend(q, k, v, torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)))
        return torch.cat(out)
    rows, _ = _pages(case)
    page = case["page"]
    if case["op"] == "paged":
        out = []
        for b, (n, L) in enumerate(zip(new, kv)):
            ids = torch.tensor(rows[b][: -(-L // page)], device=DEV)
            kb, vb = (_unpacked(s[x + "_codes"][ids.clamp(min=0)], s[x + "_par"][ids.clamp(min=0)], case["bits"])
                      .transpose(1, 2).flatten(0, 1)[:L] for x in "kv")
            hidden = torch.ones(n, L, dtype=torch.bool, device=DEV).triu(L - n + 1)
            hidden |= (ids < 0).repeat_interleave(page)[:L]
            out.append(_attend(s["q"][start[b]:start[b + 1]].double(), kb, vb, hidden))
        return torch.cat(out)
    pos = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(new, kv)])
    if case["op"] == "cache":
        q, k, v = s["qkv"].split([case["Hq"], case["Hkv"], case["Hkv"]], 1)
        return {"q": _turned(q, pos, case), "k": _kept(_nearest_half(_turned(k, pos, case)), case["bits"]), "v": _kept(v, case["bits"])}
    ids = torch.cat([torch.tensor([rows[b][p // page] for p in range(L - n, L)], device=DEV) for b, (n, L) in enumerate(zip(new, kv))])
    return {x: _unpacked(s[x + "_codes"][ids, :, pos % page], s[x + "_par"][ids, :, pos % page], case["bits"]) for x in "kv"}


# ------------------------------------------------------------------- work ----
def work(case):
    d = case["d"]
    if case["op"] == "rotary":
        n = case["T"] * case["H"] * d
        return {"bytes": 4 * n + 4 * case["T"] + 4 * case["rot"], "flops": 3 * case["T"] * case["H"] * case["rot"]}
    new, kv = _lens(case)
    T, Hq, Hkv = sum(new), case["Hq"], case["Hkv"]
    if case["op"] == "prompt":
        return {"bytes": 2 * T * d * (2 * Hq + 2 * Hkv), "flops": sum(2 * n * (n + 1) * d * Hq for n in new)}
    row = d * case["bits"] // 8 + 4
    if case["op"] == "read":
        return {"bytes": T * Hkv * 2 * (row + 2 * d), "flops": 4 * T * Hkv * d}
    if case["op"] == "cache":
        return {"bytes": T * (4 * Hq * d + 2 * Hkv * (2 * d + row) + 2 * Hkv * (row + 2 * d)),
                "flops": T * (3 * (Hq + Hkv) * case["rot"] + 10 * Hkv * d)}
    rows, _ = _pages(case)
    read, pairs = 0, 0
    for b, (n, L) in enumerate(zip(new, kv)):
        gone = [j for j, x in enumerate(rows[b]) if x < 0 and j * case["page"] < L]
        read += L - len(gone) * case["page"]
        pairs += n * (L - n) + n * (n + 1) // 2
        pairs -= sum(min(max(L - n + i + 1 - j * case["page"], 0), case["page"]) for j in gone for i in range(n))
    return {"bytes": 2 * read * Hkv * row + 4 * T * Hq * d, "flops": 4 * pairs * Hq * d}
