"""More cases over a paged K/V cache (include/dmtp_ops.h): other rotary layouts, rows in 4 bits,
capped and biased scores, whole prompts.

  rope    new q, k and v rows into the cache, rotated by interleaved or half pairs, of the whole
          head or its first part, at frequencies scaled for long contexts
  rows4   the same into a cache of E2M1 rows, and those rows read back
  attn    1..8 new rows of each sequence over its cache: E2M1 rows, and scores of any cache
          capped by a tanh or with a bias by distance
  prompt  any number of new rows of each sequence over its cache, with cap and bias, each row
          seeing an interval of positions (causal, documents, a prefix)

run() computes them from elementary torch operations, or, where `own` is set, through the
library. An E4M3 row has the scale 2^e, e the smallest integer with max|row| <= 448 2^e. An E2M1
row has s = 2^e, e the smallest with max|row| <= 2688 2^e, a scale b = E4M3(max|block| / 6s) for
each block of 16 columns, and values E2M1(x / (s b)); all round to nearest even. A page of E2M1
rows is [n_kv_heads][page_size][head_dim / 2] bytes, the lower column of a pair in the low half,
and behind them [n_kv_heads][page_size][head_dim / 16] E4M3 block scales.
"""
import math
import random

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": F8}
BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}
DEV = "cuda"


def listed():
    return [
        # a decode step's new tokens at the 32-sequence workload, interleaved pairs, bf16 cache
        dict(name="rope_decode", op="rope", batch=32, rows=1, hq=32, hkv=4, hd=128, ps=64, lo=512,
             hi=4096, dtype="bf16", cache="bf16", pairs="interleaved", dims=128, scaling="none"),
        # a prefill of four prompts, half of each head rotated, frequencies stretched eight times
        dict(name="rope_prefill", op="rope", batch=4, rows=2047, hq=32, hkv=4, hd=128, ps=64, lo=0,
             hi=30000, dtype="bf16", cache="e4m3", pairs="half", dims=64, scaling="ramp"),
        # a decode step's new tokens into a 4-bit cache and back
        dict(name="rows4_decode", op="rows4", batch=32, rows=1, hq=32, hkv=4, hd=128, ps=64,
             lo=512, hi=4096, dtype="bf16", cache="e2m1", pairs="half", dims=128, scaling="none"),
        # a prompt of one sequence into a 4-bit cache, and back as a shared prefix
        dict(name="rows4_prefill", op="rows4", batch=1, rows=4096, hq=32, hkv=4, hd=128, ps=64, lo=0,
             hi=0, dtype="bf16", cache="e2m1", pairs="interleaved", dims=128, scaling="turns"),
        # one short request on a model that caps its scores: launch latency
        dict(name="attn_cap_short", op="attn", batch=1, rows=1, hq=16, hkv=16, hd=64, ps=16, lo=77,
             hi=77, window=0, dtype="bf16", cache="bf16", cap=50.0, bias=False),
        # the 32-sequence workload's ragged contexts in 4 bits, one new token each
        dict(name="attn4_decode", op="attn", batch=32, rows=1, hq=32, hkv=4, hd=128, ps=64, lo=512,
             hi=4096, window=0, dtype="bf16", cache="e2m1", cap=0.0, bias=False),
        # long inputs in 4 bits, the 8 rows of a verify
        dict(name="attn4_verify", op="attn", batch=4, rows=8, hq=32, hkv=4, hd=128, ps=16, lo=30000,
             hi=32768, window=0, dtype="bf16", cache="e2m1", cap=0.0, bias=False),
        # the 32-sequence workload on a model with a bias by distance, the 8 rows of a verify
        dict(name="attn_bias_verify", op="attn", batch=32, rows=8, hq=32, hkv=4, hd=128, ps=64, lo=512,
             hi=4096, window=0, dtype="bf16", cache="bf16", cap=0.0, bias=True),
        # one short prompt of several documents
        dict(name="prompt_short", op="prompt", batch=1, lo=37, hi=37, past=0, hq=16, hkv=16, hd=64,
             ps=16, window=0, dtype="bf16", cache="bf16", cap=0.0, bias=False, mask="docs"),
        # four ragged prompts that each begin with a prefix seen both ways, capped scores
        dict(name="prompt_batch", op="prompt", batch=4, lo=1021, hi=2047, past=0, hq=32, hkv=4, hd=128,
             ps=64, window=0, dtype="bf16", cache="bf16", cap=30.0, bias=False, mask="prefix"),
        # chunks of two long prompts over what a 4-bit cache holds of them
        dict(name="prompt_chunk", op="prompt", batch=2, lo=512, hi=512, past=16384, hq=32, hkv=4,
             hd=128, ps=64, window=0, dtype="bf16", cache="e2m1", cap=0.0, bias=True, mask="causal"),
        # one long prompt
        dict(name="prompt_long", op="prompt", batch=1, lo=16384, hi=16384, past=0, hq=32, hkv=4, hd=128,
             ps=64, window=0, dtype="bf16", cache="bf16", cap=0.0, bias=False, mask="causal"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


HEADS = ((32, 4, 128), (16, 16, 64), (16, 2, 128), (4, 4, 32), (8, 1, 64), (24, 8, 128),
         (5, 5, 64), (12, 4, 96), (8, 2, 256))


def draw(rng: random.Random):
    op = rng.choice(("rope", "rows4", "attn", "attn", "prompt", "prompt"))
    hq, hkv, hd = rng.choice(HEADS)
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    cache = "e2m1" if op == "rows4" else rng.choice((dtype, "e4m3") if op == "rope" else (dtype, "e4m3", "e2m1"))
    case = dict(op=op, hq=hq, hkv=hkv, hd=hd, ps=rng.choice((16, 32, 64, 128)), dtype=dtype, cache=cache)
    slow = dtype == "fp32" or hd not in (64, 128)
    if op in ("rope", "rows4"):
        rows = _log_int(rng, 1, 2047)
        room = (4 * 2047 if op == "rope" else 2047) * 40 * 128 // ((hq + 2 * hkv) * hd * (2 if dtype == "fp32" else 1))
        batch = _log_int(rng, 1, max(1, min(64, room // rows)))
        return dict(case, batch=batch, rows=min(rows, room), lo=0, hi=rng.choice((0, 1000, 30000)),
                    pairs=rng.choice(("half", "interleaved")), dims=rng.choice((hd, hd // 2 // 16 * 16, 16)),
                    scaling=rng.choice(("none", "linear", "turns", "ramp")))
    cap = rng.choice((0.0, 30.0, 50.0))
    bias = rng.choice((False, True))
    if op == "attn":
        if cache != "e2m1" and not bias:
            cap = cap or 20.0
        rows = rng.choice((1, 1, 2, 5, 8))
        room = 4 * 32768 * 4 * 128 // (hkv * hd * (1 if rows * hq // hkv <= 16 else 4))
        room //= 4 if slow else 1
        hi = _log_int(rng, 16, min(32768, room))
        batch = _log_int(rng, 1, max(1, min(64, room // hi)))
        return dict(case, batch=batch, rows=rows, lo=rng.randint(rows, max(rows, hi)), hi=max(rows, hi),
                    window=rng.choice((0, 0, 0, rng.randint(1, hi))), cap=cap, bias=bias)
    # as many products as the longest listed prompt at most, an eighth of that on the CUDA cores
    pairs = 16384 * 16384 // 2 * 32 * 128 // (hq * max(hd, 128) * (8 if slow else 1))
    past = rng.choice((0, 0, _log_int(rng, 16, 16384)))
    hi = _log_int(rng, 1, min(8192, max(1, pairs // max(1, past)), math.isqrt(pairs)))
    batch = _log_int(rng, 1, max(1, min(16, pairs // (hi * (hi + past)))))
    return dict(case, batch=batch, lo=rng.randint(1, hi), hi=hi, past=past, cap=cap, bias=bias,
                window=rng.choice((0, 0, 0, rng.randint(1, hi + past))),
                mask=rng.choice(("causal", "causal", "docs", "prefix")))


# ---- rotary frequencies ---------------------------------------------------------------

ROPE = dict(theta=10000.0, factor=8.0, orig_len=4096, low=1.0, high=32.0)


def _amplitude(case):
    return 0.1 * math.log(ROPE["factor"]) + 1.0 if case["scaling"] == "ramp" else 1.0


def _frequencies(case):
    r, half = case["dims"], case["dims"] // 2
    f = ROPE["theta"] ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    if case["scaling"] == "none":
        return f
    slow = f / ROPE["factor"]
    if case["scaling"] == "linear":
        return slow
    if case["scaling"] == "turns":
        keep = ((ROPE["orig_len"] * f / (2 * math.pi) - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0, 1)
    else:
        a, b = (r * math.log(ROPE["orig_len"] / (2 * math.pi * n)) / (2 * math.log(ROPE["theta"]))
                for n in (ROPE["high"], ROPE["low"]))
        a, b = min(max(math.floor(a), 0), r - 1), min(max(math.ceil(b), 0), r - 1)
        at = torch.arange(half, device=DEV, dtype=torch.float64)
        keep = 1 - ((at - a) / max(b - a, 0.001)).clamp(0, 1)
    return f * keep + slow * (1 - keep)


# ---- inputs ---------------------------------------------------------------------------

def _e4m3_rows(x):
    """(values as E4M3, scales) of the rows of x (last dimension), computed in fp32."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    s = torch.where(amax > 0, torch.exp2(e.float().clamp(min=-126.0)), torch.ones_like(amax))
    return (x / s[..., None]).to(F8), s


def _e2m1_rows(x):
    """(codes 0..15, block scales as E4M3, row scales) of the rows of x, computed in fp32."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)                       # 2688 = 0.65625 * 2^12
    e = torch.where(m <= 0.65625, e - 12, e - 11)
    s = torch.where(amax > 0, torch.exp2(e.float().clamp(min=-126.0)), torch.ones_like(amax))
    y = (x / s[..., None]).unflatten(-1, (-1, 16))
    b = (y.abs().amax(-1) / 6).to(F8)
    bf = b.float()[..., None]
    y = y / torch.where(bf > 0, bf, torch.ones_like(bf))
    y = torch.where(bf > 0, y, torch.zeros_like(y)).flatten(-2)
    a = y.abs()
    code = sum(((a > t) if up else (a >= t)).to(torch.uint8)
               for t, up in ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)))
    return code + 8 * (y < 0).to(torch.uint8), b, s


def _e2m1_values(code, b, s):
    mag = (code & 7).float()
    v = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    v = torch.where(code > 7, -v, v)
    return (v.unflatten(-1, (-1, 16)) * b.float()[..., None]).flatten(-2) * s[..., None]


def _split(case, pages):
    """The packed values and the block scales (as bytes) of E2M1 pages, as views."""
    hkv, ps, hd = case["hkv"], case["ps"], case["hd"]
    n = hkv * ps * hd // 2
    return pages[:, :n].view(-1, hkv, ps, hd // 2), pages[:, n:].view(-1, hkv, ps, hd // 16)


def _pages(case, gen, blocks, fill):
    """Pages for case["batch"] sequences of `blocks` pages in a shuffled order."""
    B, hkv, hd, ps = case["batch"], case["hkv"], case["hd"], case["ps"]
    n = B * blocks
    shape = (n, hkv, ps, hd)
    c = {}
    for name in ("k", "v"):
        if not fill:
            c[name + "_scale"] = None if case["cache"] in ("bf16", "fp32") else torch.ones(shape[:3], device=DEV)
            if case["cache"] == "e2m1":
                c[name] = torch.zeros((n, hkv * ps * hd * 9 // 16), device=DEV, dtype=torch.uint8)
            else:
                c[name] = torch.zeros(shape, device=DEV, dtype=torch.float32).to(TYPES[case["cache"]])
            continue
        x = torch.randn(shape, device=DEV, generator=gen, dtype=torch.float32)
        x *= 0.5 + torch.rand((n, hkv, ps, 1), device=DEV, generator=gen)
        if case["cache"] == "e2m1":
            code, b, c[name + "_scale"] = _e2m1_rows(x)
            c[name] = torch.cat(((code[..., ::2] | code[..., 1::2] << 4).flatten(1), b.view(torch.uint8).flatten(1)), 1)
        elif case["cache"] == "e4m3":
            c[name], c[name + "_scale"] = _e4m3_rows(x)
        else:
            c[name], c[name + "_scale"] = x.to(TYPES[case["cache"]]), None
    c["table"] = torch.randperm(n, device=DEV, generator=gen).to(torch.int32).reshape(B, blocks)
    return c


def _rows_of(case):
    """The prompts' rows, spread from lo to hi."""
    B = case["batch"]
    return [case["lo"] + (case["hi"] - case["lo"]) * (b + 1) // B for b in range(B)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    op, B, hq, hkv, hd, ps = (case[n] for n in ("op", "batch", "hq", "hkv", "hd", "ps"))
    T = TYPES[case["dtype"]]
    s = {"case": case}
    if op in ("rope", "rows4"):
        rows = case["rows"]
        base = host.randint(case["lo"], case["hi"] + 1, B)
        s.update(_pages(case, gen, -(-(int(case["hi"]) + rows) // ps), False))
        qkv = torch.randn((B * rows, (hq + 2 * hkv) * hd), device=DEV, generator=gen).to(T)
        s["qr"] = qkv[:, :hq * hd].view(B * rows, hq, hd)
        s["kr"] = qkv[:, hq * hd:(hq + hkv) * hd].view(B * rows, hkv, hd)
        s["vr"] = qkv[:, (hq + hkv) * hd:].view(B * rows, hkv, hd)
        s["seq"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(rows)
        s["pos"] = (torch.from_numpy(base).to(DEV)[:, None]
                    + torch.arange(rows, device=DEV)).reshape(-1).to(torch.int32)
        s["q_out"] = torch.empty((B * rows, hq, hd), device=DEV, dtype=T)
        if op == "rows4":
            s["k_out"] = torch.empty((B * rows, hkv, hd), device=DEV, dtype=T)
            s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["slopes"] = None
    if case["bias"]:
        s["slopes"] = torch.exp2(-8.0 * (torch.arange(hq, device=DEV, dtype=torch.float32) + 1) / hq)
    if op == "attn":
        rows = case["rows"]
        s.update(_pages(case, gen, -(-int(case["hi"]) // ps), True))
        s["q"] = torch.randn((B, rows, hq, hd), device=DEV, generator=gen).mul_(2.0).to(T)
        s["len"] = torch.from_numpy(host.randint(case["lo"], case["hi"] + 1, B).astype(np.int32)).to(DEV)
        s["out"] = torch.empty_like(s["q"])
        return s
    rows = np.array(_rows_of(case), np.int64)
    past = host.randint(case["past"] * 3 // 4, case["past"] + 1, B)
    s.update(_pages(case, gen, -(-(int(case["past"]) + case["hi"]) // ps), True))
    n = int(rows.sum())
    s["q"] = torch.randn((n, hq, hd), device=DEV, generator=gen).mul_(2.0).to(T)
    s["len"] = torch.from_numpy((past + rows).astype(np.int32)).to(DEV)
    s["start"] = torch.from_numpy(np.concatenate(([0], np.cumsum(rows))).astype(np.int32)).to(DEV)
    s["first"] = s["end"] = None
    at = np.concatenate([p + np.arange(r) for p, r in zip(past, rows)])        # positions of the rows
    if case["mask"] == "docs":  # documents of a geometric length, a fifth of the context on average
        mean = max(2, (case["past"] + case["hi"]) // 5)
        first = []
        for p, r in zip(past, rows):
            new = host.rand(p + r) < 1.0 / mean
            first.append(np.maximum.accumulate(np.where(new, np.arange(p + r), 0))[p:])
        s["first"] = torch.from_numpy(np.concatenate(first).astype(np.int32)).to(DEV)
    if case["mask"] == "prefix":  # a third of the context, as far as it is there
        both = np.repeat((past + rows) // 3, rows)
        s["end"] = torch.from_numpy(np.maximum(at + 1, both).astype(np.int32)).to(DEV)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---- the plain forms ------------------------------------------------------------------

def _rotate(case, x, pos):
    r = case["dims"]
    ang = pos.double()[:, None] * _frequencies(case)
    cos, sin = ((f(ang) * _amplitude(case)).float()[:, None] for f in (torch.cos, torch.sin))
    if case["pairs"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., :r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_rope(s):
    case = s["case"]
    pos = s["pos"].long()
    q, k, v = _rotate(case, s["qr"].float(), pos), _rotate(case, s["kr"].float(), pos), s["vr"].float()
    page, off = s["table"][s["seq"].long(), pos // case["ps"]].long(), pos % case["ps"]
    if case["cache"] == "e2m1":
        for x, name in ((k, "k"), (v, "v")):
            code, b, s[name + "_scale"][page, :, off] = _e2m1_rows(x)
            val, blk = _split(case, s[name])
            val[page, :, off] = code[..., ::2] | code[..., 1::2] << 4
            blk[page, :, off] = b.view(torch.uint8)
    elif case["cache"] == "e4m3":
        for x, name in ((k, "k"), (v, "v")):
            y, s[name + "_scale"][page, :, off] = _e4m3_rows(x)
            s[name].view(torch.uint8)[page, :, off] = y.view(torch.uint8)
    else:
        s["k"][page, :, off], s["v"][page, :, off] = k.to(s["k"].dtype), v.to(s["v"].dtype)
    return q.to(s["qr"].dtype)


def _values(case, pages, scale, at):
    """fp32 rows of the pages that `at` picks."""
    if case["cache"] == "e2m1":
        val, blk = _split(case, pages)
        val, blk = val[at], blk[at].view(F8)
        return _e2m1_values(torch.stack((val & 15, val >> 4), -1).flatten(-2), blk, scale[at])
    if case["cache"] == "e4m3":
        return pages.view(torch.uint8)[at].view(F8).float() * scale[at][..., None]
    return pages[at].float()


def _plain_read(s):
    case = s["case"]
    pos = s["pos"].long()
    at = (s["table"][s["seq"].long(), pos // case["ps"]].long(), slice(None), pos % case["ps"])
    T = TYPES[case["dtype"]]
    return _values(case, s["k"], s["k_scale"], at).to(T), _values(case, s["v"], s["v_scale"], at).to(T)


def _attend(s, q, at, lo, hi):
    """Rows q [B, R, hq, hd] at positions `at`, seeing lo <= j < hi ([B, R] each)."""
    case = s["case"]
    B, R, hq, hd = q.shape
    hkv, table = case["hkv"], s["table"].long()
    L = table.shape[1] * case["ps"]
    g = hq // hkv
    j = torch.arange(L, device=q.device)
    there = (j < s["len"].long()[:, None])[:, None, :, None]

    def dense(x, scale):
        x = _values(case, x, scale, table)
        return torch.where(there, x.permute(0, 2, 1, 3, 4).reshape(B, hkv, L, hd), 0.0)

    qg = q.reshape(B, R, hkv, g, hd).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * R, hd)
    sc = (qg @ dense(s["k"], s["k_scale"]).transpose(-1, -2)).mul_(1 / math.sqrt(hd)).view(B, hkv, g, R, L)
    if case["cap"]:
        sc = sc.div_(case["cap"]).tanh_().mul_(case["cap"])
    if s["slopes"] is not None:
        far = (at[..., None] - j).abs().float()[:, None, None]
        sc.addcmul_(far, s["slopes"].view(1, hkv, g, 1, 1), value=-1.0)
    seen = (j >= lo[..., None]) & (j < hi[..., None])
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    tot = sc.sum(-1, keepdim=True)
    o = (sc.view(B, hkv, g * R, L) @ dense(s["v"], s["v_scale"])).view(B, hkv, g, R, hd)
    o = o / torch.where(tot > 0, tot, torch.ones_like(tot))
    return o.permute(0, 3, 1, 2, 4).reshape(B, R, hq, hd)


def _plain_attn(s):
    case = s["case"]
    rows = case["rows"]
    at = s["len"].long()[:, None] - rows + torch.arange(rows, device=DEV)
    lo = at - case["window"] + 1 if case["window"] else torch.zeros_like(at)
    return _attend(s, s["q"].float(), at, lo, at + 1).to(s["q"].dtype)


def _plain_prompt(s):
    case = s["case"]
    q, n = s["q"], s["q"].shape[0]
    B, R = case["batch"], case["hi"]
    start = s["start"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(R, device=DEV)
    live = i < count[:, None]
    row = torch.where(live, start[:-1, None] + i, n - 1)                       # [B, R]
    at = s["len"].long()[:, None] - count[:, None] + i
    hi = at + 1 if s["end"] is None else s["end"].long()[row]
    hi = torch.minimum(hi, s["len"].long()[:, None])
    lo = torch.zeros_like(at) if s["first"] is None else s["first"].long()[row]
    if case["window"]:
        lo = torch.maximum(lo, at - case["window"] + 1)
    o = _attend(s, q[row].float(), at, lo, hi)
    return o[live].to(q.dtype)


# ---- the library's calls --------------------------------------------------------------

def _cache(s):
    if "cache" not in s:  # the handle that a program makes once
        from mtp_block_draft_gb300 import DmtpPagedCache
        s["cache"] = DmtpPagedCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"],
                                    dtype=TYPES[s["case"]["dtype"]])
    return s["cache"]


def _rope(s):
    if "rope" not in s:  # the same
        from mtp_block_draft_gb300 import DmtpRope
        case = s["case"]
        how = {} if case["scaling"] == "none" else dict(ROPE, scaling=case["scaling"])
        s["rope"] = DmtpRope(**{**dict(theta=ROPE["theta"]), **how}, dims=case["dims"],
                             interleaved=case["pairs"] == "interleaved", amplitude=_amplitude(case))
    return s["rope"]


def _own(s):
    case = s["case"]
    op = case["op"]
    c = _cache(s)
    if op in ("rope", "rows4"):
        c.write(s["kr"], s["vr"], s["seq"], s["pos"], q=s["qr"], q_out=s["q_out"], rope=_rope(s))
        return s["q_out"]
    if op == "attn":
        return c.attention(s["q"], s["len"], window=case["window"], cap=case["cap"], slopes=s["slopes"],
                           out=s["out"])
    return c.prompt_attention(s["q"], s["start"], s["len"], window=case["window"], cap=case["cap"],
                              slopes=s["slopes"], first=s["first"], end=s["end"], out=s["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        r = _own(state)
    else:
        r = {"rope": _plain_rope, "rows4": _plain_rope, "attn": _plain_attn, "prompt": _plain_prompt}[op](state)
    if op == "rope":  # the updated cache is the state's own
        return {"q": r, "k": state["k"], "v": state["v"], "k_scale": state["k_scale"],
                "v_scale": state["v_scale"]}
    if op == "rows4":
        if own:
            k, v = state["cache"].read(state["seq"], state["pos"], k_out=state["k_out"], v_out=state["v_out"])
        else:
            k, v = _plain_read(state)
        return {"q": r, "k": k, "v": v}
    return r


# ---- the definitions in 64 bits -------------------------------------------------------

def _np(x):
    return x.float().cpu().numpy().astype(np.float64)


def _grid(y, lowest, bits):
    """Nearest-even value with `bits` bits behind the leading one, spacing 2^lowest at least."""
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -40))) - bits, lowest)
    return np.rint(y / step) * step


def _scale_of(amax, top):
    """The smallest power of two whose `top` multiple reaches amax; 1 for 0."""
    e = np.ceil(np.log2(np.maximum(amax, 1e-300) / top))
    e = np.where(amax > top * 2.0 ** e, e + 1, e)
    e = np.where(amax <= top * 2.0 ** (e - 1), e - 1, e)
    return np.where(amax > 0, 2.0 ** np.maximum(e, -126.0), 1.0)


def _exact_e4m3(x):
    sc = _scale_of(np.abs(x).max(-1), 448.0)
    return _grid(x / sc[..., None], -9, 3), sc


def _exact_e2m1(x):
    """What E2M1 rows of x stand for."""
    sc = _scale_of(np.abs(x).max(-1), 2688.0)[..., None, None]
    y = x.reshape(*x.shape[:-1], -1, 16) / sc
    b = _grid(np.abs(y).max(-1, keepdims=True) / 6.0, -9, 3)
    z = np.where(b > 0, y / np.where(b > 0, b, 1.0), 0.0)
    return (np.clip(_grid(np.clip(z, -6.0, 6.0), -1, 1), -6.0, 6.0) * b * sc).reshape(x.shape)


def _cached(case, s, name):
    """Every row of the pages in 64 bits, [n_pages, n_kv_heads, page_size, head_dim]."""
    if case["cache"] != "e2m1":
        x = _np(s[name])
        return x if case["cache"] != "e4m3" else x * _np(s[name + "_scale"])[..., None]
    hkv, ps, hd = case["hkv"], case["ps"], case["hd"]
    raw = s[name].cpu().numpy()
    half = hkv * ps * hd // 2
    nib = np.empty((raw.shape[0], half * 2), np.int64)
    nib[:, 0::2], nib[:, 1::2] = raw[:, :half] & 15, raw[:, :half] >> 4
    level = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    v = np.concatenate((level, -level))[nib].reshape(-1, hkv, ps, hd // 16, 16)
    u = raw[:, half:].astype(np.int64)
    b = np.where(u >> 3 == 0, (u & 7) * 2.0 ** -9, (1 + (u & 7) / 8) * 2.0 ** ((u >> 3) - 7.0))
    v = v * b.reshape(-1, hkv, ps, hd // 16, 1)
    return v.reshape(-1, hkv, ps, hd) * _np(s[name + "_scale"])[..., None]


def exact(case, seed):
    op = case["op"]
    if work(case)["flops"] > 5e11:
        return None
    s = prepare(case, seed)
    ps, hkv, table = case["ps"], case["hkv"], s["table"].long().cpu().numpy()
    if op in ("rope", "rows4"):
        seq, pos = s["seq"].long().cpu().numpy(), s["pos"].long().cpu().numpy()
        q, k, v = _np(s["qr"]), _np(s["kr"]), _np(s["vr"])
        f = _frequencies(case).cpu().numpy()
        turn = (np.exp(1j * pos[:, None] * f) * _amplitude(case))[:, None]
        r, h = case["dims"], case["dims"] // 2
        for x in (q, k):
            ia, ib = (slice(0, h), slice(h, r)) if case["pairs"] == "half" else (slice(0, r, 2), slice(1, r, 2))
            z = (x[..., ia] + 1j * x[..., ib]) * turn
            x[..., ia], x[..., ib] = z.real, z.imag
        if op == "rows4":
            return {"q": q, "k": _exact_e2m1(k), "v": _exact_e2m1(v)}
        page, off = table[seq, pos // ps], pos % ps
        kc, vc = _np(s["k"]), _np(s["v"])
        ks = vs = None
        if case["cache"] == "e4m3":
            ks, vs = _np(s["k_scale"]), _np(s["v_scale"])
            k, ks[page, :, off] = _exact_e4m3(k)
            v, vs[page, :, off] = _exact_e4m3(v)
        kc[page, :, off], vc[page, :, off] = k, v
        return {"q": q, "k": kc, "v": vc, "k_scale": ks, "v_scale": vs}
    q, lens = s["q"].double(), s["len"].tolist()
    hq, hd = q.shape[-2:]
    g = hq // hkv
    slope = None if s["slopes"] is None else s["slopes"].double().view(hkv, g, 1, 1)
    kc, vc = _cached(case, s, "k"), _cached(case, s, "v")
    o = torch.zeros_like(q)
    start = None if op == "attn" else s["start"].tolist()
    for b, n in enumerate(lens):
        got = table[b][:-(-n // ps)]
        k, v = (torch.from_numpy(np.ascontiguousarray(np.moveaxis(c[got], 1, 0).reshape(hkv, -1, hd)[:, :n])).to(DEV)
                for c in (kc, vc))
        rows = slice(0, case["rows"]) if op == "attn" else slice(start[b], start[b + 1])
        count = rows.stop - rows.start
        qb = q[b] if op == "attn" else q[rows]
        res = torch.zeros_like(qb)
        for i0 in range(0, count, 256):  # 256 rows at a time
            i1 = min(count, i0 + 256)
            p = torch.arange(n - count + i0, n - count + i1, device=DEV)[:, None]
            j = torch.arange(n, device=DEV)[None]
            see = j <= p
            if op == "prompt" and s["end"] is not None:
                see = j < s["end"][rows][i0:i1, None]
            if op == "prompt" and s["first"] is not None:
                see = see & (j >= s["first"][rows][i0:i1, None])
            if case["window"]:
                see = see & (p - j < case["window"])
            a = torch.einsum("rhgd,hld->hgrl", qb[i0:i1].reshape(-1, hkv, g, hd), k) / math.sqrt(hd)
            if case["cap"]:
                a = case["cap"] * torch.tanh(a / case["cap"])
            if slope is not None:
                a = a - slope * (p - j).abs()
            a = torch.softmax(a.masked_fill(~see, -math.inf), -1).masked_fill(~see.any(-1, keepdim=True), 0.0)
            res[i0:i1] = torch.einsum("hgrl,hld->rhgd", a, v).reshape(-1, hq, hd)
        if op == "attn":
            o[b] = res
        else:
            o[rows] = res
    return o.cpu().numpy()


# ---- what a pass cannot do without ----------------------------------------------------

def _row_bytes(case):
    """One cached position, k and v."""
    hkv, hd = case["hkv"], case["hd"]
    if case["cache"] == "e2m1":
        return 2 * hkv * (hd * 9 // 16 + 4)
    return 2 * hkv * (hd * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0))


def work(case):
    op, hq, hkv, hd, B = (case[n] for n in ("op", "hq", "hkv", "hd", "batch"))
    t, row = BYTES[case["dtype"]], _row_bytes(case)
    if op in ("rope", "rows4"):
        n = B * case["rows"]
        back = 2 * hkv * hd * t + row if op == "rows4" else 0
        return {"bytes": n * ((2 * hq + 2 * hkv) * hd * t + row + 8 + back), "flops": 6 * n * (hq + hkv) * hd}
    if op == "attn":
        n = B * case["rows"]
        mean = (case["lo"] + case["hi"]) / 2
        seen = min(mean, case["window"] + case["rows"] - 1) if case["window"] else mean
        per_row = min(mean, case["window"]) if case["window"] else mean
        return {"bytes": B * (seen * row + 4 * -(-case["hi"] // case["ps"])) + 2 * n * hq * hd * t,
                "flops": 4 * n * hq * hd * per_row}
    rows = _rows_of(case)
    past = case["past"] * 7 / 8
    pairs = 0.0
    for r in rows:
        mean = past + (r + 1) / 2                       # positions that a row sees
        if case["mask"] == "docs":
            mean = min(mean, max(2, (case["past"] + case["hi"]) // 5))
        if case["mask"] == "prefix":
            both = (past + r) / 3
            mean += max(0.0, both - past) ** 2 / (2 * r)
        pairs += r * (min(mean, case["window"]) if case["window"] else mean)
    cached = sum(min(past + r, case["window"] + r) if case["window"] else past + r for r in rows)
    return {"bytes": cached * row + 2 * sum(rows) * hq * hd * t, "flops": 4 * hq * hd * pairs}
