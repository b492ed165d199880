"""Cases of the decode-step operators over a paged cache (include/dmtp_ops.h).

Five operators, as one decode step of a served model calls them:

  write      rotary positions on new q and k rows, k and v stored in the paged cache
             (as they are, or as E4M3 rows with power-of-two scales)
  read       rows of the paged cache back as dense rows
  attention  1..8 new rows of each sequence over its paged cache
  norm       residual addition, RMS norm, E4M3 rows with power-of-two scales
  sample     temperature, top-k, top-p and min-p from one given uniform number per row

run() computes them from elementary torch operations, or, where `own` is set, through
the library. An E4M3 row is the framework's: scale 2^e with e the smallest integer such
that max|row| <= 448 * 2^e, values rounded to nearest even.
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
        # the new token of a decode step at the 32-sequence workload, 8-bit cache
        dict(name="write_decode", op="write", batch=32, rows=1, hq=32, hkv=4, hd=128, ps=64,
             lo=512, hi=4096, dtype="bf16", cache="e4m3", theta=10000.0),
        # a prefill of four prompts at the same model, bf16 cache
        dict(name="write_prefill", op="write", batch=4, rows=2047, hq=32, hkv=4, hd=128, ps=64,
             lo=0, hi=0, dtype="bf16", cache="bf16", theta=10000.0),
        # one short sequence's rows back from a bf16 cache (a request that moves)
        dict(name="read_short", op="read", batch=1, rows=37, hkv=16, hd=64, ps=16,
             dtype="bf16", cache="bf16"),
        # a shared prefix of 8 sequences back from an 8-bit cache
        dict(name="read_prefix", op="read", batch=8, rows=4096, hkv=2, hd=128, ps=64,
             dtype="bf16", cache="e4m3"),
        # one new token of one sequence at the smallest useful context: launch latency
        dict(name="attn_short", op="attention", batch=1, rows=1, hq=16, hkv=16, hd=64, ps=16,
             lo=77, hi=77, window=0, dtype="bf16", cache="bf16"),
        # the 32-sequence workload's ragged contexts, one new token each
        dict(name="attn_decode", op="attention", batch=32, rows=1, hq=32, hkv=4, hd=128, ps=64,
             lo=512, hi=4096, window=0, dtype="bf16", cache="bf16"),
        # the same contexts in 8 bits, the 8 rows of a verify
        dict(name="attn_verify_e4m3", op="attention", batch=32, rows=8, hq=32, hkv=4, hd=128,
             ps=64, lo=512, hi=4096, window=0, dtype="bf16", cache="e4m3"),
        # four long inputs, one new token each, 8-bit cache
        dict(name="attn_long_e4m3", op="attention", batch=4, rows=1, hq=32, hkv=4, hd=128, ps=16,
             lo=32768, hi=32768, window=0, dtype="bf16", cache="e4m3"),
        # between two sublayers of a decode step: fp32 residual stream
        dict(name="norm_decode", op="norm", n=32, d=2048, xtype="fp32", ytype="fp32"),
        # the same over a prefill's rows with bf16 streams
        dict(name="norm_prefill", op="norm", n=8188, d=2048, xtype="bf16", ytype="bf16"),
        # one sequence's next token under the usual filters
        dict(name="sample_one", op="sample", n=1, V=151936, ltype="fp32", t=0.7, k=50, p=0.9,
             m=0.0, spread=3.0),
        # every row of a verify: top-p and min-p over the whole vocabulary
        dict(name="sample_verify", op="sample", n=256, V=151936, ltype="fp32", t=1.0, k=0, p=0.95,
             m=0.01, spread=2.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


HEADS = ((32, 4, 128), (16, 16, 64), (16, 2, 128), (4, 4, 32), (8, 1, 64), (24, 8, 128),
         (5, 5, 64), (12, 4, 96), (8, 2, 256))


def draw(rng: random.Random):
    op = rng.choice(("write", "read", "attention", "attention", "norm", "sample"))
    if op == "norm":
        d = 8 * _log_int(rng, 16, 1024)
        return dict(op=op, n=_log_int(rng, 1, max(1, 8188 * 2048 // d)), d=d,
                    xtype=rng.choice(("fp32", "bf16")), ytype=rng.choice(("fp32", "bf16")))
    if op == "sample":
        V = _log_int(rng, 512, 151936)
        return dict(op=op, n=_log_int(rng, 1, 256), V=V, ltype=rng.choice(("fp32", "bf16")),
                    t=rng.choice((0.0, 0.3, 0.7, 1.0, 1.5)), k=rng.choice((0, 1, 20, 50, 1000)),
                    p=rng.choice((1.0, 0.95, 0.8, 0.5)), m=rng.choice((0.0, 0.02, 0.1)),
                    spread=round(rng.uniform(0.5, 4.0), 2))
    hq, hkv, hd = rng.choice(HEADS)
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    case = dict(op=op, hq=hq, hkv=hkv, hd=hd, ps=rng.choice((16, 32, 64, 128)), dtype=dtype,
                cache=rng.choice((dtype, "e4m3")))
    if op == "attention":
        rows = rng.choice((1, 1, 2, 5, 8))
        room = 4 * 32768 * 4 * 128 // (hkv * hd * (1 if rows * hq // hkv <= 16 else 4))
        room //= 4 if dtype == "fp32" or hd not in (64, 128) else 1
        hi = _log_int(rng, 16, min(32768, room))
        batch = _log_int(rng, 1, max(1, min(64, room // hi)))
        return dict(case, batch=batch, rows=rows, lo=rng.randint(rows, max(rows, hi)), hi=max(rows, hi),
                    window=rng.choice((0, 0, 0, rng.randint(1, hi))))
    if op == "write":
        rows = _log_int(rng, 1, 2047)
        n_room = 4 * 2047 * 40 * 128 // ((hq + 2 * hkv) * hd * (2 if dtype == "fp32" else 1))
        batch = _log_int(rng, 1, max(1, min(64, n_room // rows)))
        return dict(case, batch=batch, rows=min(rows, n_room), lo=0, hi=rng.choice((0, 1000, 4000)),
                    theta=rng.choice((0.0, 10000.0, 1000000.0)))
    del case["hq"]
    rows = _log_int(rng, 1, 4096)
    n_room = 8 * 4096 * 2 * 128 // (hkv * hd * (2 if dtype == "fp32" else 1))
    return dict(case, batch=_log_int(rng, 1, max(1, min(64, n_room // rows))), rows=min(rows, n_room))


# ---- inputs ---------------------------------------------------------------------------

def _e4m3_rows(x):
    """(values as E4M3, scales) of the rows of x (last dimension), computed in fp32."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    s = torch.where(amax > 0, torch.exp2(e.float().clamp(min=-126.0)), torch.ones_like(amax))
    return (x / s[..., None]).to(F8), s


def _pages(case, gen, blocks, fill):
    """Pages for case["batch"] sequences of `blocks` pages in a shuffled order."""
    B, hkv, hd, ps = case["batch"], case["hkv"], case["hd"], case["ps"]
    n = B * blocks
    shape = (n, hkv, ps, hd)
    c = {}
    for name in ("k", "v"):
        if not fill:
            x = torch.zeros(shape, device=DEV, dtype=TYPES[case["dtype"]])
            if case["cache"] == "e4m3":
                c[name], c[name + "_scale"] = x.to(F8), torch.ones(shape[:3], device=DEV)
            else:
                c[name], c[name + "_scale"] = x, None
            continue
        x = torch.randn(shape, device=DEV, generator=gen, dtype=torch.float32)
        x *= 0.5 + torch.rand((n, hkv, ps, 1), device=DEV, generator=gen)
        if case["cache"] == "e4m3":
            c[name], c[name + "_scale"] = _e4m3_rows(x)
        else:
            c[name], c[name + "_scale"] = x.to(TYPES[case["cache"]]), None
    c["table"] = torch.randperm(n, device=DEV, generator=gen).to(torch.int32).reshape(B, blocks)
    return c


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    host = np.random.RandomState(int(seed) % (1 << 31))
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        n, d = case["n"], case["d"]
        s["x"] = torch.randn((n, d), device=DEV, generator=gen).mul_(3.0).to(TYPES[case["xtype"]])
        s["y"] = torch.randn((n, d), device=DEV, generator=gen).to(TYPES[case["ytype"]])
        s["gain"] = (1 + 0.1 * torch.randn(d, device=DEV, generator=gen)).to(torch.bfloat16)
        s["x_out"] = torch.empty_like(s["x"])
        s["q"] = torch.empty((n, d), device=DEV, dtype=F8)
        s["scale"] = torch.empty(n, device=DEV)
        return s
    if op == "sample":
        n, V = case["n"], case["V"]
        s["logits"] = torch.randn((n, V), device=DEV, generator=gen).mul_(case["spread"]).to(
            TYPES[case["ltype"]])
        s["u"] = torch.rand(n, device=DEV, generator=gen)
        s["t"] = torch.full((n,), case["t"], device=DEV)
        s["k"] = torch.full((n,), case["k"], device=DEV, dtype=torch.int32)
        s["p"] = torch.full((n,), case["p"], device=DEV)
        s["m"] = torch.full((n,), case["m"], device=DEV)
        s["ids"] = torch.empty(n, device=DEV, dtype=torch.int32)
        s["kept"] = torch.empty(n, device=DEV, dtype=torch.int32)
        return s
    B, rows, hkv, hd, ps = case["batch"], case["rows"], case["hkv"], case["hd"], case["ps"]
    T = TYPES[case["dtype"]]
    if op == "read":
        s.update(_pages(case, gen, -(-rows // ps), True))
        s["seq"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(rows)
        s["pos"] = torch.arange(rows, device=DEV, dtype=torch.int32).repeat(B)
        s["k_out"] = torch.empty((B * rows, hkv, hd), device=DEV, dtype=T)
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    hq = case["hq"]
    base = host.randint(case["lo"], case["hi"] + 1, B)
    if op == "write":
        s.update(_pages(case, gen, -(-(int(case["hi"]) + rows) // ps), False))
        qkv = torch.randn((B * rows, (hq + 2 * hkv) * hd), device=DEV, generator=gen).to(T)
        s["qr"] = qkv[:, :hq * hd].view(B * rows, hq, hd)
        s["kr"] = qkv[:, hq * hd:(hq + hkv) * hd].view(B * rows, hkv, hd)
        s["vr"] = qkv[:, (hq + hkv) * hd:].view(B * rows, hkv, hd)
        s["seq"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(rows)
        s["pos"] = (torch.from_numpy(base).to(DEV)[:, None]
                    + torch.arange(rows, device=DEV)).reshape(-1).to(torch.int32)
        s["q_out"] = torch.empty((B * rows, hq, hd), device=DEV, dtype=T)
        return s
    s.update(_pages(case, gen, -(-int(case["hi"]) // ps), True))
    s["q"] = torch.randn((B, rows, hq, hd), device=DEV, generator=gen).mul_(2.0).to(T)
    s["len"] = torch.from_numpy(base.astype(np.int32)).to(DEV)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---- the plain forms ------------------------------------------------------------------

def _rotate(x, pos, theta):
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    ang = pos.double()[:, None] * freq
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_write(s):
    case = s["case"]
    q, k, v, pos = s["qr"].float(), s["kr"].float(), s["vr"].float(), s["pos"].long()
    if case["theta"]:
        q, k = _rotate(q, pos, case["theta"]), _rotate(k, pos, case["theta"])
    page, off = s["table"][s["seq"].long(), pos // case["ps"]].long(), pos % case["ps"]
    if case["cache"] == "e4m3":
        kq, ks = _e4m3_rows(k)
        vq, vs = _e4m3_rows(v)
        s["k"].view(torch.uint8)[page, :, off] = kq.view(torch.uint8)
        s["v"].view(torch.uint8)[page, :, off] = vq.view(torch.uint8)
        s["k_scale"][page, :, off], s["v_scale"][page, :, off] = ks, vs
    else:
        s["k"][page, :, off], s["v"][page, :, off] = k.to(s["k"].dtype), v.to(s["v"].dtype)
    return q.to(s["qr"].dtype)


def _plain_read(s):
    case = s["case"]
    pos = s["pos"].long()
    page, off = s["table"][s["seq"].long(), pos // case["ps"]].long(), pos % case["ps"]
    T = TYPES[case["dtype"]]
    if case["cache"] == "e4m3":
        k = s["k"].view(torch.uint8)[page, :, off].view(F8).float() * s["k_scale"][page, :, off][..., None]
        v = s["v"].view(torch.uint8)[page, :, off].view(F8).float() * s["v_scale"][page, :, off][..., None]
        return k.to(T), v.to(T)
    return s["k"][page, :, off].to(T), s["v"][page, :, off].to(T)


def _plain_attention(s):
    case = s["case"]
    q = s["q"].float()
    B, rows, hq, hd = q.shape
    hkv, ps, table = case["hkv"], case["ps"], s["table"].long()
    L = table.shape[1] * ps

    def dense(x, scale):
        x = (x.view(torch.uint8)[table].view(F8) if x.dtype == F8 else x[table]).float()
        if scale is not None:
            x = x * scale[table][..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, hkv, L, hd)

    j = torch.arange(L, device=q.device)
    at = s["len"].long()[:, None] - rows + torch.arange(rows, device=q.device)       # [B, rows]
    seen = j <= at[..., None]
    if case["window"]:
        seen &= j > at[..., None] - case["window"]
    there = (j < s["len"].long()[:, None])[:, None, :, None]
    k = torch.where(there, dense(s["k"], s["k_scale"]), 0.0)
    v = torch.where(there, dense(s["v"], s["v_scale"]), 0.0)
    g = hq // hkv
    qg = q.reshape(B, rows, hkv, g, hd).permute(0, 2, 1, 3, 4).reshape(B, hkv, rows * g, hd)
    sc = (qg @ k.transpose(-1, -2)) / math.sqrt(hd)
    seen = seen[:, None, :, None].expand(B, hkv, rows, g, L).reshape(B, hkv, rows * g, L)
    sc = sc.masked_fill(~seen, -math.inf)
    top = sc.amax(-1, keepdim=True)
    w = torch.exp(sc - torch.where(top.isinf(), torch.zeros_like(top), top))
    tot = w.sum(-1, keepdim=True)
    o = (w @ v) / torch.where(tot > 0, tot, torch.ones_like(tot))
    return o.reshape(B, hkv, rows, g, hd).permute(0, 2, 1, 3, 4).reshape(B, rows, hq, hd).to(s["q"].dtype)


def _plain_norm(s):
    x = s["x"].float() + s["y"].float()
    r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + 1e-6).float()
    q, scale = _e4m3_rows(x * r * s["gain"].float())
    return {"x": x.to(s["x"].dtype), "q": q, "scale": scale}


def _plain_sample(s):
    z = s["logits"].double()
    n, V = z.shape
    t = s["t"].double()[:, None]
    top = z.amax(-1, keepdim=True)
    w = torch.exp((z - top) / torch.where(t > 0, t, torch.ones_like(t)))
    zs, order = torch.sort(z, dim=-1, descending=True, stable=True)
    ws = w.gather(-1, order)
    rank = torch.arange(V, device=z.device)
    k = torch.where(s["k"] > 0, s["k"], V).long()[:, None]
    k = torch.where(t > 0, k, torch.ones_like(k))
    keep = (rank < k) & (zs > -math.inf)
    mass = torch.where(keep, ws, torch.zeros_like(ws))
    run_ = mass.cumsum(-1)
    p = s["p"].double()[:, None]
    keep &= (p >= 1) | (run_ - mass < p * run_[:, -1:]) | (rank == 0)
    keep &= ws >= s["m"].double()[:, None]
    kept = keep.sum(-1)
    w = torch.where(torch.zeros_like(keep).scatter_(-1, order, keep), w, torch.zeros_like(w))
    run_ = w.cumsum(-1)
    ids = (run_ <= s["u"].double()[:, None] * run_[:, -1:]).sum(-1)
    return {"ids": ids.to(torch.int32), "kept": kept.to(torch.int32)}


# ---- the library's calls --------------------------------------------------------------

def _cache(s):
    if "cache" not in s:  # the handle that a program makes once
        from mtp_block_draft_gb300 import DmtpPagedCache
        s["cache"] = DmtpPagedCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"],
                                    dtype=TYPES[s["case"]["dtype"]])
    return s["cache"]


def _own(s):
    case = s["case"]
    op = case["op"]
    if op == "write":
        _cache(s).write(s["kr"], s["vr"], s["seq"], s["pos"], q=s["qr"], q_out=s["q_out"],
                        rope_theta=case["theta"])
        return s["q_out"]
    if op == "read":
        return _cache(s).read(s["seq"], s["pos"], k_out=s["k_out"], v_out=s["v_out"])
    if op == "attention":
        return _cache(s).attention(s["q"], s["len"], window=case["window"], out=s["out"])
    if op == "norm":
        from mtp_block_draft_gb300 import add_rmsnorm_e4m3
        add_rmsnorm_e4m3(s["x"], s["y"], s["gain"], 1e-6, x_out=s["x_out"], q=s["q"],
                         scale=s["scale"])
        return {"x": s["x_out"], "q": s["q"], "scale": s["scale"]}
    from mtp_block_draft_gb300 import sample_rows
    sample_rows(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"],
                ids=s["ids"], kept=s["kept"])
    return {"ids": s["ids"], "kept": s["kept"]}


def run(state):
    op = state["case"]["op"]
    if own:
        r = _own(state)
    else:
        r = {"write": _plain_write, "read": _plain_read, "attention": _plain_attention,
             "norm": _plain_norm, "sample": _plain_sample}[op](state)
    if op == "write":  # the updated cache is the state's own
        return {"q": r, "k": state["k"], "v": state["v"], "k_scale": state["k_scale"],
                "v_scale": state["v_scale"]}
    if op == "read":
        return {"k": r[0], "v": r[1]}
    return r


# ---- the definitions in 64 bits -------------------------------------------------------

def _exact_e4m3(x):
    """Nearest-even E4M3 values and power-of-two scales of the rows of a float64 array, from
    the grid's spacing: 2^-9 up to 2^-6, then an eighth of the value's power of two."""
    amax = np.abs(x).max(-1)
    e = np.ceil(np.log2(np.maximum(amax, 1e-300) / 448.0))
    e = np.where(amax > 448.0 * 2.0 ** e, e + 1, e)
    e = np.where(amax <= 448.0 * 2.0 ** (e - 1), e - 1, e)
    sc = np.where(amax > 0, 2.0 ** np.maximum(e, -126.0), 1.0)
    y = x / sc[..., None]
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -20))) - 3, -9)
    return np.rint(y / step) * step, sc


def _np(x):
    return x.float().cpu().numpy().astype(np.float64)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "norm":
        x = _np(s["x"]) + _np(s["y"])
        h = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * _np(s["gain"])
        q, sc = _exact_e4m3(h)
        return {"x": x, "q": q, "scale": sc}
    if op == "sample":
        if case["n"] * case["V"] > 8_000_000:
            return None
        z, u = _np(s["logits"]), _np(s["u"])
        ids, kept = [], []
        t, k, p, m = (float(s[c][0]) for c in ("t", "k", "p", "m"))  # as the operator gets them
        for zr, ur in zip(z, u):
            if t <= 0:
                ids.append(int(np.argmax(zr)))
                kept.append(1)
                continue
            order = np.lexsort((np.arange(zr.size), -zr))
            if k > 0:
                order = order[:int(k)]
            w = np.exp((zr[order] - zr[order[0]]) / t)
            if p < 1:
                before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
                cut = max(1, int(np.searchsorted(before, p * w.sum(), side="left")))
                order, w = order[:cut], w[:cut]
            order = np.sort(order[w >= m])
            w = np.exp((zr[order] - zr[order].max()) / t)
            run_ = np.cumsum(w)
            ids.append(int(order[min(order.size - 1, np.searchsorted(run_, ur * run_[-1], side="right"))]))
            kept.append(order.size)
        return {"ids": np.array(ids, np.int32), "kept": np.array(kept, np.int32)}
    seq_pos = (s["seq"].long().cpu().numpy(), s["pos"].long().cpu().numpy()) if op != "attention" else None
    ps, table = case["ps"], s["table"].long().cpu().numpy()
    kc, vc = _np(s["k"]), _np(s["v"])
    if case["cache"] == "e4m3" and op != "write":
        kc, vc = kc * _np(s["k_scale"])[..., None], vc * _np(s["v_scale"])[..., None]
    if op == "read":
        page, off = table[seq_pos[0], seq_pos[1] // ps], seq_pos[1] % ps
        return {"k": kc[page, :, off], "v": vc[page, :, off]}
    if op == "write":
        q, k, v = _np(s["qr"]), _np(s["kr"]), _np(s["vr"])
        if case["theta"]:
            half = case["hd"] // 2
            turn = np.exp(1j * seq_pos[1][:, None] * case["theta"] ** (-np.arange(half) / half))[:, None]
            q, k = ((x[..., :half] + 1j * x[..., half:]) * turn for x in (q, k))
            q, k = (np.concatenate((x.real, x.imag), -1) for x in (q, k))
        page, off = table[seq_pos[0], seq_pos[1] // ps], seq_pos[1] % ps
        ks = vs = None
        if case["cache"] == "e4m3":
            ks, vs = _np(s["k_scale"]), _np(s["v_scale"])
            k, ks[page, :, off] = _exact_e4m3(k)
            v, vs[page, :, off] = _exact_e4m3(v)
        kc[page, :, off], vc[page, :, off] = k, v
        return {"q": q, "k": kc, "v": vc, "k_scale": ks, "v_scale": vs}
    q, lens = s["q"].double(), s["len"].tolist()
    B, rows, hq, hd = q.shape
    hkv = case["hkv"]
    o = torch.zeros_like(q)
    for b, n in enumerate(lens):
        got = table[b][:-(-n // ps)]
        k, v = (torch.from_numpy(np.moveaxis(c[got], 1, 0).reshape(hkv, -1, hd)[:, :n]).to(DEV)
                for c in (kc, vc))
        for i in range(rows):
            end = n - rows + i + 1
            first = max(0, end - case["window"]) if case["window"] else 0
            if end <= 0:
                continue
            a = torch.einsum("hgd,hld->hgl", q[b, i].view(hkv, hq // hkv, hd), k[:, first:end])
            a = torch.softmax(a / math.sqrt(hd), -1)
            o[b, i] = torch.einsum("hgl,hld->hgd", a, v[:, first:end]).reshape(hq, hd)
    return o.cpu().numpy()


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        n, d = case["n"], case["d"]
        return {"bytes": n * d * (2 * BYTES[case["xtype"]] + BYTES[case["ytype"]] + 1) + 2 * d + 4 * n,
                "flops": 8 * n * d}
    if op == "sample":
        return {"bytes": case["n"] * (case["V"] * BYTES[case["ltype"]] + 28),
                "flops": 4 * case["n"] * case["V"]}
    hkv, hd = case["hkv"], case["hd"]
    e8 = case["cache"] == "e4m3"
    t, cell = BYTES[case["dtype"]], BYTES[case["cache"]]
    row = 2 * hkv * (hd * cell + (4 if e8 else 0))          # one cached position
    n = case["batch"] * case["rows"]
    if op == "read":
        return {"bytes": n * (row + 2 * hkv * hd * t + 12), "flops": 2 * n * hkv * hd}
    hq = case["hq"]
    if op == "write":
        return {"bytes": n * ((2 * hq + 2 * hkv) * hd * t + row + 12), "flops": 6 * n * (hq + hkv) * hd}
    mean = (case["lo"] + case["hi"]) / 2
    seen = min(mean, case["window"] + case["rows"] - 1) if case["window"] else mean
    per_row = min(mean, case["window"]) if case["window"] else mean
    return {"bytes": case["batch"] * (seen * row + 4 * -(-case["hi"] // case["ps"])) + 2 * n * hq * hd * t,
            "flops": 4 * n * hq * hd * per_row}
