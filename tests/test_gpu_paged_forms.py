"""The paged cache's other forms on the GPU, against float64: rotary layouts and frequencies, rows in
4 bits, capped and biased scores, attention of many rows.

Tolerances are derived, as in test_gpu_decode_ops.py: a rounding to a type is off by at most half a
step (fp32 2^-24, bf16 2^-8 of the value), and the arithmetic before it is counted where each bound
is formed.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_decode_ops import BF, F8, FP, HALF, U, gen, i32, np64, randn

pytestmark = pytest.mark.gpu

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
ROWS = ["raw", "e4m3", "e2m1"]
KINDS = [(d, r) for d in (BF, FP) for r in ROWS]


def new_cache(B, blocks, ps, hkv, hd, dtype=BF, rows="raw", seed=0, extra=3, poison=True):
    """A cache whose sequences own shuffled pages, every slot of it poisoned with NaN."""
    from mtp_block_draft_gb300 import DmtpPagedCache
    n = B * blocks + extra
    perm = np.random.RandomState(seed).permutation(n)[:B * blocks].astype(np.int32)
    table = torch.from_numpy(perm.reshape(B, blocks)).cuda()
    c = DmtpPagedCache.alloc(n, ps, hkv, hd, table, dtype=dtype, e4m3=rows == "e4m3", e2m1=rows == "e2m1")
    if poison:
        for t in (c.k, c.v):
            if rows == "raw":
                t.fill_(float("nan"))
            else:
                t.view(torch.uint8).fill_(0x7f)
    return c


def e4m3_values(u):
    u = u.astype(np.int64)
    mag = np.where(u & 0x78, (1 + (u & 7) / 8) * 2.0 ** (((u >> 3) & 15) - 7.0), (u & 7) * 2.0 ** -9)
    mag = np.where((u & 0x7f) == 0x7f, np.nan, mag)
    return np.where(u & 0x80, -mag, mag)


def pages64(c, which):
    """Every row of the pages in float64, [n_pages, hkv, ps, hd]."""
    x, s = (c.k, c.k_scale) if which == "k" else (c.v, c.v_scale)
    if s is None:
        return np64(x)
    n, h, ps = s.shape
    if x.dtype is F8:
        return np64(x) * np64(s)[..., None]
    raw, cut = x.cpu().numpy(), h * ps * c.head_dim // 2
    code = np.stack((raw[:, :cut] & 15, raw[:, :cut] >> 4), -1)
    v = np.concatenate((LEVELS, -LEVELS))[code].reshape(n, h, ps, c.head_dim // 16, 16)
    v = v * e4m3_values(raw[:, cut:]).reshape(n, h, ps, c.head_dim // 16, 1)
    return v.reshape(n, h, ps, c.head_dim) * np64(s)[..., None]


def stored(c, lens):
    table, ps = c.table.cpu().numpy(), c.c.page_size
    k, v = pages64(c, "k"), pages64(c, "v")
    return [[np.moveaxis(x[table[b][:-(-max(n, 0) // ps)]], 1, 0).reshape(c.n_kv_heads, -1, c.head_dim)[:, :max(n, 0)]
             for x in (k, v)] for b, n in enumerate(lens)]


def fill_cache(c, lens, g, kmul=1.0):
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [[]]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens] + [[]]).astype(np.int32)
    n = len(seq)
    if n:
        spread = 0.25 + 2 * torch.rand((n, c.n_kv_heads, 1), device="cuda", generator=g)
        k = (torch.randn((n, c.n_kv_heads, c.head_dim), device="cuda", generator=g) * spread * kmul)
        v = torch.randn((n, c.n_kv_heads, c.head_dim), device="cuda", generator=g) * spread
        c.write(k.to(c.dtype), v.to(c.dtype), i32(seq), i32(pos))
    return stored(c, lens)


# ---- rotary positions -----------------------------------------------------------------

def frequencies(dims, theta, scaling=None, factor=1.0, orig_len=0.0, low=1.0, high=32.0):
    i = np.arange(dims // 2, dtype=np.longdouble)
    f = np.longdouble(theta) ** (-2 * i / dims)
    if scaling is None:
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "turns":
        w = np.clip((orig_len * f / (2 * np.pi) - low) / (high - low), 0, 1)
    else:
        at = [dims * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
        a, b = (min(max(x, 0), dims - 1) for x in (math.floor(at[0]), math.ceil(at[1])))
        w = 1 - np.clip((i - a) / max(b - a, 0.001), 0, 1)
    return w * f + (1 - w) * f / factor


def rotated(x, pos, dims, interleaved, amplitude, freq):
    ang = (np.asarray(pos, np.longdouble)[:, None] * freq)[:, None]
    c, s = ((fn(ang) * np.longdouble(np.float32(amplitude))).astype(np.float64) for fn in (np.cos, np.sin))
    out = x.copy()
    a, b = (slice(0, dims, 2), slice(1, dims, 2)) if interleaved else (slice(0, dims // 2), slice(dims // 2, dims))
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return out


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="turns", factor=8.0, orig_len=4096, low=1.0, high=4.0),
            dict(scaling="ramp", factor=16.0, orig_len=2048, low=1.0, high=32.0)]


@pytest.mark.parametrize("dtype,rows", [(BF, "raw"), (FP, "raw"), (BF, "e4m3"), (BF, "e2m1"), (FP, "e2m1")])
@pytest.mark.parametrize("hq,hkv,hd,dims", [(3, 2, 16, 16), (4, 4, 64, 32), (6, 2, 96, 48), (32, 4, 128, 128),
                                            (32, 4, 128, 16), (5, 1, 256, 208), (2, 2, 256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [10, 700])
def test_write_with_a_rope(dtype, rows, hq, hkv, hd, dims, interleaved, n):
    """q and k against the definition, v as it is, nothing else touched; few rows and many."""
    from mtp_block_draft_gb300 import DmtpRope
    how = SCALINGS[(hd + dims + n) // 2 % 4]
    theta, amplitude = 10000.0, 1.25
    B, ps, blocks = 3, 7, 110
    g = gen(hd + hq)
    c = new_cache(B, blocks, ps, hkv, hd, dtype, rows)
    r = np.random.RandomState(n)
    slots = r.permutation(B * blocks * ps)[:n]
    seq, pos = slots // (blocks * ps), slots % (blocks * ps)
    seq[1], seq[n - 2] = -1, -7
    qkv = randn((n, (hq + 2 * hkv) * hd + 4), g, dtype, 2.0)     # strided views, an odd pitch
    q = qkv[:, :hq * hd].view(n, hq, hd)
    k = qkv[:, hq * hd:(hq + hkv) * hd].view(n, hkv, hd)
    v = qkv[:, (hq + hkv) * hd:(hq + 2 * hkv) * hd].view(n, hkv, hd)
    before = [t.clone() for t in (c.k, c.v)]
    q_out = torch.full((n, hq, hd), 7.0, dtype=dtype, device="cuda")
    rope = DmtpRope(theta, dims=dims, interleaved=interleaved, amplitude=amplitude, **how)
    assert c.write(k, v, i32(seq), i32(pos), q=q, q_out=q_out, rope=rope) is q_out
    k_out = torch.full((n, hkv, hd), 7.0, dtype=dtype, device="cuda")
    v_out = k_out.clone()
    c.read(i32(seq), i32(pos), k_out, v_out)
    c.check()
    live = seq >= 0
    f = frequencies(dims, theta, **how)
    rq, rk, rv = (rotated(np64(q), pos, dims, interleaved, amplitude, f),
                  rotated(np64(k), pos, dims, interleaved, amplitude, f), np64(v))
    # fp32 sines within 2^-22 (two units) times the amplitude, two products, one sum
    mag = lambda x: 2.0 ** -20.5 * np.abs(x).max(-1, keepdims=True) * math.sqrt(2) * amplitude
    dq = np.abs(np64(q_out) - rq)
    assert (dq <= HALF[dtype] * np.abs(rq) + mag(np64(q)))[live].all()
    assert (np64(q_out)[~live] == 7).all() and (np64(k_out)[~live] == 7).all()
    assert np.array_equal(np64(q_out)[live][..., dims:], np64(q)[live][..., dims:])
    dk = np.abs(np64(k_out) - rk)
    if rows == "raw":
        assert np.array_equal(np64(v_out)[live], rv[live])
        assert (dk <= HALF[dtype] * np.abs(rk) + mag(np64(k)))[live].all()
    elif rows == "e4m3":
        # half a step: 2^-4 of the value, or 2^-10 scales (2^-9 near 0) of max|row| / 224 at most
        top = np.abs(rk).max(-1, keepdims=True)
        assert (dk <= 2.0 ** -4 * np.abs(rk) + 2.0 ** -10 * top / 224 + 2 * mag(np64(k)))[live].all()
    else:
        # half a step of E2M1 is 1 at most, 2 beyond 6 times the block's scale (which is off by
        # 2^-4 of itself, so that a block's largest is up to 6.4 of it); the scale is max / 5.647 at
        # most, and its own spacing 2^-10 max|row| / 1344
        block = np.abs(rk).reshape(*rk.shape[:-1], -1, 16).max(-1).repeat(16, -1)
        top = np.abs(rk).max(-1, keepdims=True)
        assert (dk <= block / 5.6 + 6 * 2.0 ** -10 * top / 1344 + HALF[dtype] * np.abs(rk) + 2 * mag(np64(k)))[live].all()
    # nothing else of the cache changed
    if rows != "e2m1":
        page = c.table.cpu().numpy()[seq[live], pos[live] // ps]
        touched = torch.zeros(c.k.shape[0], ps, dtype=torch.bool)
        touched[torch.from_numpy(page).long(), torch.from_numpy(pos[live] % ps).long()] = True
        for t, was in zip((c.k, c.v), before):
            a = t.view(torch.uint8).cpu().reshape(c.k.shape[0], hkv, ps, -1).permute(0, 2, 1, 3)
            z = was.view(torch.uint8).cpu().reshape(c.k.shape[0], hkv, ps, -1).permute(0, 2, 1, 3)
            assert torch.equal(a[~touched], z[~touched])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows", ROWS)
def test_a_plain_rope_is_the_write_s_own(dtype, rows):
    """Whole heads, half pairs, no scaling: what rope_theta does, but for the sums' contraction."""
    from mtp_block_draft_gb300 import DmtpRope
    g = gen(3)
    k, v, q = randn((40, 4, 128), g, dtype), randn((40, 4, 128), g, dtype), randn((40, 8, 128), g, dtype)
    seq, pos = i32([0] * 40), i32(np.arange(40) * 50)
    a, b = (new_cache(1, 32, 64, 4, 128, dtype, rows, poison=False) for _ in range(2))
    qa = a.write(k, v, seq, pos, q=q, rope_theta=10000.0)
    qb = b.write(k, v, seq, pos, q=q, rope=DmtpRope(10000.0))
    d = np.abs(np64(qa) - np64(qb))
    assert (d <= 2 * HALF[dtype] * np.abs(np64(qa)) + 2.0 ** -22 * 8).all()
    assert torch.equal(a.v, b.v)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pos", [1, 4095, 10 ** 6, 2 ** 30 + 12345])
def test_far_positions_keep_their_angles(pos, interleaved):
    from mtp_block_draft_gb300 import DmtpPagedCache, DmtpRope
    table = torch.zeros((1, 33000), dtype=torch.int32, device="cuda")
    c = DmtpPagedCache.alloc(1, 65000, 1, 128, table, dtype=FP)
    x = randn((1, 1, 128), gen(pos % 97), FP)
    how = dict(scaling="ramp", factor=32.0, orig_len=32768, low=1.0, high=32.0)
    q = c.write(x, x, i32([0]), i32([pos]), q=x, rope=DmtpRope(1e6, interleaved=interleaved, **how))
    c.check()
    ref = rotated(np64(x), [pos], 128, interleaved, 1.0, frequencies(128, 1e6, **how))
    # the frequencies are doubles, formed in about ten operations: pos 2^-50 radians more
    bound = (2.0 ** -20.5 + 2 * pos * 2.0 ** -50) * np.abs(np64(x)).max() * 2
    assert np.abs(np64(q) - ref).max() <= bound


def test_queries_rotated_in_place():
    from mtp_block_draft_gb300 import DmtpRope
    for dtype in (BF, FP):
        for n in (3, 900):
            c = new_cache(1, 20, 64, 2, 128, dtype)
            k, q = randn((n, 2, 128), gen(1), dtype), randn((n, 6, 128), gen(2), dtype)
            seq, pos, rope = i32([0] * n), i32(range(n)), DmtpRope(dims=96)
            want = c.write(k, k, seq, pos, q=q, rope=rope)
            assert c.write(k, k, seq, pos, q=q, q_out=q, rope=rope) is q and torch.equal(want, q)


# ---- rows in 4 bits -------------------------------------------------------------------

def e2m1_of(x):
    """What E2M1 rows of x (fp32) stand for, by the definition, the quotients in fp32."""
    x = x.astype(np.float32)
    fin = np.where(np.isfinite(x), np.abs(x), 0).astype(np.float32)
    m, e = np.frexp(fin.max(-1))
    e = np.where(m <= 0.65625, e - 12, e - 11)
    s = np.where(fin.max(-1) > 0, np.exp2(np.maximum(e, -126).astype(np.float64)), 1.0)
    y = (x.astype(np.float64) / s[..., None]).astype(np.float32).reshape(*x.shape[:-1], -1, 16)
    odd = ~np.isfinite(y).all(-1)
    b = (np.where(np.isfinite(y), np.abs(y), 0).max(-1) / np.float32(6)).astype(np.float64)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(b, 2.0 ** -30))) - 3, -9))
    b = np.rint(b / step) * step
    with np.errstate(all="ignore"):
        z = (y / b[..., None].astype(np.float32)).astype(np.float64)
        z = np.where(b[..., None] > 0, z, 0.0)
        a = np.minimum(np.abs(z), 6.0)
        st = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))) - 1, -1))
        a = np.rint(a / st) * st
    v = np.where(odd[..., None], np.nan, np.sign(z) * a * b[..., None])
    return v.reshape(x.shape) * s[..., None], s


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hkv,hd,ps", [(1, 16, 1), (3, 48, 5), (2, 64, 16), (4, 128, 64), (2, 240, 7), (5, 256, 3)])
def test_e2m1_rows_are_the_definition_s(dtype, hkv, hd, ps):
    """Values over many magnitudes, ties, zero rows and blocks, tiny and huge rows, NaN, infinities."""
    n = 300
    g = gen(hd)
    c = new_cache(2, -(-n // ps), ps, hkv, hd, dtype, "e2m1", extra=2)
    x = torch.randn((n, hkv, hd), device="cuda", generator=g)
    x *= torch.exp2(torch.randint(-12, 6, (n, hkv, hd // 16), device="cuda", generator=g).float()).repeat_interleave(16, -1)
    x[0] = 0
    x[1, :, :16] = 0
    x[2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * (hd // 8), device="cuda")  # ties
    x[3] *= 1e-38
    x[4] *= 2.0 ** 120
    x[5, 0, 0], x[6, :, hd - 1], x[7, 0, 3] = float("nan"), float("inf"), -float("inf")
    x[8] = float("nan")
    x = x.to(dtype)
    v = torch.flip(x, (0,))
    seq, pos = i32([1] * n), i32(np.random.RandomState(0).permutation(n))
    c.write(x, v, seq, pos)
    k_out, v_out = c.read(seq, pos)
    c.check()
    pg, off = c.table.cpu().numpy()[1, pos.cpu().numpy() // ps], pos.cpu().numpy() % ps
    for got, src, which, scale in ((k_out, x, "k", c.k_scale), (v_out, v, "v", c.v_scale)):
        want, s = e2m1_of(np64(src))
        assert np.array_equal(np64(scale)[pg, :, off], s)
        assert np.array_equal(pages64(c, which)[pg, :, off], want, equal_nan=True)
        # read: the value (six bits times a power of two from 2^-136 on: exact in fp32), rounded once
        # to the rows' type, whose spacing below 2^-126 is 2^-133 for bf16
        exact = torch.from_numpy(want.astype(np.float32)).to(dtype)
        assert np.array_equal(np64(got), np64(exact), equal_nan=True)


def test_every_e2m1_byte_and_block_scale():
    from mtp_block_draft_gb300 import DmtpPagedCache
    hd, ps = 16, 64
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    c = DmtpPagedCache.alloc(8, ps, 1, hd, table, dtype=FP, e2m1=True)
    r = np.random.RandomState(0)
    for t in (c.k, c.v):
        raw = r.randint(0, 256, t.shape).astype(np.uint8)
        raw[:, ps * hd // 2:] = np.arange(8 * ps).reshape(8, ps) % 256
        t.copy_(torch.from_numpy(raw))
    c.k_scale.copy_(torch.from_numpy(np.exp2(r.randint(-30, 30, (8, 1, ps)))))
    k, v = c.read(i32([0] * 512), i32(range(512)))
    for got, which in ((k, "k"), (v, "v")):
        want = pages64(c, which)[:, 0].reshape(512, 1, hd)
        assert np.array_equal(np64(got), want, equal_nan=True)


def test_e2m1_cache_s_rows_around_a_write_stay():
    c = new_cache(2, 6, 16, 3, 64, BF, "e2m1")
    g = gen(0)
    fill_cache(c, [96, 96], g)
    k0, v0 = pages64(c, "k"), pages64(c, "v")
    x = randn((3, 3, 64), g)
    c.write(x, x, i32([0, 1, -1]), i32([17, 95, 3]))
    k1, v1 = pages64(c, "k"), pages64(c, "v")
    t = c.table.cpu().numpy()
    same = np.ones(k0.shape[:1] + (16,), bool)
    same[t[0, 1], 1] = same[t[1, 5], 15] = False
    for a, b in ((k0, k1), (v0, v1)):
        a, b = np.moveaxis(a, 2, 1)[same], np.moveaxis(b, 2, 1)[same]
        assert np.array_equal(a, b, equal_nan=True)


def test_bad_indices_of_an_e2m1_cache_are_skipped_and_reported():
    from mtp_block_draft_gb300 import DmtpError
    c = new_cache(2, 2, 16, 2, 64, BF, "e2m1")
    c.table[1, 1] = 1000                       # no such page
    k = randn((4, 2, 64), gen(0))
    before = c.k.clone()
    for seq, pos, bit in ((2, 0, 32), (0, 32, 2), (0, -1, 2), (1, 16, 16)):
        c.write(k[:1], k[:1], i32([seq]), i32([pos]))
        with pytest.raises(DmtpError) as e:
            c.check()
        assert e.value.word == bit and torch.equal(before, c.k)
        o = torch.full((1, 2, 64), 3.0, dtype=BF, device="cuda")
        c.read(i32([seq]), i32([pos]), o, o.clone())
        with pytest.raises(DmtpError) as e:
            c.check()
        assert e.value.word == bit and (o == 3).all()


# ---- attention ------------------------------------------------------------------------

def reference(q, kv, spans, scale, hd, weights, cap=0.0, slopes=None, kbits=0.0):
    """Rows q [n, hq, hd]; spans: of each row (sequence, own position, lo, hi). (out, bound) in
    float64. weights: the rounding of a weight, 2^-16 (bf16 pairs), 2^-11 (fp16), 2^-8 (bf16) or
    2^-24.

    Bound. A score is a sum of hd fp32 products (and one scaling): off by at most (hd + 4) u
    sum|q k| scale; a cap's tanh by 4e-7 of it, a bias by three roundings of it and of the sum; a
    weight's relative error is twice e^(that) - 1 over (itself and the sum), plus 2^-21 for the
    base-2 exponential, its argument's rounding (|s| log2(e) 2^-24) and the factor that joins parts
    (the same again), plus its own rounding (2^-25 absolute below fp16's normal range); sums over
    n positions add n u. All relative to sum_j w_j |v_j|."""
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for r, (b, p, lo, hi) in enumerate(spans):
        if lo >= hi:
            continue
        k, v = kv[b]
        g = q.shape[1] // k.shape[0]
        far = np.abs(np.arange(lo, hi) - p)
        for h in range(q.shape[1]):
            kk, vv = k[h // g][lo:hi], v[h // g][lo:hi]
            s = kk @ q[r, h] * scale
            mag = np.max(np.abs(kk) @ np.abs(q[r, h])) * abs(scale)
            ds = (hd + 4) * U * mag + kbits * mag
            if cap:
                s = cap * np.tanh(s / cap)
                ds += 4e-7 * np.abs(s).max()
            if slopes is not None:
                s = s - slopes[h] * far
                ds += 4 * U * (abs(slopes[h]) * far).max()
                mag += (abs(slopes[h]) * far).max()
            w = np.exp(s - s.max())
            w /= w.sum()
            out[r, h] = w @ vv
            wv = w @ np.abs(vv)
            ew = 2 * math.expm1(2 * ds) + 2.0 ** -21 + 8 * mag * U + weights
            tol[r, h] = (ew + 2 * len(w) * U + kbits) * wv
            if weights == 2.0 ** -11:
                tol[r, h] += len(w) * 2.0 ** -25 * np.abs(vv).max(0) + 2.0 ** -25 * np.abs(vv).max()
    return out, tol


def close(out, ref, tol, dtype, where=None):
    got = np64(out)
    tol = tol * (1 + 2.0 ** -8) + HALF[dtype] * np.abs(ref) + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    if where is not None:
        bad &= where
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])


def slopes_of(hq):
    return torch.exp2(-8.0 * (torch.arange(hq, device="cuda", dtype=FP) + 1) / hq)


def check_attention(c, q, lens, kv, window=0, scale=None, cap=0.0, slopes=None, **kw):
    out = c.attention(q, i32(lens), window=window, scale=scale, cap=cap, slopes=slopes, **kw)
    c.check()
    sc = c.head_dim ** -0.5 if scale is None else float(np.float32(scale))
    R = q.shape[1]
    spans = [(b, n - R + i, max(0, n - R + i - window + 1) if window else 0, n - R + i + 1)
             for b, n in enumerate(lens) for i in range(R)]
    w = 2.0 ** -16 if c.k_scale is None or c.dtype is FP else 2.0 ** -11
    ref, tol = reference(np64(q).reshape(-1, *q.shape[2:]), kv, spans, sc, c.head_dim, w, cap,
                         None if slopes is None else np64(slopes))
    close(out, ref.reshape(q.shape), tol.reshape(q.shape), c.dtype)
    return out


SHAPES = [(16, 16, 64, 1, 16), (32, 4, 128, 1, 64), (32, 4, 128, 8, 16), (8, 1, 64, 3, 5), (5, 5, 64, 8, 128),
          (4, 4, 32, 8, 16), (12, 4, 96, 2, 32), (8, 2, 256, 1, 64), (48, 1, 128, 8, 48), (6, 2, 128, 5, 1),
          (3, 1, 16, 4, 16), (20, 2, 128, 4, 64), (16, 1, 64, 8, 33), (4, 2, 240, 2, 16), (16, 4, 128, 4, 7)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hq,hkv,hd,rows,ps", SHAPES)
def test_attention_over_e2m1_rows(hq, hkv, hd, rows, ps, dtype):
    lens = [0, 1, rows, 63, 64, 65, 200, 517]
    g = gen(hq * 1000 + hd + rows)
    c = new_cache(len(lens), -(-517 // ps), ps, hkv, hd, dtype, "e2m1")
    kv = fill_cache(c, lens, g)
    q = randn((len(lens), rows, hq, hd), g, dtype, 1.5)
    a = check_attention(c, q, lens, kv)
    assert torch.equal(a, c.attention(q, i32(lens)))  # the same call, the same bits


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("hq", [1, 8, 24, 64])
def test_attention_over_long_e2m1_caches(hq, hd):
    """Split units, every width of the tensor-core kernel."""
    lens = [5000, 17, 3333]
    c = new_cache(3, 160, 32, 1, hd, BF, "e2m1")
    g = gen(hq)
    kv = fill_cache(c, lens, g)
    check_attention(c, randn((3, 1, hq, hd), g, BF, 1.5), lens, kv)


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("cap,bias", [(5.0, False), (0.0, True), (30.0, True), (1e30, False), (0.25, False)])
@pytest.mark.parametrize("hq,hkv,hd,R,ps", [(16, 16, 64, 1, 16), (32, 4, 128, 3, 64), (12, 4, 96, 2, 32),
                                            (8, 2, 256, 1, 5), (16, 1, 128, 8, 16), (4, 4, 32, 8, 33)])
def test_attention_with_capped_and_biased_scores(dtype, rows, cap, bias, hq, hkv, hd, R, ps):
    lens = [0, 1, R, 64, 333]
    g = gen(hq + hd)
    c = new_cache(len(lens), -(-333 // ps), ps, hkv, hd, dtype, rows)
    kv = fill_cache(c, lens, g)
    q = randn((len(lens), R, hq, hd), g, dtype, 3.0)
    check_attention(c, q, lens, kv, cap=cap, slopes=slopes_of(hq) if bias else None)


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("window", [1, 7, 64, 100])
def test_attention_window_with_a_bias(dtype, rows, window):
    lens = [0, 1, 5, 64, 130, 400]
    c = new_cache(len(lens), 25, 16, 2, 64, dtype, rows)
    g = gen(window)
    kv = fill_cache(c, lens, g)
    check_attention(c, randn((len(lens), 5, 8, 64), g, dtype), lens, kv, window=window, slopes=slopes_of(8), cap=20.0)


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_scores_as_they_are_are_the_plain_call_s(dtype, rows):
    c = new_cache(2, 20, 16, 2, 128, dtype, rows)
    g = gen(1)
    fill_cache(c, [300, 20], g)
    q = randn((2, 2, 8, 128), g, dtype)
    a = c.attention(q, i32([300, 20]))
    zero = torch.zeros(8, device="cuda")
    b = c.attention(q, i32([300, 20]), slopes=zero)
    assert np.abs(np64(a) - np64(b)).max() <= 2 * HALF[dtype] * np.abs(np64(a)).max() + 2.0 ** -20


# ---- attention of many rows -----------------------------------------------------------

def tensor_cores(c):
    return c.dtype is BF and c.head_dim <= 128


def check_prompt(c, q, start, lens, kv, window=0, scale=None, cap=0.0, slopes=None, first=None, end=None, **kw):
    out = torch.full_like(q, 7.0)
    got = c.prompt_attention(q, i32(start), i32(lens), window=window, scale=scale, cap=cap, slopes=slopes,
                             first=None if first is None else i32(first), end=None if end is None else i32(end),
                             out=out, **kw)
    c.check()
    assert got is out
    sc = c.head_dim ** -0.5 if scale is None else float(np.float32(scale))
    spans, live = [(0, 0, 0, 0)] * q.shape[0], np.zeros(q.shape[0], bool)
    for b, n in enumerate(lens):
        count = start[b + 1] - start[b]
        for i in range(count):
            r, p = start[b] + i, n - count + i
            lo = 0 if first is None else max(0, int(first[r]))
            if window:
                lo = max(lo, p - window + 1)
            spans[r] = (b, p, lo, min(p + 1 if end is None else int(end[r]), n))
            live[r] = True
    ref, tol = reference(np64(q), kv, spans, sc, c.head_dim, 2.0 ** -8 if tensor_cores(c) else 2.0 ** -24, cap,
                         None if slopes is None else np64(slopes))
    close(out, ref, tol, c.dtype, live[:, None, None])
    assert (np64(out)[~live] == 7).all()
    return out


def starts(rows, lead=0):
    return [lead] + list(lead + np.cumsum(rows))


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("hq,hkv,hd,ps", [(16, 16, 64, 16), (32, 4, 128, 64), (8, 1, 64, 5), (4, 4, 32, 16),
                                          (12, 4, 96, 32), (8, 2, 256, 64), (5, 1, 128, 1), (3, 1, 16, 16),
                                          (6, 3, 80, 33), (2, 1, 144, 7)])
def test_prompt_attention(hq, hkv, hd, ps, dtype, rows):
    """Sequences with no row, one, a few, more than a tile's; whole prompts and chunks; rows of none
    before and behind them."""
    count = [0, 1, 3, 37, 0, 70, 130, 1]
    lens = [9, 1, 200, 37, 0, 65 + 70, 130, 300]
    g = gen(hq * 1000 + hd)
    c = new_cache(len(lens), -(-300 // ps), ps, hkv, hd, dtype, rows)
    kv = fill_cache(c, lens, g)
    st = starts(count, 2)
    q = randn((st[-1] + 3, hq, hd), g, dtype, 1.5)
    a = check_prompt(c, q, st, lens, kv)
    b = torch.full_like(q, 7.0)
    c.prompt_attention(q, i32(st), i32(lens), out=b)
    assert torch.equal(a, b)  # the same call, the same bits


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("mask", ["docs", "prefix", "both", "window", "docs+window", "all"])
@pytest.mark.parametrize("hd", [64, 128, 192])
def test_prompt_masks(dtype, rows, mask, hd):
    count, lens = [100, 260, 33], [100, 300, 400]
    g = gen(7)
    c = new_cache(3, 25, 16, 2, hd, dtype, rows)
    kv = fill_cache(c, lens, g)
    st = starts(count)
    q = randn((st[-1], 4, hd), g, dtype)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, count)])
    own = np.repeat(np.arange(3), count)
    kw = {}
    if "docs" in mask or mask == "both":
        cuts = [0, 1, 2, 65, 66, 128, 250, 399]
        kw["first"] = np.array([max(x for x in cuts if x <= p) for p in pos])
    if mask in ("prefix", "both"):
        kw["end"] = np.maximum(pos + 1, np.array([50, 290, 10])[own])
    if mask == "both":
        kw["end"] = np.maximum(pos + 1, kw["first"] + 20)
    if mask == "all":  # every row sees all of its sequence, and past it
        kw["end"] = np.full(len(pos), 10 ** 6)
    if "window" in mask:
        kw["window"] = 48
    check_prompt(c, q, st, lens, kv, **kw)


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("cap,bias", [(5.0, False), (0.0, True), (30.0, True)])
@pytest.mark.parametrize("hq,hkv,hd", [(8, 2, 64), (16, 2, 128), (4, 4, 96), (2, 1, 256)])
def test_prompt_scores(dtype, rows, cap, bias, hq, hkv, hd):
    count, lens = [150, 20], [150, 300]
    g = gen(hd)
    c = new_cache(2, 19, 16, hkv, hd, dtype, rows)
    kv = fill_cache(c, lens, g)
    st = starts(count)
    q = randn((st[-1], hq, hd), g, dtype, 3.0)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, count)])
    check_prompt(c, q, st, lens, kv, cap=cap, slopes=slopes_of(hq) if bias else None, end=np.maximum(pos + 1, 60))


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_prompt_rows_that_see_nothing(dtype, rows):
    """More rows than positions, intervals that are empty or past the length, no length at all."""
    c = new_cache(4, 10, 16, 2, 64, dtype, rows)
    g = gen(0)
    lens = [10, 0, 70, 40]
    kv = fill_cache(c, lens, g)
    st = starts([30, 5, 70, 40])
    q = randn((st[-1], 4, 64), g, dtype)
    check_prompt(c, q, st, lens, kv)
    first = np.random.RandomState(0).randint(-5, 90, st[-1])
    end = np.random.RandomState(1).randint(-5, 90, st[-1])
    first[3], end[4], first[5], end[6] = 2 ** 31 - 1, -2 ** 31, -2 ** 31, 2 ** 31 - 1
    check_prompt(c, q, st, lens, kv, first=first, end=end)
    out = c.prompt_attention(q, i32(st), i32([-5, 0, 0, -2 ** 31]))
    c.check()
    assert (out == 0).all()


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_prompt_over_a_long_cache(dtype, rows):
    """Few rows, many positions: keys are split and joined."""
    c = new_cache(2, 200, 32, 2, 128, dtype, rows)
    g = gen(4)
    lens = [6400, 3001]
    kv = fill_cache(c, lens, g)
    st = starts([5, 1])
    q = randn((st[-1], 8, 128), g, dtype)
    check_prompt(c, q, st, lens, kv)
    check_prompt(c, q, st, lens, kv, slopes=slopes_of(8), window=3000)


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_reaches_the_rows_that_see_it(dtype, rows, value):
    c = new_cache(2, 20, 16, 2, 64, dtype, rows)
    g = gen(0)
    lens = [300, 50]
    fill_cache(c, lens, g)
    x, z = randn((3, 2, 64), g, dtype), randn((3, 2, 64), g, dtype)
    z[:, :, 5] = value
    at = [100, 290, 17]
    clean = stored(c, lens)
    q = randn((350, 4, 64), g, dtype)
    plain = c.prompt_attention(q, i32([0, 300, 350]), i32(lens))
    for bad_k in (False, True):
        c.write(z if bad_k else x, x if bad_k else z, i32([0, 0, 1]), i32(at))
        first = np.zeros(350, int)
        first[200:300] = 150                # a document that begins behind the first bad position
        got = c.prompt_attention(q, i32([0, 300, 350]), i32(lens), first=i32(first))
        c.check()
        sees = np.zeros(350, bool)
        sees[100:200] = sees[290:300] = sees[317:350] = True
        odd = ~np.isfinite(np64(got)).all((1, 2))
        assert not odd[~sees].any()
        if not bad_k:                       # (an infinite key's score may be minus infinity)
            assert odd[sees].all()
        same = ~sees
        same[150:300] = False               # (those rows see fewer positions than in the plain call)
        d = np.abs(np64(got) - np64(plain))[same]
        assert (d <= 2 * HALF[dtype] * np.abs(np64(plain))[same] + 2.0 ** -10 * 8).all()
        fill = clean[0][0], clean[0][1]
        assert np.isfinite(fill[0]).all() and np.isfinite(fill[1]).all()


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_prompt_pages_that_no_row_sees_are_not_looked_up(dtype, rows):
    from mtp_block_draft_gb300 import DmtpError
    ps = 16
    c = new_cache(2, 40, ps, 2, 64, dtype, rows)
    g = gen(0)
    lens = [600, 333]
    kv = fill_cache(c, lens, g)
    st = starts([64, 10])
    q = randn((st[-1], 4, 64), g, dtype)
    table = c.table.cpu()
    for b, (n, r) in enumerate(zip(lens, (64, 10))):
        table[b, :(n - r - 99) // ps] = -1
        table[b, -(-n // ps):] = 10 ** 6
    c.table.copy_(table)
    check_prompt(c, q, st, lens, kv, window=100)
    # a bad page that is seen: reported, its positions left out
    c.table[0, 590 // ps] = -3
    out = c.prompt_attention(q, i32(st), i32(lens), window=100)
    with pytest.raises(DmtpError) as e:
        c.check()
    assert e.value.word == 16 and np.isfinite(np64(out)).all()


def test_prompt_row_starts_that_do_not_fit_are_reported():
    from mtp_block_draft_gb300 import DmtpError
    c = new_cache(3, 4, 16, 2, 64, BF)
    g = gen(0)
    fill_cache(c, [64, 64, 64], g)
    q = randn((40, 4, 64), g)
    for start in ([0, 10, 5, 40], [-3, 10, 20, 40], [0, 10, 20, 41], [0, 10 ** 9, 10 ** 9, 10 ** 9]):
        out = torch.full_like(q, 7.0)
        c.prompt_attention(q, i32(start), i32([64] * 3), out=out)
        with pytest.raises(DmtpError) as e:
            c.check()
        assert e.value.word == 64 and np.isfinite(np64(out)).all()
    c.prompt_attention(q, i32([0, 10, 20, 40]), i32([64, 65, 64]))
    with pytest.raises(DmtpError) as e:
        c.check()
    assert e.value.word == 2


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_prompt_strides_scale_and_workspace(dtype, rows):
    c = new_cache(1, 200, 16, 2, 64, dtype, rows)
    g = gen(0)
    kv = fill_cache(c, [3000], g)
    big = randn((9, 13, 3 * 64), g, dtype)
    q = big[1:8, 2:6, 64:128]
    out = torch.full((7, 4, 128), 7.0, dtype=dtype, device="cuda")
    n = c.prompt_workspace(7, 4)
    ws = torch.full((max(n, 1),), 0xff, dtype=torch.uint8, device="cuda")
    for scale in (0.02, -0.1, 0.0):
        a = c.prompt_attention(q, i32([0, 7]), i32([3000]), scale=scale, out=out[:, :, :64], workspace=ws)
        spans = [(0, 2993 + i, 0, 2994 + i) for i in range(7)]
        ref, tol = reference(np64(q), kv, spans, float(np.float32(scale)), 64, 2.0 ** -8 if tensor_cores(c) else 2.0 ** -24)
        close(a, ref, tol, dtype)
        assert (out[:, :, 64:] == 7).all()


def test_prompt_graph_replay_streams_and_empty_calls():
    """A captured call follows its inputs; calls on two streams at once have workspaces of their own."""
    c = new_cache(2, 100, 16, 2, 128, BF, "e2m1")
    g = gen(0)
    fill_cache(c, [1600, 1000], g)
    q, st, ln = randn((20, 8, 128), g), i32([0, 12, 20]), i32([1500, 900])
    out = torch.empty_like(q)
    n = c.prompt_workspace(20, 8)
    ws = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = c.prompt_attention(q, st, ln)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.prompt_attention(q, st, ln, out=out, workspace=ws[0])
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        c.prompt_attention(q, st, ln, out=out, workspace=ws[0])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    ln.copy_(i32([1600, 20]))
    st.copy_(i32([0, 3, 19]))
    out.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    fresh = torch.full_like(q, 7)
    c.prompt_attention(q, st, ln, out=fresh)
    assert torch.equal(out, fresh) and (out[19] == 7).all()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.full_like(q, 7) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                c.prompt_attention(q, st, ln, out=outs[i], workspace=ws[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fresh) and torch.equal(outs[1], fresh)
    assert c.prompt_attention(q[:0], i32([0, 0, 0]), ln).shape == (0, 8, 128)
    c.check()


def test_a_prompt_then_decode_steps():
    """The operators together: a prompt written in chunks with a rope into a 4-bit cache, its
    attention, then decode steps; each against float64 over what the cache holds."""
    from mtp_block_draft_gb300 import DmtpRope
    hq, hkv, hd = 8, 2, 128
    c = new_cache(2, 12, 32, hkv, hd, BF, "e2m1")
    g = gen(9)
    rope = DmtpRope(1e6, dims=64, interleaved=True, scaling="turns", factor=4.0, orig_len=256, high=4.0)
    slopes, cap = slopes_of(hq), 20.0
    at = [0, 0]
    for chunk in ([100, 33], [7, 200], [1, 1], [1, 0], [1, 1], [60, 1]):
        n = sum(chunk)
        seq = np.repeat([0, 1], chunk)
        pos = np.concatenate([np.arange(at[b], at[b] + chunk[b]) for b in range(2)])
        q = c.write(randn((n, hkv, hd), g), randn((n, hkv, hd), g), i32(seq), i32(pos),
                    q=randn((n, hq, hd), g), rope=rope)
        at = [a + m for a, m in zip(at, chunk)]
        kv = stored(c, at)
        out = check_prompt(c, q, starts(chunk), at, kv, cap=cap, slopes=slopes)
        if chunk == [1, 1]:  # the decode form of the same step
            one = check_attention(c, q.view(2, 1, hq, hd), at, kv, cap=cap, slopes=slopes)
            # both are within their bounds: 2^-8 of the weights of one, 2^-11 of the other's
            assert np.abs(np64(one)[:, 0] - np64(out)).max() <= 2.0 ** -6 * 4


# ---- what the larger pieces of the kernels could get wrong ------------------------------

@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("ps", [8, 64, 128, 256])
@pytest.mark.parametrize("window", [3, 10, 129, 700])
def test_prompt_windows_inside_pages(dtype, rows, ps, window):
    """Intervals that begin and end inside a page, pages that no row sees not named at all."""
    count, lens = [1, 40, 100], [777, 1000, 100]
    g = gen(ps + window)
    c = new_cache(3, -(-1024 // ps), ps, 1, 128, dtype, rows)
    kv = fill_cache(c, lens, g)
    table = c.table.cpu()
    for b, (n, r) in enumerate(zip(lens, count)):
        table[b, :max(0, n - r - window + 1) // ps] = -1
        table[b, -(-n // ps):] = 10 ** 6
    c.table.copy_(table)
    st = starts(count)
    q = randn((st[-1], 6, 128), g, dtype)
    check_prompt(c, q, st, lens, kv, window=window)
    check_prompt(c, q, st, lens, kv, window=window, slopes=slopes_of(6), cap=15.0)


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("hd,ps", [(128, 128), (64, 32), (128, 24)])
def test_prompt_of_several_tiles(dtype, rows, hd, ps):
    """A prompt over several tiles and blocks of keys, scores of every kind."""
    n = 700
    g = gen(hd + ps)
    c = new_cache(2, -(-900 // ps), ps, 1, hd, dtype, rows)
    lens = [n, 900]
    kv = fill_cache(c, lens, g)
    st = starts([n, 130])
    q = randn((st[-1], 3, hd), g, dtype, 2.0)
    for kw in (dict(), dict(cap=8.0), dict(slopes=slopes_of(3)), dict(cap=60.0), dict(scale=-0.05, cap=3.0, slopes=-slopes_of(3))):
        check_prompt(c, q, st, lens, kv, **kw)


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_prompt_with_a_bias_that_leaves_only_near_positions(dtype, rows):
    c = new_cache(1, 30, 32, 2, 64, dtype, rows)
    g = gen(2)
    kv = fill_cache(c, [900], g)
    q = randn((900, 2, 64), g, dtype)
    for slopes in ([50.0, 0.0], [1000.0, -0.5], [0.01, 3.0]):
        check_prompt(c, q, [0, 900], [900], kv, slopes=torch.tensor(slopes, device="cuda"))


@pytest.mark.parametrize("dtype,rows", [(d, r) for d in (BF, FP) for r in ("e4m3", "e2m1")])
def test_scales_that_are_no_powers_of_two(dtype, rows):
    """Prompts on the tensor cores take such rows rounded to bf16."""
    c = new_cache(2, 10, 32, 2, 128, dtype, rows)
    g = gen(1)
    fill_cache(c, [300, 300], g)
    for s in (c.k_scale, c.v_scale):
        s.mul_(0.5 + torch.rand(s.shape, device="cuda", generator=g))
    kv = stored(c, [300, 300])
    q = randn((310, 4, 128), g, dtype)
    out = c.prompt_attention(q, i32([0, 300, 310]), i32([300, 300]))
    spans = [(0, i, 0, i + 1) for i in range(300)] + [(1, 290 + i, 0, 291 + i) for i in range(10)]
    tc = tensor_cores(c)
    ref, tol = reference(np64(q), kv, spans, 128 ** -0.5, 128, 2.0 ** -8 if tc else 2.0 ** -24, kbits=2.0 ** -8 if tc else 0.0)
    close(out, ref, tol, dtype)
    check_attention(c, randn((2, 3, 4, 128), g, dtype), [300, 300], kv)


@pytest.mark.parametrize("dtype,rows", KINDS)
def test_few_rows_over_a_long_cache_with_values_that_are_not_finite(dtype, rows):
    """Split keys: the range with such a value is computed row by row, the rest as ever."""
    c = new_cache(1, 100, 64, 1, 128, dtype, rows)
    g = gen(5)
    fill_cache(c, [6000], g)
    q = randn((6, 4, 128), g, dtype)
    want = c.prompt_attention(q, i32([0, 6]), i32([6000]), first=i32([3100] * 6))
    bad = torch.full((1, 1, 128), float("nan"), dtype=dtype, device="cuda")
    c.write(bad, bad, i32([0]), i32([3090]))        # in the first block of keys, seen by none
    got = c.prompt_attention(q, i32([0, 6]), i32([6000]), first=i32([3100] * 6))
    c.check()
    d = np.abs(np64(got) - np64(want))
    assert (d <= 2 * HALF[dtype] * np.abs(np64(want)) + 2.0 ** -8 * 0.5).all()
    assert np.isnan(np64(c.prompt_attention(q, i32([0, 6]), i32([6000])))).all()


@pytest.mark.parametrize("dtype,rows", KINDS)
@pytest.mark.parametrize("cap,bias", [(0.0, False), (10.0, True)])
def test_decode_rows_that_do_not_see_what_is_not_finite(dtype, rows, cap, bias):
    c = new_cache(2, 20, 16, 2, 64, dtype, rows)
    g = gen(0)
    lens = [300, 100]
    fill_cache(c, lens, g)
    q = randn((2, 8, 4, 64), g, dtype)
    sl = slopes_of(4) if bias else None
    want = np64(c.attention(q, i32(lens), cap=cap, slopes=sl, window=50))
    z = torch.full((3, 2, 64), float("nan"), dtype=dtype, device="cuda")
    c.write(z, z, i32([0, 0, 1]), i32([296, 200, 97]))      # seen by rows 4.., by none, by rows 5..
    got = np64(c.attention(q, i32(lens), cap=cap, slopes=sl, window=50))
    c.check()
    assert np.isnan(got[0, 4:]).all() and np.isnan(got[1, 5:]).all()
    for b, n in ((0, 4), (1, 5)):
        d = np.abs(got[b, :n] - want[b, :n])
        assert (d <= 2 * HALF[dtype] * np.abs(want[b, :n]) + 2.0 ** -10 * 4).all()
