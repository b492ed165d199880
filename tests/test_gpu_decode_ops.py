"""The decode-step operators of include/dmtp_ops.h on the GPU, against plain float64 forms.

Tolerances are derived, not fitted. A rounding to a type is off by at most half a step
(finfo(t).eps / 2 of the value: fp32 2^-24, bf16 2^-8, E4M3 2^-4 or half the subnormal
spacing 2^-9), and the arithmetic before it is counted operation by operation where each
bound is formed.
"""
import math

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

BF, FP, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -24}
U = 2.0 ** -24


def np64(t):
    return t.float().cpu().numpy().astype(np.float64)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=BF, mul=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * mul).to(dtype)


def new_cache(B, blocks, ps, hkv, hd, dtype=BF, e4m3=False, seed=0, extra=3, fill=None):
    """A cache whose sequences own shuffled pages; fill: a value put into every slot."""
    from mtp_block_draft_gb300 import DmtpPagedCache
    n = B * blocks + extra
    perm = np.random.RandomState(seed).permutation(n)[:B * blocks].astype(np.int32)
    table = torch.from_numpy(perm.reshape(B, blocks)).cuda()
    c = DmtpPagedCache.alloc(n, ps, hkv, hd, table, dtype=dtype, e4m3=e4m3)
    if fill is not None:
        if e4m3:
            c.k.view(torch.uint8).fill_(0x7f)
            c.v.view(torch.uint8).fill_(0x7f)
            c.k_scale.fill_(fill)
            c.v_scale.fill_(fill)
        else:
            c.k.fill_(fill)
            c.v.fill_(fill)
    return c


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def fill_cache(c, lens, g, kmul=1.0):
    """Writes random rows at positions 0..len-1 of every sequence; returns what is stored, as
    float64 [hkv, len, hd] per sequence."""
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [[]]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens] + [[]]).astype(np.int32)
    n = len(seq)
    if n:
        spread = 0.25 + 2 * torch.rand((n, c.n_kv_heads, 1), device="cuda", generator=g)
        k = (torch.randn((n, c.n_kv_heads, c.head_dim), device="cuda", generator=g) * spread * kmul)
        v = torch.randn((n, c.n_kv_heads, c.head_dim), device="cuda", generator=g) * spread
        c.write(k.to(c.dtype), v.to(c.dtype), i32(seq), i32(pos))
    return stored(c, lens)


def stored(c, lens):
    table, ps = c.table.cpu().numpy(), c.c.page_size
    kd, vd = np64(c.k), np64(c.v)
    if c.k_scale is not None:
        kd, vd = kd * np64(c.k_scale)[..., None], vd * np64(c.v_scale)[..., None]
    out = []
    for b, n in enumerate(lens):
        pg = table[b][:-(-n // ps)] if n else table[b][:0]
        out.append([np.moveaxis(x[pg], 1, 0).reshape(c.n_kv_heads, -1, c.head_dim)[:, :max(n, 0)]
                    for x in (kd, vd)])
    return out


def reference(q, kv, lens, rows, window, scale, pair):
    """(out, bound) in float64. pair: weights carry 16 bits (bf16 pairs) or are fp32; else 11
    bits (fp16).

    Bound. A score is a sum of hd fp32 products (and one scaling): off by at most
    (hd + 4) u sum|q k| scale; a weight's relative error is twice e^(that) - 1 over (itself and
    the sum), plus 2^-21 for the base-2 exponential, its argument's rounding
    (|s| log2(e) 2^-24) and the factor that joins parts (the same again), plus its own
    rounding (2^-16 as a pair, 2^-11 as fp16, and 2^-25 absolute below fp16's normal range);
    sums over n positions add n u. All relative to sum_j w_j |v_j|."""
    B, R, hq, hd = q.shape
    g = hq // kv[0][0].shape[0]
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        k, v = kv[b]
        for i in range(R):
            p = lens[b] - R + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0 or lo > p:
                continue
            for h in range(hq):
                kk, vv = k[h // g][lo:p + 1], v[h // g][lo:p + 1]
                s = kk @ q[b, i, h] * scale
                mag = np.max(np.abs(kk) @ np.abs(q[b, i, h])) * abs(scale)
                w = np.exp(s - s.max())
                w /= w.sum()
                out[b, i, h] = w @ vv
                wv = w @ np.abs(vv)
                ds = (hd + 4) * U * mag
                ew = 2 * math.expm1(2 * ds) + 2.0 ** -21 + 8 * mag * U + (2.0 ** -16 if pair else 2.0 ** -11)
                tol[b, i, h] = (ew + 2 * len(w) * U) * wv
                if not pair:
                    tol[b, i, h] += len(w) * 2.0 ** -25 * np.abs(vv).max(0) + 2.0 ** -25 * np.abs(vv).max()
    return out, tol


def check_attention(c, q, lens, kv, window=0, scale=None, **kw):
    out = c.attention(q, i32(lens), window=window, scale=scale, **kw)
    c.check()
    sc = c.head_dim ** -0.5 if scale is None else float(np.float32(scale))
    ref, tol = reference(np64(q), kv, lens, q.shape[1], window, sc, pair=c.k_scale is None or c.dtype is FP)
    got = np64(out)
    tol = tol * (1 + 2 ** -8) + HALF[c.dtype] * np.abs(ref) + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
    return out


# ---- write and read -------------------------------------------------------------------

def rotated(x, pos, theta):
    half = x.shape[-1] // 2
    if not theta:
        return x
    # extended precision: a float64 angle at position 2^30 has lost 2^-23 of a radian
    f = np.float128(float(np.float32(theta))) ** (-np.arange(half, dtype=np.float128) / half)
    a = (np.asarray(pos, np.float128)[:, None] * f)[:, None]
    c, s = np.cos(a).astype(np.float64), np.sin(a).astype(np.float64)
    return np.concatenate((x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s), -1)


@pytest.mark.parametrize("hq,hkv,hd", [(4, 4, 32), (5, 1, 64), (6, 2, 96), (32, 4, 128), (2, 2, 256), (3, 3, 16)])
@pytest.mark.parametrize("dtype,e4m3", [(BF, False), (BF, True), (FP, False), (FP, True)])
@pytest.mark.parametrize("theta", [0.0, 10000.0])
def test_write_then_read(hq, hkv, hd, dtype, e4m3, theta):
    B, blocks, ps = 3, 5, 7
    g = gen(hd + hq)
    c = new_cache(B, blocks, ps, hkv, hd, dtype, e4m3, fill=float("nan"))
    seq = [2, 0, 0, 2, 1, -1, 0, 2, 1, -5]
    pos = [34, 0, 6, 33, 7, 3, 13, 1, 28, 99999]
    n = len(seq)
    qkv = randn((n, (hq + 2 * hkv) * hd + 4), g, dtype, 2.0)     # strided views, an odd pitch
    q = qkv[:, :hq * hd].view(n, hq, hd)
    k = qkv[:, hq * hd:(hq + hkv) * hd].view(n, hkv, hd)
    v = qkv[:, (hq + hkv) * hd:(hq + 2 * hkv) * hd].view(n, hkv, hd)
    before = c.k.clone()
    q_out = torch.full((n, hq, hd), 7.0, dtype=dtype, device="cuda")
    assert c.write(k, v, i32(seq), i32(pos), q=q, q_out=q_out, rope_theta=theta) is q_out
    k_out = torch.full((n, hkv, hd), 7.0, dtype=dtype, device="cuda")
    v_out = k_out.clone()
    c.read(i32(seq), i32(pos), k_out, v_out)
    c.check()
    live = np.array(seq) >= 0
    p = np.where(live, pos, 0)
    rq, rk, rv = rotated(np64(q), p, theta), rotated(np64(k), p, theta), np64(v)
    # rotation: fp32 sines within 2^-22 (two units), two products, one sum: 2^-21 of |a| + |b|
    mag = lambda x: 2.0 ** -21 * np.linalg.norm(x, axis=-1, keepdims=True) if theta else 0.0
    dq = np.abs(np64(q_out) - rq)
    assert (dq <= HALF[dtype] * np.abs(rq) + mag(rq))[live].all()
    assert (np64(q_out)[~live] == 7).all() and (np64(k_out)[~live] == 7).all()
    if e4m3:
        # v is not rotated: exactly the oracle's row quantisation
        want = np.stack([np.stack([np.multiply(*fp8.quantize_rows(r[None])).reshape(-1) for r in x]) for x in rv])
        assert (np64(v_out) == want)[live].all()
        sc = np.stack([np.array([fp8.pow2_scale(np.abs(r).max()) for r in x]) for x in rk])[..., None]
        # (a maximum within the rotation's error of 448 s may take the other scale)
        dk = np.abs(np64(k_out) - rk)
        assert (dk <= 2.0 ** -4 * np.abs(rk) + 2.0 ** -9 * sc + 2 * mag(rk))[live].all()
        assert (np.log2(np64(c.k_scale)[np64(c.k_scale) > 0]) % 1 == 0).all()
    else:
        assert (np64(v_out) == rv)[live].all()
        assert (np.abs(np64(k_out) - rk) <= HALF[dtype] * np.abs(rk) + mag(rk))[live].all()
    # nothing else of the cache changed
    page = c.table.cpu().numpy()[np.array(seq)[live], np.array(pos)[live] // ps]
    touched = torch.zeros(c.k.shape[0], ps, dtype=torch.bool)
    touched[torch.from_numpy(page).long(), torch.from_numpy(np.array(pos)[live] % ps).long()] = True
    a = c.k.view(torch.uint8).cpu().reshape(c.k.shape[0], hkv, ps, -1).permute(0, 2, 1, 3)
    z = before.view(torch.uint8).cpu().reshape(c.k.shape[0], hkv, ps, -1).permute(0, 2, 1, 3)
    assert torch.equal(a[~touched], z[~touched])


@pytest.mark.parametrize("pos", [0, 1, 4095, 10 ** 6, 2 ** 30 + 12345])
def test_far_positions_keep_their_angles(pos):
    hd = 128
    table = torch.zeros((1, 33000), dtype=torch.int32, device="cuda")
    from mtp_block_draft_gb300 import DmtpPagedCache
    c = DmtpPagedCache.alloc(1, 65000, 1, hd, table, dtype=FP)
    x = randn((1, 1, hd), gen(pos % 97), FP)
    q = c.write(x, x, i32([0]), i32([pos]), q=x, rope_theta=10000.0)
    c.check()
    ref = rotated(np64(x), [pos], 10000.0)
    # the frequencies are doubles: pos 2^-53 radians more
    bound = (2.0 ** -21 + 2 * pos * 2.0 ** -53) * np.abs(np64(x)).max() * 2
    assert np.abs(np64(q) - ref).max() <= bound


def test_write_special_values_and_in_place_queries():
    """NaN and infinities become the E4M3 NaN and leave the row's scale to its finite values;
    zero rows take scale 1; tiny rows stop at the smallest normal scale; q rotated in place."""
    c = new_cache(1, 1, 8, 1, 32, FP, True)
    v = torch.zeros((5, 1, 32), device="cuda")
    v[0, 0, 3] = float("nan")
    v[0, 0, 4] = 3.0
    v[1, 0, 0] = float("-inf")
    v[1, 0, 1] = 448.0
    v[3, 0, 0] = 1e-42
    v[4, 0, 0] = 3.0e38
    q = randn((5, 2, 32), gen(1), FP)
    want = rotated(np64(q), np.arange(5), 100.0)
    got = c.write(v, v, i32([0] * 5), i32(range(5)), q=q, q_out=q, rope_theta=100.0)
    c.write(v, v, i32([0] * 5), i32(range(5)))
    assert got is q and np.abs(np64(q) - want).max() <= 2.0 ** -20 * 8
    _, r = c.read(i32([0] * 5), i32(range(5)))
    r, s = np64(r)[:, 0], np64(c.v_scale)[int(c.table[0, 0]), 0, :5]
    assert np.isnan(r[0, 3]) and r[0, 4] == 3.0 and s[0] == 2.0 ** -7
    assert np.isnan(r[1, 0]) and r[1, 1] == 448.0 and s[1] == 1.0
    assert (r[2] == 0).all() and s[2] == 1.0
    assert s[3] == 2.0 ** -126 and abs(r[3, 0] - 1e-42) <= 2.0 ** -136
    assert s[4] == 2.0 ** 120 and abs(r[4, 0] / 3.0e38 - 1) <= 2.0 ** -4


def test_bad_indices_are_skipped_and_reported():
    from mtp_block_draft_gb300 import DmtpError
    c = new_cache(2, 2, 16, 2, 64)
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
    # attention: positions of a bad page are left out, lengths are cut at the table's reach
    c.check()
    kv = fill_cache(c, [32, 16], gen(3))
    q = randn((2, 1, 2, 64), gen(4))
    out = c.attention(q, i32([40, 20]))
    with pytest.raises(DmtpError) as e:
        c.check()
    assert e.value.word == 18
    ref, tol = reference(np64(q), kv, [32, 16], 1, 0, 64 ** -0.5, True)
    assert (np.abs(np64(out) - ref) <= tol * 1.01 + HALF[BF] * np.abs(ref) + 1e-30).all()


# ---- attention ------------------------------------------------------------------------

KINDS = [(BF, False), (BF, True), (FP, False), (FP, True)]


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("hq,hkv,hd,rows,ps", [
    (16, 16, 64, 1, 16), (32, 4, 128, 1, 64), (32, 4, 128, 8, 16), (8, 1, 64, 3, 5), (5, 5, 64, 8, 128),
    (4, 4, 32, 8, 16), (12, 4, 96, 2, 32), (8, 2, 256, 1, 64), (48, 1, 128, 8, 48), (6, 2, 128, 5, 1),
    (3, 1, 16, 4, 16), (20, 2, 128, 4, 64), (16, 1, 64, 8, 33)])
def test_attention(hq, hkv, hd, rows, ps, dtype, e4m3):
    """Lengths from none and one to several tiles, in one ragged batch."""
    lens = [0, 1, rows, 63, 64, 65, 200, 517]
    blocks = -(-517 // ps)
    g = gen(hq * 1000 + hd + rows)
    c = new_cache(len(lens), blocks, ps, hkv, hd, dtype, e4m3, fill=float("nan"))
    kv = fill_cache(c, lens, g)
    q = randn((len(lens), rows, hq, hd), g, dtype, 1.5)
    a = check_attention(c, q, lens, kv)
    b = c.attention(q, i32(lens))
    assert torch.equal(a, b)  # the same call, the same bits


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("window", [1, 2, 7, 64, 100, 5000])
def test_attention_window(dtype, e4m3, window):
    lens = [0, 1, 5, 64, 130, 400]
    c = new_cache(len(lens), 25, 16, 2, 64, dtype, e4m3, fill=float("nan"))
    g = gen(window)
    kv = fill_cache(c, lens, g)
    check_attention(c, randn((len(lens), 5, 8, 64), g, dtype), lens, kv, window=window)


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("ps", [1, 5, 16, 48, 64])
@pytest.mark.parametrize("rows,window", [(1, 1), (3, 40), (8, 130)])
def test_pages_before_the_window_are_not_looked_up(dtype, e4m3, ps, rows, window):
    """Blocks that no row sees any more, and those past the length, may name pages that are none."""
    for lens in ([0, 2, 60, 64, 333, 320], [700] * 40):
        c = new_cache(len(lens), -(-704 // ps), ps, 2, 64, dtype, e4m3, fill=float("nan"))
        g = gen(window)
        kv = fill_cache(c, lens, g)
        table = c.table.cpu()
        for b, n in enumerate(lens):
            low = max(0, n - rows + 1 - window)
            table[b, :low // ps] = -1
            table[b, -(-n // ps):] = 10 ** 6
        c.table.copy_(table)
        check_attention(c, randn((len(lens), rows, 8, 64), g, dtype), lens, kv, window=window)


@pytest.mark.parametrize("dtype,e4m3", KINDS)
def test_a_window_past_every_position_is_none(dtype, e4m3):
    c = new_cache(2, 40, 16, 2, 64, dtype, e4m3)
    g = gen(0)
    kv = fill_cache(c, [600, 0], g)
    q = randn((2, 8, 4, 64), g, dtype)
    a = check_attention(c, q, [600, 0], kv)
    for window in (640, 2 ** 31 - 1):
        assert torch.equal(a, c.attention(q, i32([600, 0]), window=window))


@pytest.mark.parametrize("dtype,e4m3", [(BF, True), (FP, False)])
def test_attention_many_sequences(dtype, e4m3):
    """More sequences than a grid dimension holds, most of them short, some idle."""
    n, hd, ps = 66000, 64, 16
    r = np.random.RandomState(1)
    lens = r.randint(0, ps + 1, n)
    lens[12345], lens[-1] = 0, 16
    from mtp_block_draft_gb300 import DmtpPagedCache
    table = torch.from_numpy(r.permutation(n).astype(np.int32)[:, None]).cuda()
    c = DmtpPagedCache.alloc(n, ps, 1, hd, table, dtype=dtype, e4m3=e4m3)
    g = gen(2)
    x = randn((n * ps, 1, hd), g, dtype)
    seq, pos = np.repeat(np.arange(n), ps), np.tile(np.arange(ps), n)
    c.write(x, x.flip(0), i32(seq), i32(pos))
    q = randn((n, 1, 2, hd), g, dtype)
    got = np64(c.attention(q, i32(lens)))
    c.check()
    k, v = (np64(t).reshape(n, ps, hd) for t in c.read(i32(seq), i32(pos)))
    s = np.einsum("nhd,nld->nhl", np64(q)[:, 0], k) / 8
    s = np.where(np.arange(ps)[None, None] < lens[:, None, None], s, -np.inf)
    w = np.exp(s - np.where(lens > 0, s.max((1, 2)), 0)[:, None, None])
    w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
    ref = np.einsum("nhl,nld->nhd", w, v)[:, None]
    # as in reference(), with the largest sum of magnitudes of any score
    mag = np.einsum("nhd,nld->nhl", np.abs(np64(q)[:, 0]), np.abs(k)).max() / 8
    ew = (2 * math.expm1(2 * (hd + 4) * U * mag) + 2.0 ** -21 + 8 * mag * U
          + (2.0 ** -11 if e4m3 else 0) + 2 * ps * U)
    tol = ew * np.einsum("nhl,nld->nhd", w, np.abs(v))[:, None] * 1.01 + HALF[dtype] * np.abs(ref) + 17 * 2.0 ** -25 * 448
    assert (np.abs(got - ref) <= (tol if e4m3 else tol - 17 * 2.0 ** -25 * 448 + 1e-30)).all()
    assert (got[lens == 0] == 0).all()


def test_two_threads_on_two_streams():
    """Calls from two host threads, on streams of their own, over one cache."""
    import threading
    from mtp_block_draft_gb300 import sample_rows
    lens = [900, 1700]
    c = new_cache(2, 110, 16, 2, 128, BF, True)
    g = gen(6)
    fill_cache(c, lens, g)
    q = [randn((2, 1, 8, 128), g) for _ in range(2)]
    z = randn((4, 30000), g, FP, 3.0)
    u, k = torch.rand(4, device="cuda", generator=g), i32([5, 0, 40, 9])
    ln = i32(lens)
    want = [(c.attention(x, ln), sample_rows(z, u, top_k=k)) for x in q]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(200):
                a, b = c.attention(q[i], ln), sample_rows(z, u, top_k=k)
            s.synchronize()
            if not (torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])):
                bad.append(i)

    t = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for x in t:
        x.start()
    for x in t:
        x.join()
    assert not bad
    c.check()


@pytest.mark.parametrize("dtype,e4m3", KINDS)
def test_attention_one_long_sequence_among_short_ones(dtype, e4m3):
    """One unit split over many CTAs beside units that fit in one; peaked scores."""
    lens = [20000, 3, 0, 190]
    c = new_cache(len(lens), -(-20000 // 64), 64, 2, 128, dtype, e4m3)
    g = gen(9)
    kv = fill_cache(c, lens, g, kmul=2.0)
    check_attention(c, randn((len(lens), 2, 8, 128), g, dtype, 2.0), lens, kv)


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("hd", [32, 64, 128])
def test_values_that_a_row_does_not_see_do_not_reach_it(dtype, e4m3, hd):
    """NaN and infinite keys and values at the positions of later rows, or before a row's
    window: rows that do not see them are what they are without them; rows that do get them."""
    n, rows, win = 150, 4, 40
    g = gen(5)
    for window, where in ((0, [n - 1, n - 2]), (win, [n - rows - win + 1, n - rows - win + 2])):
        c = new_cache(1, 10, 16, 2, hd, dtype, e4m3)
        fill_cache(c, [n], g)
        q = randn((1, rows, 8, hd), g, dtype)
        clean = c.attention(q, i32([n]), window=window)
        k, v = c.read(i32([0] * len(where)), i32(where))
        k[0], v[0] = float("nan"), float("inf")
        v[1, 0, 3:5] = float("nan")
        c.write(k, v, i32([0] * len(where)), i32(where))
        got = c.attention(q, i32([n]), window=window)
        c.check()
        for i in range(rows):
            p = n - rows + i
            sees = [j <= p and (not window or j > p - window) for j in where]
            same = torch.equal(got[0, i], clean[0, i])
            assert same == (not any(sees)), (window, i)
            if sees[0]:
                assert torch.isnan(got[0, i]).any()
            elif sees[1]:
                assert torch.isnan(got[0, i, :4, 3:5]).all() and torch.isfinite(got[0, i, 4:]).all()


def test_attention_strides_shared_pages_and_pools():
    """A pool that holds two layers, a prefix page that two sequences share, q as a strided
    view and out as a slice."""
    from mtp_block_draft_gb300 import DmtpPagedCache
    hkv, ps, hd, hq = 2, 16, 128, 8
    pool = torch.full((9, 2, 2, hkv, ps, hd), float("nan"), dtype=BF, device="cuda")  # page, layer, k/v
    table = torch.full((2, 6), 12345, dtype=torch.int32, device="cuda")[:, 1:5]       # strided rows
    table[:] = i32([[7, 2, 4, 0], [7, 2, 5, 1]])
    c = DmtpPagedCache(pool[:, 1, 0], pool[:, 1, 1], table)
    g = gen(0)
    lens = [61, 40]
    fill_cache(c, [61, 0], g)
    k = randn((8, hkv, hd), g)
    c.write(k, k, i32([1] * 8), i32(range(32, 40)))
    kv = stored(c, lens)
    assert torch.isnan(pool[:, 0]).all()
    big = randn((2, 3, 3 * hq, hd + 8), g)
    q = big[:, :, hq:2 * hq, 8:]
    box = torch.full((2, 5, hq, hd), 7.0, dtype=BF, device="cuda")
    check_attention(c, q, lens, kv, out=box[:, 1:4])
    assert (box[:, 0] == 7).all() and (box[:, 4] == 7).all()


def test_attention_past_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^31."""
    from mtp_block_draft_gb300 import DmtpPagedCache
    hkv, ps, hd = 1, 64, 128
    stride = 3 * 2 ** 29 + 1024
    buf = [torch.zeros(2 * stride + ps * hd, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = (b.view(F8).as_strided((3, hkv, ps, hd), (stride, ps * hd, hd, 1)) for b in buf)
    ks, vs = (torch.ones((3, hkv, ps), device="cuda") for _ in range(2))
    c = DmtpPagedCache(k, v, i32([[2, 0, 1]]), ks, vs)
    g = gen(2)
    kk = randn((190, 1, hd), g)
    c.write(kk, kk, i32([0] * 190), i32(range(190)))
    r, _ = c.read(i32([0] * 190), i32(range(190)))
    assert (np.abs(np64(r) - np64(kk)) <= 2.0 ** -4 * np.abs(np64(kk)) + 2.0 ** -9).all()
    assert int(buf[0][2 * stride:].count_nonzero()) > 0
    kd = np.moveaxis(np64(r), 1, 0)
    check_attention(c, randn((1, 1, 4, hd), g), [190], [[kd, kd]])


@pytest.mark.parametrize("dtype,e4m3", [(BF, False), (BF, True), (FP, False)])
def test_attention_extreme_scores(dtype, e4m3):
    """Scores far apart and all equal, a scale of zero, zero rows and rows of very different
    size in one cache."""
    hd, n = 64, 300
    c = new_cache(1, 20, 16, 1, hd, dtype, e4m3)
    g = gen(1)
    k, v = randn((n, 1, hd), g, dtype), randn((n, 1, hd), g, dtype)
    k *= torch.logspace(-6, 1.2, n, device="cuda")[:, None, None].to(dtype)
    v *= torch.logspace(3, -6, n, device="cuda")[:, None, None].to(dtype)
    k[17], v[40] = 0, 0
    c.write(k, v, i32([0] * n), i32(range(n)))
    kv = stored(c, [n])
    q = randn((1, 2, 4, hd), g, dtype, 3.0)
    q[0, 0, 1] = 0
    q[0, 1, 2] *= 1e-20
    check_attention(c, q, [n], kv)
    check_attention(c, q, [n], kv, scale=0.0)
    check_attention(c, q, [n], kv, scale=-0.25)


@pytest.mark.parametrize("hd,rows", [(64, 1), (128, 8)])
def test_attention_of_value_rows_of_very_different_sizes(hd, rows):
    """E4M3 value rows near 0 (scale 2^-126, an fp32 row of 1e-36 as a bf16 one) next to ordinary
    ones: they add next to nothing to the output, but their weights count in full. Alone, they
    are good to n 2^-76: a weight times 2^(e + 60) is rounded to fp16, by 2^-25 at most where it
    is below the normal range, of values up to 448 in units of 2^-60."""
    lens = [1, 16, 333, 2000]
    for tiny in ("some", "most", "all"):
        c = new_cache(len(lens), 40, 64, 2, hd, BF, True, fill=1.0)
        g = gen(hd)
        n = sum(lens)
        seq = np.concatenate([np.full(x, b) for b, x in enumerate(lens)])
        pos = np.concatenate([np.arange(x) for x in lens])
        small = torch.rand((n, 2, 1), device="cuda", generator=g) < {"some": 0.5, "most": 0.95, "all": 2}[tiny]
        v = randn((n, 2, hd), g, FP)
        v = torch.where(small, v * 1e-36, v)
        c.write(randn((n, 2, hd), g, BF, 1.5), v.to(BF), i32(seq), i32(pos))
        kv = stored(c, lens)
        q = randn((len(lens), rows, 8, hd), g, BF, 1.5)
        if tiny != "all":
            check_attention(c, q, lens, kv)
            continue
        assert float(c.v_scale.min()) == 2.0 ** -126
        out = np64(c.attention(q, i32(lens)))
        ref, _ = reference(np64(q), kv, lens, rows, 0, hd ** -0.5, pair=False)
        assert (np.abs(out - ref).max((1, 2, 3)) <= np.asarray(lens) * 2.0 ** -76).all()


def test_attention_streams_graphs_and_workspaces():
    """On a side stream; two calls captured into two graphs with workspaces of their own,
    replayed at once on two streams with lengths that changed since the capture."""
    lens = [300, 77]
    c = new_cache(2, 20, 16, 4, 128)
    g = gen(3)
    kv = fill_cache(c, lens, g)
    q = randn((2, 1, 16, 128), g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s1):
        out = c.attention(q, i32(lens))
    torch.cuda.synchronize()
    assert torch.equal(out, check_attention(c, q, lens, kv))
    n = c.attention_workspace(1, 16)
    state = []
    for _ in range(2):
        ln, o = i32([5, 6]), torch.empty_like(q)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        ids = torch.empty(2, dtype=torch.int32, device="cuda")
        u = torch.full((2,), 0.5, device="cuda")
        gr = torch.cuda.CUDAGraph()
        c.attention(q, ln, out=o, workspace=ws)
        torch.cuda.synchronize()
        from mtp_block_draft_gb300 import add_rmsnorm_e4m3, sample_rows
        x = o.view(2, -1)
        with torch.cuda.graph(gr):
            c.attention(q, ln, out=o, workspace=ws)
            y = add_rmsnorm_e4m3(x, None, torch.ones(x.shape[1], device="cuda"))
            sample_rows(x, u, ids=ids)
        state.append((gr, ln, o, ids, u, y))
    state[0][1].copy_(i32(lens))
    state[1][1].copy_(i32([lens[0], 0]))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (gr, *_) in zip((s1, s2), state):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(state[0][2], out)
    assert torch.equal(state[1][2][0], out[0]) and (state[1][2][1] == 0).all()
    for gr, ln, o, ids, u, y in state:
        assert torch.equal(ids, sample_rows(o.view(2, -1), u))
        assert torch.equal(y[1].view(torch.uint8), add_rmsnorm_e4m3(o.view(2, -1), None, torch.ones(2048, device="cuda"))[1].view(torch.uint8))


# ---- norm -----------------------------------------------------------------------------

@pytest.mark.parametrize("xt", [BF, FP])
@pytest.mark.parametrize("yt", [BF, FP, None])
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 520), (32, 2048), (5, 2056), (7, 5120), (2, 16384), (300, 1024), (2, 8200)])
def test_add_rmsnorm_e4m3(rows, d, xt, yt):
    from mtp_block_draft_gb300 import add_rmsnorm_e4m3
    g = gen(rows + d)
    big = randn((rows, d + 8), g, xt, 3.0)
    x = big[:, :d]
    y = None if yt is None else randn((rows, d), g, yt)
    gain = randn((d,), g, BF if d % 16 else FP) + 1
    xo, q, s = add_rmsnorm_e4m3(x, y, gain, 1e-5)
    if yt is None:
        assert xo is x
        sm = np64(x)
    else:
        sm = (x.float() + y.float())
        assert torch.equal(xo, sm.to(xt))
        sm = np64(sm)
    h = sm / np.sqrt((sm ** 2).mean(-1, keepdims=True) + float(np.float32(1e-5))) * np64(gain)
    sc = np64(s)[:, None]
    # h carries the factor's rounding and two products: 3 u; E4M3's rounding is monotone, so the
    # stored value lies between the roundings of h (1 -+ 3u); the scale belongs to one of them
    amax = np.abs(h).max(-1)
    for r in range(rows):
        assert sc[r, 0] in {fp8.pow2_scale(amax[r] * (1 - 4 * U)), fp8.pow2_scale(amax[r] * (1 + 4 * U))}
        a, b = (fp8.round_e4m3(np.clip(h[r] * (1 + e * 4 * U) / sc[r, 0], -448, 448)) for e in (-1, 1))
        got = np64(q[r])
        assert ((got >= np.minimum(a, b)) & (got <= np.maximum(a, b))).all()


def test_norm_in_place_special_rows_and_padding():
    from mtp_block_draft_gb300 import add_rmsnorm_e4m3
    d = 64
    x = randn((6, d), gen(0), FP)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e-30
    y = torch.zeros_like(x)
    gain = torch.ones(d, device="cuda")
    q = torch.zeros((8, d + 8), dtype=torch.uint8, device="cuda").view(F8)
    s = torch.full((8,), -1.0, device="cuda")
    xi = x.clone()
    xo, _, _ = add_rmsnorm_e4m3(xi, y, gain, 0.0, x_out=xi, q=q[:6, :d], scale=s[:6])
    assert xo is xi and torch.equal(xi.nan_to_num(9), x.nan_to_num(9))
    v = q.float().cpu()
    assert (v[1, :d] == 0).logical_or(v[1, :d].isnan()).all()       # 0 / 0 with eps 0
    assert v[2, :d].isnan().all()
    assert v[3, 7].isnan() and (v[3, :7] == 0).all()
    assert (v[6:] == 0).all() and (v[:6, d:] == 0).all() and (s[6:] == -1).all()
    one = add_rmsnorm_e4m3(x[:1].clone(), y[:1], gain, 0.0)[1]
    assert torch.equal(one.view(torch.uint8), q[:1, :d].view(torch.uint8))  # rows do not meet


# ---- sampling -------------------------------------------------------------------------

def plain_pick(z, u, t=1.0, k=0, p=1.0, m=0.0):
    """(id, kept) of one row in float64."""
    z = np.asarray(z, np.float64)
    ok = z > -np.inf
    if not ok.any():
        return -1, 0
    if not t > 0:
        return int(np.argmax(np.where(ok, z, -np.inf))), 1
    order = np.lexsort((np.arange(z.size), -np.where(ok, z, -np.inf)))[:ok.sum()]
    if k > 0:
        order = order[:k]
    top = z[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(z[order] == top, 1.0, np.exp((z[order] - top) / t))
    if p < 1:
        before = np.cumsum(w) - w
        stay = before < p * w.sum()
        stay[0] = True
        order, w = order[stay], w[stay]
    stay = w >= min(m, 1.0)
    order, w = order[stay], w[stay]
    w, order = w[np.argsort(order)], np.sort(order)
    run = np.cumsum(w)
    u = 0.0 if not u > 0 else u
    return int(order[min(np.searchsorted(run, u * run[-1], side="right"), len(order) - 1)]), len(order)


def run_sample(z, u, t=None, k=None, p=None, m=None):
    from mtp_block_draft_gb300 import sample_rows
    kept = torch.full((z.shape[0],), -9, dtype=torch.int32, device="cuda")
    f = lambda a, dt: None if a is None else torch.as_tensor(a, dtype=dt, device="cuda")
    ids = sample_rows(z, f(u, FP), f(t, FP), f(k, torch.int32), f(p, FP), f(m, FP), kept=kept)
    return ids.cpu().numpy(), kept.cpu().numpy()


def check_rows(z, u, t, k, p, m):
    ids, kept = run_sample(z, u, t, k, p, m)
    f = lambda a, i, d: d if a is None else float(np.float32(a[i]))
    zz = np64(z)
    for i in range(z.shape[0]):
        want = plain_pick(zz[i], f(u, i, 0), f(t, i, 1.0), int(f(k, i, 0)), f(p, i, 1.0), f(m, i, 0.0))
        assert (ids[i], kept[i]) == want, (i, ids[i], kept[i], want)


@pytest.mark.parametrize("V,n", [(1, 24), (2, 24), (31, 24), (512, 24), (513, 60), (2049, 24), (5000, 60), (8193, 24),
                                 (32000, 24), (151936, 24), (262144, 12), (8193, 130), (20001, 128), (32000, 127),
                                 (32000, 140), (151936, 129), (262144, 128), (32000, 13), (50176, 24),
                                 (50177, 30), (32000, 60), (100352, 40), (100353, 40), (50176, 154)])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_sample_rows(V, n, dtype):
    """Every mixture of filters, one per row, for few rows and many. bf16 logits tie often."""
    r = np.random.RandomState(V + n)
    big = randn((n, V + 3), gen(V), dtype, 2.5)
    z = big[:, :V] if V % 2 else big[:, 3:].clone()
    check_rows(z, r.rand(n), r.choice([0.0, 0.3, 0.7, 1.0, 2.0], n), r.choice([0, 1, 2, 50, 1000, V], n),
               r.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0], n), r.choice([0.0, 0.01, 0.2, 1.0], n))
    check_rows(z, r.rand(n), None, None, None, None)


@pytest.mark.parametrize("copies", [1, 22])
def test_sample_ties_and_flat_rows(copies):
    V = 9000
    z = torch.zeros((6, V), device="cuda")
    z[1, ::2] = 1.0
    z[2, 5:] = -1.0
    z[3] = torch.arange(V, device="cuda") % 3
    z[4, ::2] = -0.0
    u = [0.0, 0.25, 0.5, 0.75, 0.5, 0.999]
    for k in (0, 1, 7, 4500, 4501):
        for p in (0.0, 0.25, 0.5, 1.0):
            for m in (0.0, 0.5, 1.0):
                if copies == 1:
                    check_rows(z, u, [1.0] * 6, [k] * 6, [p] * 6, [m] * 6)
                    continue
                ids, kept = run_sample(z.repeat(copies, 1), u * copies, [1.0] * 6 * copies, [k] * 6 * copies,
                                       [p] * 6 * copies, [m] * 6 * copies)
                one = run_sample(z, u, [1.0] * 6, [k] * 6, [p] * 6, [m] * 6)
                assert (ids.reshape(copies, 6) == one[0]).all() and (kept.reshape(copies, 6) == one[1]).all()


@pytest.mark.parametrize("V,copies", [(100, 1), (20000, 1), (20000, 13)])
def test_sample_masked_rows_and_odd_numbers(V, copies):
    inf, nan = float("inf"), float("nan")
    z = randn((10, V), gen(0), FP, 3.0)
    z[0] = -inf
    z[1] = nan
    z[2, 1:] = -inf
    z[3, :-1] = torch.finfo(FP).min
    z[4] = torch.finfo(FP).min
    z[5, 10], z[5, 20] = inf, inf
    z[6, ::2] = -inf
    z[6, 1::4] = nan
    z[7] = torch.finfo(FP).max
    z[8, 50] = torch.finfo(FP).max
    z[9, :3000] -= 40.0                    # the largest logits come late in the row
    u = [0.5, 0.5, 0.9, 0.3, 0.6, 0.7, 0.2, 0.99, 0.5, 0.5] * copies
    n = 10 * copies
    for t in (1.0, 0.0, 1e-38, 1e-3, 1e6):
        for k, p, m in ((0, 1.0, 0.0), (3, 0.9, 0.0), (0, 0.5, 0.1)):
            check_rows(z.repeat(copies, 1), u, [t] * n, [k] * n, [p] * n, [m] * n)
    # numbers outside their ranges
    x = z[9:].expand(6, V).contiguous()
    ids, kept = run_sample(x, [-1.0, nan, 1.0, 2.0, inf, 0.0], [1.0] * 6, [50] * 6)
    assert ids[0] == ids[1] == ids[5] and ids[2] == ids[3] == ids[4] and (kept == 50).all()
    best = int(np.argmax(np64(x)[0]))
    ids, kept = run_sample(x, [0.5] * 6, [nan, -1.0, 0.0, 1.0, 1.0, 1.0], [0, 0, 0, -4, 1, 0],
                           [1.0, 1.0, 1.0, nan, 1.0, -1.0], [0.0, 0.0, 0.0, nan, 0.0, 0.0])
    assert [ids[i] for i in (0, 1, 2, 4, 5)] == [best] * 5 and kept[3] == V


@pytest.mark.parametrize("V,copies", [(100, 1), (20000, 1), (20000, 33), (104001, 33)])
def test_sample_temperatures_past_their_range(V, copies):
    """Above 1e30, infinity among them, a temperature counts as 1e30: ordinary logits weigh the
    same, the type's lowest value still weighs nothing."""
    z = randn((4, V), gen(5), FP, 3.0)
    z[1, ::3] = torch.finfo(FP).min
    z[2, 1::2] = -float("inf")
    z[3] = torch.finfo(FP).min
    n = 4 * copies
    u = [0.1, 0.5, 0.7, 0.999] * copies
    for t in (1e30, 1e35, float("inf")):
        for k, p, m in ((0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.5, 0.0), (40, 0.9, 0.5)):
            args = [k] * n, [p] * n, [m] * n
            ids, kept = run_sample(z.repeat(copies, 1), u, [t] * n, *args)
            want = [plain_pick(np64(z)[i % 4], float(np.float32(u[i])), 1e30, k, float(np.float32(p)), m) for i in range(4)]
            assert [(int(a), int(b)) for a, b in zip(ids, kept)] == want * copies, (t, k, p)


def test_sample_masked_rows_among_many_of_a_large_vocabulary():
    inf, nan, V, copies = float("inf"), float("nan"), 104001, 14
    z = randn((10, V), gen(0), FP, 3.0)
    z[0] = -inf
    z[1] = nan
    z[2, 1:] = -inf
    z[3, :-1] = torch.finfo(FP).min
    z[4] = torch.finfo(FP).min
    z[5, 10], z[5, 20] = inf, inf
    z[6, ::2] = -inf
    z[6, 1::4] = nan
    z[7] = torch.round(z[7])               # large groups of ties
    z[8, 50] = torch.finfo(FP).max
    z[9, :3000] -= 40.0                    # the largest logits come late in the row
    u = [0.5, 0.5, 0.9, 0.3, 0.6, 0.7, 0.2, 0.99, 0.5, 0.5]
    zz = np64(z)
    for t in (1.0, 0.0, 1e-3, 1e6):
        for k, p, m in ((0, 1.0, 0.0), (3, 0.9, 0.0), (5000, 0.7, 0.0), (0, 0.5, 0.1)):
            n = 10 * copies
            ids, kept = run_sample(z.repeat(copies, 1), u * copies, [t] * n, [k] * n, [p] * n, [m] * n)
            want = [plain_pick(zz[i], float(np.float32(u[i])), float(np.float32(t)), k, float(np.float32(p)),
                               float(np.float32(m))) for i in range(10)]
            assert [(int(a), int(b)) for a, b in zip(ids, kept)] == want * copies, (t, k, p, m)


def test_sample_frequencies():
    """Evenly spread u visit every kept token in proportion to its weight: with n numbers
    (i + 1/2) / n the count of a token is within one of n times its probability."""
    V, n = 600, 4096
    z = randn((1, V), gen(8), FP, 2.0)
    ids, _ = run_sample(z.expand(n, V).contiguous(), (np.arange(n) + 0.5) / n, [0.8] * n, [40] * n)
    w = np.exp((np64(z)[0] - np64(z).max()) / float(np.float32(0.8)))
    w[np.argsort(-w, kind="stable")[40:]] = 0
    assert np.abs(np.bincount(ids, minlength=V) - n * w / w.sum()).max() <= 1.0 + 1e-3


# ---- together -------------------------------------------------------------------------

@pytest.mark.parametrize("e4m3", [False, True])
def test_a_decode_loop(e4m3):
    """Ten steps of a small model whose attention, norm and sampling are the operators, against
    the same steps in float64 from the operators' own stored values (so that each step is
    compared, not the drift): qkv -> write -> attention -> add + norm -> logits -> sample."""
    from mtp_block_draft_gb300 import add_rmsnorm_e4m3, sample_rows
    B, d, hq, hkv, hd, V = 3, 256, 8, 2, 64, 1000
    g = gen(4)
    c = new_cache(B, 4, 16, hkv, hd, BF, e4m3)
    emb, wqkv = randn((V, d), g, BF), randn(((hq + 2 * hkv) * hd, d), g, BF, 0.06)
    wo, head = randn((d, hq * hd), g, BF, 0.06), randn((V, d), g, BF, 0.1)
    gain = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(BF)
    lens, tok = np.array([0, 13, 30]), i32([1, 2, 3])
    fill_cache(c, list(lens), g)
    for step in range(10):
        x = emb[tok.long()].float()
        qkv = (x.to(BF) @ wqkv.T)
        q, k, v = (qkv[:, a * hd:b * hd].view(B, -1, hd) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        qr = c.write(k, v, i32(range(B)), i32(lens), q=q, rope_theta=10000.0)
        lens = lens + 1
        kv = stored(c, list(lens))
        att = check_attention(c, qr.view(B, 1, hq, hd), list(lens), kv)
        y = att.view(B, -1) @ wo.T
        x2, hq8, s = add_rmsnorm_e4m3(x, y, gain)
        assert torch.equal(x2, x + y.float())
        h = np64(x2)
        h = h / np.sqrt((h ** 2).mean(-1, keepdims=True) + 1e-6) * np64(gain)
        deq = np64(hq8) * np64(s)[:, None]
        assert (np.abs(deq - h) <= 2.0 ** -4 * np.abs(h) + 2.0 ** -9 * np64(s)[:, None]).all()
        logits = torch.from_numpy(deq).cuda().float() @ head.float().T
        u = torch.rand(B, device="cuda", generator=g)
        t, kk, p = torch.full((B,), 0.8, device="cuda"), i32([0, 20, 5]), torch.tensor([0.9, 1.0, 0.7], device="cuda")
        tok = sample_rows(logits, u, t, kk, p)
        zz = np64(logits)
        for b in range(B):
            want, _ = plain_pick(zz[b], float(u[b]), float(t[b]), int(kk[b]), float(p[b]))
            assert int(tok[b]) == want
    c.check()


def test_the_norm_matches_the_draft_heads_rows():
    """Without y the operator is the draft heads' own row quantisation: the logits of the
    no-alloc head on a dequantised row equal those on the row up to E4M3's rounding."""
    from mtp_block_draft_gb300 import add_rmsnorm_e4m3
    x = randn((16, 512), gen(0), FP, 5.0)
    gain = (1 + 0.1 * torch.randn(512, device="cuda", generator=gen(1))).to(BF)
    _, q, s = add_rmsnorm_e4m3(x, None, gain)
    h = np64(x)
    h = h / np.sqrt((h ** 2).mean(-1, keepdims=True) + 1e-6) * np64(gain)
    want, sc = fp8.quantize_rows(h)
    # float64 and fp32 agree unless a value lies within 4u of a rounding border
    assert (np64(s) == sc).all() and np.mean(np64(q) != want) < 1e-3


@pytest.mark.parametrize("hq,hkv", [(8, 1), (32, 4), (128, 8)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_written_together_and_apart_are_the_same(hq, hkv, e4m3):
    """Many rows in one call, and the same in calls of a few: the same bits, whatever the form."""
    n, hd = 1301, 64
    g = gen(hq)
    k, v, q = randn((n, hkv, hd), g), randn((n, hkv, hd), g), randn((n, hq, hd), g)
    caches = [new_cache(3, 28, 16, hkv, hd, BF, e4m3) for _ in range(2)]
    seq, pos = i32([i % 4 - 1 for i in range(n)]), i32([i // 4 for i in range(n)])
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    caches[0].write(k, v, seq, pos, q=q, q_out=a, rope_theta=1e4)
    for i in range(0, n, 50):
        s = slice(i, i + 50)
        caches[1].write(k[s], v[s], seq[s], pos[s], q=q[s], q_out=b[s], rope_theta=1e4)
    assert torch.equal(a, b)
    for x, y in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    if e4m3:
        assert torch.equal(caches[0].k_scale, caches[1].k_scale)
        assert torch.equal(caches[0].v_scale, caches[1].v_scale)


@pytest.mark.parametrize("hq,hkv,rows", [(24, 1, 1), (17, 1, 1), (8, 2, 8), (32, 4, 8), (33, 1, 5), (48, 2, 8)])
@pytest.mark.parametrize("ps,window", [(16, 0), (64, 0), (5, 0), (64, 1), (16, 70), (48, 200)])
def test_attention_of_many_queries(hq, hkv, rows, ps, window):
    """More than 16 queries of a kv head in E4M3: steps of one and two tiles, split and whole."""
    for lens in ([0, 1, rows, 63, 64, 65, 127, 128, 129, 191, 250], [1400, 3, 2111, 640, 0, 1]):
        g = gen(hq + ps + window)
        c = new_cache(len(lens), -(-max(lens) // ps), ps, hkv, 128, BF, True, fill=float("nan"))
        kv = fill_cache(c, lens, g)
        q = randn((len(lens), rows, hq, 128), g, BF, 1.5)
        a = check_attention(c, q, lens, kv, window=window)
        assert torch.equal(a, c.attention(q, i32(lens), window=window))


@pytest.mark.parametrize("rows,window", [(8, 0), (4, 40), (3, 300)])
def test_attention_of_many_queries_keeps_odd_values_to_the_rows_that_see_them(rows, window):
    n, hq = 1000, 24
    g = gen(7)
    where = [n - 1, n - 2] if not window else [n - rows - window + 1, n - rows - window + 2]
    c = new_cache(1, 63, 16, 2, 128, BF, True)
    fill_cache(c, [n], g)
    q = randn((1, rows, hq, 128), g)
    clean = c.attention(q, i32([n]), window=window)
    k, v = c.read(i32([0, 0]), i32(where))
    k[0], v[0] = float("nan"), float("inf")
    v[1, 0, 3:5] = float("nan")
    c.write(k, v, i32([0, 0]), i32(where))
    got = c.attention(q, i32([n]), window=window)
    c.check()
    for i in range(rows):
        p = n - rows + i
        sees = [j <= p and (not window or j > p - window) for j in where]
        assert torch.equal(got[0, i], clean[0, i]) == (not any(sees)), i
        if sees[0]:
            assert torch.isnan(got[0, i]).all()
        elif sees[1]:
            assert torch.isnan(got[0, i, :12, 3:5]).all() and torch.isfinite(got[0, i, 12:]).all()


def test_attention_of_many_queries_leaves_bad_pages_out():
    lens, rows = [700, 64, 333], 8
    g = gen(9)
    c = new_cache(3, 44, 16, 2, 128, BF, True)
    kv = fill_cache(c, lens, g)
    q = randn((3, rows, 16, 128), g)
    good = c.attention(q, i32(lens))
    c.check()
    c.table[0, 10] = -5
    out = c.attention(q, i32(lens))
    from mtp_block_draft_gb300 import DmtpError
    with pytest.raises(DmtpError) as e:
        c.check()
    assert e.value.word == 16 and torch.equal(out[1:], good[1:])
    keep = np.r_[0:160, 176:700]
    cut = [[x[:, keep] for x in kv[0]]]
    ref, tol = reference(np64(q[:1]), cut, [684], rows, 0, 128 ** -0.5, False)
    assert (np.abs(np64(out[:1]) - ref) <= tol * 1.01 + HALF[BF] * np.abs(ref) + 1e-30).all()
