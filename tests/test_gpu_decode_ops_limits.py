"""The decode-step operators at the ends of what they document: numbers, sizes and calls where
one part of a kernel hands over to another. Plain forms and bounds are those of
test_gpu_decode_ops.py."""

import numpy as np
import pytest
import torch

from test_gpu_decode_ops import (BF, F8, FP, check_attention, check_rows, gen, i32, new_cache, np64, plain_pick, randn,
                                 run_sample, stored)

pytestmark = pytest.mark.gpu

f32 = lambda x: float(np.float32(x))


# ---- sampling -------------------------------------------------------------------------

def near_zero_rows(V, seed):
    """Logits around zero in the smallest steps of fp32: no two of the numbers are far enough apart
    to fall into different bins of weight, so that the cut is found by the numbers' bits alone."""
    r = np.random.RandomState(seed)
    z = np.zeros((6, V), np.float32)
    z[0] = -1e-40 * r.randint(0, 4, V)
    z[0, 0] = 1.9999999
    z[1] = 1.4e-45 * r.randint(-3, 4, V)
    z[2] = -1.4e-45 * r.randint(0, 3, V)
    z[3] = np.where(r.rand(V) < 0.5, -0.0, -1e-38)
    z[4] = np.where(r.rand(V) < 0.9, 0.0, -3e-39)
    z[5] = -r.rand(V) * 1e-37
    return z


@pytest.mark.parametrize("V", [7, 100, 3000, 20000])
@pytest.mark.parametrize("t", [1.0, 1000.0])
def test_sample_zeros_beside_the_smallest_negative_logits(V, t):
    z = torch.from_numpy(near_zero_rows(V, V)).cuda()
    u = [0.1, 0.3, 0.5, 0.7, 0.9, 0.99]
    for k in sorted({0, 1, V // 7, V // 2, V - 2}):
        for p in (1.0, 0.37, 0.913):
            for m in (0.0, 1.0):
                check_rows(z, u, [t] * 6, [k] * 6, [p] * 6, [m] * 6)


def check_copies(z, copies, u, t, k, p, m=0.0):
    """The rows of z, each `copies` times in one call, against the plain form of each."""
    n = z.shape[0]
    ids, kept = run_sample(z.repeat(copies, 1), list(u) * copies, [t] * n * copies, [k] * n * copies,
                           [p] * n * copies, [m] * n * copies)
    zz = np64(z)
    want = [plain_pick(zz[i], f32(u[i]), f32(t), k, f32(p), f32(m)) for i in range(n)]
    assert [(int(a), int(b)) for a, b in zip(ids, kept)] == want * copies, (t, k, p, m)


def test_sample_zeros_beside_the_smallest_negative_logits_of_many_large_rows():
    V = 104001
    z = torch.from_numpy(near_zero_rows(V, 1)).cuda()
    for k, p in ((0, 0.37), (3, 1.0), (V // 2, 1.0), (V // 2, 0.913), (V - 5, 0.5)):
        check_copies(z, 22, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], 1.0, k, p)


@pytest.mark.parametrize("V,copies", [(60, 1), (20000, 2), (20000, 33), (104001, 33)])
def test_sample_top_p_right_after_a_top_k_that_takes_whole_bins(V, copies):
    """top_k ends at a bin's end, or in a bin of one number's ties, so that nothing has to be split
    before top_p's search begins; the same call gives the same rows each time."""
    r = np.random.RandomState(V)
    z = np.zeros((4, V), np.float32)
    z[0] = -(np.arange(V) % 20)                 # groups of ties, bins apart
    z[1] = -(np.arange(V) // (V // 4))
    z[2] = r.permutation(np.where(np.arange(V) < V // 3, 7.0, -1.0))
    z[3] = 1e4 * r.randint(0, 3, V)
    zz, z = z.astype(np.float64), torch.from_numpy(z).cuda()
    u = [0.15, 0.45, 0.65, 0.85]
    for t in (1.0, 1e-9):
        for k in (V // 20, V // 4, V // 3, 2, V // 2):
            want = [plain_pick(zz[i], f32(u[i]), f32(t), k, f32(0.613), 0.0) for i in range(4)]
            for _ in range(10):
                ids, kept = run_sample(z.repeat(copies, 1), u * copies, [t] * 4 * copies, [k] * 4 * copies,
                                       [0.613] * 4 * copies, None)
                assert [(int(a), int(b)) for a, b in zip(ids, kept)] == want * copies, (t, k)


def tied_rows(V):
    """Rows of which nearly every logit has the same weight, with many bits set in it."""
    z = np.zeros((5, V), np.float32)
    z[1, 5:] = -0.25
    z[2, 1:] = -2.5
    z[3, V // 3:] = -0.7
    z[4] = np.where(np.arange(V) % 1000 == 7, 3.0, 2.9375)
    return z


@pytest.mark.parametrize("V", [131073, 151936, 200003, 262144])
@pytest.mark.parametrize("copies", [1, 26])
def test_sample_large_vocabularies_of_ties(V, copies):
    """More than 2^17 logits of one weight: the weights of a bin add up past 32 bits in each part."""
    z = torch.from_numpy(tied_rows(V)).cuda()
    u = [0.1, 0.35, 0.6, 0.85, 0.999]
    for k, p, m in ((0, 0.9, 0.0), (0, 0.31, 0.5), (V - 3, 0.77, 0.0)):
        check_copies(z, copies, u, 1.0, k, p, m)
    if copies == 1:  # the same logits in bf16
        zb = z.to(torch.bfloat16)
        check_copies(zb, 1, u, 0.7, 0, 0.9)


# ---- attention ------------------------------------------------------------------------

@pytest.mark.parametrize("hd,hq,rows", [(64, 2, 1), (128, 2, 1), (128, 16, 1), (64, 8, 4), (128, 16, 8)])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-6, 1e-9])
@pytest.mark.parametrize("zeros", ["first", "one", "last", "half", "sink"])
def test_attention_of_small_values_beside_rows_of_zeros(hd, hq, rows, size, zeros):
    """E4M3 value rows of zeros have scale 1 whatever the others' size. They weigh in the sum of
    weights alone: what the other rows add is as exact as without them."""
    lens = [40, 333, 1500]
    c = new_cache(len(lens), 24, 64, 2, hd, BF, True, fill=1.0)
    g = gen(hd + rows)
    n = sum(lens)
    seq = np.concatenate([np.full(x, b) for b, x in enumerate(lens)])
    pos = np.concatenate([np.arange(x) for x in lens])
    k, v = randn((n, 2, hd), g), (randn((n, 2, hd), g, torch.float32) * size).to(BF)
    q = randn((len(lens), rows, hq, hd), g, BF, 1.5)
    if zeros == "half":
        v[torch.rand((n, 2), device="cuda", generator=g) < 0.5] = 0
    else:
        at = {"first": 0, "one": 17, "last": -rows, "sink": 3}[zeros]
        at = [int(np.flatnonzero(seq == b)[at]) for b in range(len(lens))]
        v[at] = 0
        if zeros == "sink":  # a score some 15 above the others', for every query
            q[..., 0], k[:, :, 0] = 8.0, 0.0
            k[at] = 0
            k[at, :, 0] = 1.9 * hd ** 0.5
    c.write(k, v, i32(seq), i32(pos))
    assert (np64(c.v_scale) == 1).any() and (size > 1e-3 or float(c.v_scale.min()) < 2.0 ** -15)
    check_attention(c, q, lens, stored(c, lens))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hkv,ps", [(1, 16), (4, 1)])
def test_pages_of_one_head_or_one_row_with_other_strides(dtype, hkv, ps):
    """A pool kept as [pages, rows, heads, head_dim] is dense page by page when one of the two is 1."""
    from mtp_block_draft_gb300 import DmtpPagedCache
    hd, n = 64, 90
    blocks = -(-n // ps)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").flip(0)[None]
    made = [torch.zeros((blocks, ps, hkv, hd), dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2)]
    c = DmtpPagedCache(made[0], made[1], table)
    d = DmtpPagedCache.alloc(blocks, ps, hkv, hd, table, dtype=dtype)
    g = gen(hkv)
    k, v, q = randn((n, hkv, hd), g, dtype), randn((n, hkv, hd), g, dtype), randn((1, 2, 8, hd), g, dtype)
    for x in (c, d):
        x.write(k, v, i32([0] * n), i32(range(n)), rope_theta=1e4)
    a, b = (x.attention(q, i32([n])) for x in (c, d))
    assert torch.equal(c.k, d.k) and torch.equal(c.v, d.v) and torch.equal(a, b)
    check_attention(c, q, [n], stored(c, [n]))


# ---- the error word -------------------------------------------------------------------

def test_the_error_word_is_clear_before_a_call_on_another_stream():
    """The stream that is current when a cache is made may be busy; a call on another one may come first."""
    from mtp_block_draft_gb300 import DmtpError
    k = torch.zeros((1, 2, 64), dtype=BF, device="cuda")
    seq, pos, table = i32([7]), i32([0]), i32([[0, 1], [2, 3]])
    from mtp_block_draft_gb300 import DmtpPagedCache
    side = torch.cuda.Stream()
    for _ in range(2):                         # (kernels are loaded at their first call, which waits)
        c = DmtpPagedCache.alloc(4, 16, 2, 64, table)
        with torch.cuda.stream(side):
            c.write(k, k, i32([0]), pos)
        c.check()
    torch.cuda._sleep(200_000_000)             # about 0.1 s of the current stream
    c = DmtpPagedCache.alloc(4, 16, 2, 64, table)
    with torch.cuda.stream(side):
        c.write(k, k, seq, pos)                # no such sequence
    with pytest.raises(DmtpError) as e:
        c.check()
    assert e.value.word == 32
    c.check()


def test_check_clears_what_it_reports_and_nothing_else():
    """A call that goes wrong between check()'s reading of the word and its clearing counts for the next."""
    from mtp_block_draft_gb300 import DmtpError
    c = new_cache(2, 2, 16, 2, 64)
    k = torch.zeros((1, 2, 64), dtype=BF, device="cuda")
    bad_pos, bad_seq, at = (i32([0]), i32([32])), i32([7]), i32([0])
    read, late = c.err.item, []

    def item():
        word = read()
        if not late:
            late.append(1)
            c.write(k, k, bad_seq, at)
            c.write(k, k, *bad_pos)
            torch.cuda.synchronize()
        return word

    c.write(k, k, *bad_pos)
    c.err.item = item
    for word in (2, 32):
        with pytest.raises(DmtpError) as e:
            c.check()
        assert e.value.word == word
    c.check()


# ---- norm -----------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [40, 200])
@pytest.mark.parametrize("d", [64, 520, 2048, 4104, 8200])
@pytest.mark.parametrize("xt,yt", [(FP, None), (BF, BF), (FP, BF)])
def test_norm_of_rows_with_infinities_and_nan(rows, d, xt, yt):
    """An infinity makes the row's mean infinite: finite values become 0 and it itself NaN, wherever it
    stands; a NaN (or infinities that cancel in x + y) makes all of the row NaN."""
    from mtp_block_draft_gb300 import add_rmsnorm_e4m3
    r = np.random.RandomState(rows + d)
    x = randn((rows, d), gen(d), xt)
    y = None if yt is None else randn((rows, d), gen(d + 1), yt)
    odd = torch.zeros((rows, d), dtype=torch.bool)
    nan = torch.zeros(rows, dtype=torch.bool)
    for i in range(rows):
        at = i * 8 // rows + 8 * r.randint(0, d // 8) if i % 4 else r.randint(0, d)  # each place of eight
        if i % 5 == 4:
            continue                           # an ordinary row
        odd[i, at] = True
        into = y if y is not None and i % 2 else x
        into[i, at] = float("inf") if i % 3 else -float("inf")
        if i % 5 == 3:
            nan[i] = True
            if y is not None and i % 2 == 0:
                y[i, at] = -x[i, at]           # infinity less infinity
            else:
                x[i, (at + 11) % d] = float("nan")
        elif i % 5 == 2:                       # several of them
            odd[i, ::7] = True
            x[i, ::7] = float("inf")
            if y is not None:
                y[i, ::7] = 1.0
    gain = torch.rand(d, device="cuda", generator=gen(2)) + 0.5
    xo, q, s = add_rmsnorm_e4m3(x, y, gain, 1e-6)
    v, s = q.float().cpu(), s.cpu()
    plain = torch.arange(rows) % 5 == 4
    assert torch.isnan(v[nan]).all()
    rest = ~nan & ~plain
    assert (torch.isnan(v[rest]) == odd[rest]).all()
    assert (v[rest][~odd[rest]] == 0).all() and (s[rest] == 1).all()
    assert torch.isfinite(v[plain]).all() and bool((v[plain] != 0).any())
    one = [add_rmsnorm_e4m3(x[i:i + 1], None if y is None else y[i:i + 1], gain, 1e-6)[1] for i in range(4, rows, 35)]
    for i, t in zip(range(4, rows, 35), one):  # a row is what it is alone
        assert torch.equal(t.view(torch.uint8), q[i:i + 1].view(torch.uint8))
