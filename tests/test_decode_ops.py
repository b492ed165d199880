"""The decode-step operators of include/dmtp_ops.h: argument checks on the host (no GPU).

Every refused call below is refused before any CUDA call, so the pointers are plain
integers; each starts from a set of valid arguments and spoils one of them."""
import ctypes as C

import pytest
import torch

from mtp_block_draft_gb300 import DmtpError, DmtpPagedCache, binding, build, load_library

EINVAL, ENOMEM = -1, -2
PTR = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return load_library()


def cache(**kw):
    c = binding.dmtp_paged_kv()
    v = dict(k=PTR, v=PTR, k_scale=PTR, v_scale=PTR, table=PTR, page_stride=4 * 64 * 128,
             scale_stride=4 * 64, table_stride=32, n_pages=64, page_size=64, n_kv_heads=4,
             head_dim=128, n_seqs=3, max_blocks=32, dtype=1, e4m3=1)
    v.update(kw)
    for k, x in v.items():
        setattr(c, k, x)
    return c


BAD_CACHE = [dict(k=None), dict(v=None), dict(table=None), dict(k_scale=None), dict(v_scale=None),
             dict(k=PTR + 8), dict(v=PTR + 8), dict(k_scale=PTR + 2), dict(table=PTR + 2),
             dict(page_stride=4 * 64 * 128 - 16), dict(page_stride=4 * 64 * 128 + 8),
             dict(scale_stride=4 * 64 - 1), dict(table_stride=31), dict(n_pages=0),
             dict(page_size=0), dict(page_size=65537, page_stride=1 << 40),
             dict(n_kv_heads=0), dict(n_kv_heads=5000, page_stride=1 << 40, scale_stride=1 << 40),
             dict(head_dim=0), dict(head_dim=8), dict(head_dim=120), dict(head_dim=272, page_stride=1 << 20),
             dict(n_seqs=0), dict(max_blocks=0), dict(max_blocks=1 << 26, table_stride=1 << 26),
             dict(dtype=2), dict(dtype=-1), dict(e4m3=2)]


def rows(**kw):
    r = binding.dmtp_paged_rows()
    v = dict(q=PTR, k=PTR, v=PTR, q_out=PTR, q_row=4096, q_head=128, k_row=512, k_head=128,
             v_row=512, v_head=128, qo_row=4096, qo_head=128, seq=PTR, pos=PTR, n_rows=5,
             n_heads=32, rope_theta=1e4)
    v.update(kw)
    for k, x in v.items():
        setattr(r, k, x)
    return r


def query(**kw):
    a = binding.dmtp_paged_query()
    v = dict(q=PTR, out=PTR, q_seq=4096, q_row=4096, q_head=128, o_seq=4096, o_row=4096,
             o_head=128, kv_len=PTR, rows=1, n_heads=32, window=0, scale=0.1)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


@pytest.mark.parametrize("bad", BAD_CACHE, ids=str)
def test_every_call_refuses_a_bad_cache(lib, bad):
    c = cache(**bad)
    n = C.c_size_t()
    assert lib.dmtp_paged_write(C.byref(c), C.byref(rows()), None, None) == EINVAL
    assert lib.dmtp_paged_read(C.byref(c), PTR, PTR, 5, PTR, PTR, None, None) == EINVAL
    assert lib.dmtp_paged_attention_workspace(C.byref(c), C.byref(query()), C.byref(n)) == EINVAL
    assert lib.dmtp_paged_attention(C.byref(c), C.byref(query()), PTR, 1 << 40, None, None) == EINVAL


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(seq=None), dict(pos=None),
                                 dict(n_rows=-1), dict(k=PTR + 4), dict(v=PTR + 2),
                                 dict(q=PTR + 4), dict(q_out=None), dict(q_out=PTR + 4),
                                 dict(k_row=510), dict(v_head=126), dict(k_head=124),
                                 dict(q_row=4094), dict(qo_head=64), dict(n_heads=0),
                                 dict(n_heads=5000), dict(rope_theta=-1.0),
                                 dict(rope_theta=0.5), dict(rope_theta=float("nan")),
                                 dict(rope_theta=float("inf")), dict(seq=PTR + 1),
                                 dict(k_row=-512)], ids=str)
def test_write_refuses(lib, bad):
    assert lib.dmtp_paged_write(C.byref(cache()), C.byref(rows(**bad)), None, None) == EINVAL


def test_null_structs_and_empty_calls(lib):
    c, n = cache(), C.c_size_t()
    assert lib.dmtp_paged_write(None, C.byref(rows()), None, None) == EINVAL
    assert lib.dmtp_paged_write(C.byref(c), None, None, None) == EINVAL
    assert lib.dmtp_paged_write(C.byref(c), C.byref(rows()), PTR + 1, None) == EINVAL
    assert lib.dmtp_paged_attention_workspace(C.byref(c), C.byref(query()), None) == EINVAL
    assert lib.dmtp_paged_attention_workspace(C.byref(c), None, C.byref(n)) == EINVAL
    assert lib.dmtp_add_rmsnorm_e4m3(None, None) == EINVAL
    assert lib.dmtp_sample_rows(None, None) == EINVAL
    # no rows: nothing to do
    assert lib.dmtp_paged_write(C.byref(c), C.byref(rows(n_rows=0)), None, None) == 0
    assert lib.dmtp_paged_read(C.byref(c), PTR, PTR, 0, PTR, PTR, None, None) == 0
    assert lib.dmtp_add_rmsnorm_e4m3(C.byref(norm(rows=0)), None) == 0
    assert lib.dmtp_sample_rows(C.byref(sample(rows=0)), None) == 0


@pytest.mark.parametrize("args", [(None, PTR, 5, PTR, PTR), (PTR, None, 5, PTR, PTR),
                                  (PTR, PTR, -1, PTR, PTR), (PTR, PTR, 5, None, PTR),
                                  (PTR, PTR, 5, PTR, PTR + 8), (PTR + 2, PTR, 5, PTR, PTR)])
def test_read_refuses(lib, args):
    assert lib.dmtp_paged_read(C.byref(cache()), *args, None, None) == EINVAL


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(kv_len=None), dict(rows=0),
                                 dict(rows=9), dict(n_heads=0), dict(n_heads=30),
                                 dict(window=-1), dict(q=PTR + 8), dict(out=PTR + 4),
                                 dict(kv_len=PTR + 2), dict(q_seq=4100), dict(q_row=4),
                                 dict(q_head=-128), dict(o_head=64), dict(o_row=4),
                                 dict(scale=float("nan")), dict(scale=float("inf"))], ids=str)
def test_attention_refuses(lib, bad):
    assert lib.dmtp_paged_attention(C.byref(cache()), C.byref(query(**bad)), PTR, 1 << 40, None,
                                    None) == EINVAL


def test_attention_workspace(lib):
    c, a, n = cache(), query(), C.c_size_t()
    assert lib.dmtp_paged_attention_workspace(C.byref(c), C.byref(a), C.byref(n)) == 0 and n.value
    assert lib.dmtp_paged_attention(C.byref(c), C.byref(a), PTR, n.value - 1, None, None) == ENOMEM
    assert lib.dmtp_paged_attention(C.byref(c), C.byref(a), None, n.value, None, None) == EINVAL
    assert lib.dmtp_paged_attention(C.byref(c), C.byref(a), PTR + 64, n.value, None, None) == EINVAL
    # tiles past 2^31 are refused
    big = cache(n_seqs=60000, max_blocks=1 << 20, table_stride=1 << 20, n_kv_heads=64,
                page_stride=1 << 30, scale_stride=1 << 30)
    assert lib.dmtp_paged_attention_workspace(C.byref(big), C.byref(query(n_heads=64)),
                                              C.byref(n)) == EINVAL


def norm(**kw):
    a = binding.dmtp_norm_args()
    v = dict(x=PTR, y=PTR, gain=PTR, x_out=PTR, q=PTR, scale=PTR, x_row=2048, y_row=2048,
             xo_row=2048, q_row=2048, rows=3, d=2048, x_dtype=0, y_dtype=1, gain_dtype=1, eps=1e-6)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


@pytest.mark.parametrize("bad", [dict(x=None), dict(gain=None), dict(q=None), dict(scale=None),
                                 dict(x_out=None), dict(rows=-1), dict(d=0), dict(d=2044),
                                 dict(d=16392), dict(x_dtype=2), dict(y_dtype=-1),
                                 dict(gain_dtype=2), dict(x=PTR + 8), dict(y=PTR + 8),
                                 dict(x_out=PTR + 8), dict(q=PTR + 4), dict(gain=PTR + 2),
                                 dict(x_row=2040), dict(x_row=2052), dict(y_row=2047),
                                 dict(xo_row=2049), dict(q_row=2040), dict(eps=-1.0),
                                 dict(eps=float("nan"))], ids=str)
def test_norm_refuses(lib, bad):
    assert lib.dmtp_add_rmsnorm_e4m3(C.byref(norm(**bad)), None) == EINVAL


def sample(**kw):
    a = binding.dmtp_sample_args()
    v = dict(logits=PTR, ld=1000, rows=2, vocab=1000, dtype=0, u=PTR, ids=PTR)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


@pytest.mark.parametrize("bad", [dict(logits=None), dict(u=None), dict(ids=None), dict(ld=999),
                                 dict(rows=-1), dict(vocab=0), dict(vocab=262145, ld=262145),
                                 dict(dtype=2), dict(logits=PTR + 2), dict(u=PTR + 1),
                                 dict(top_k=PTR + 2), dict(kept=PTR + 3),
                                 dict(rows=(1 << 24) + 1)], ids=str)
def test_sample_refuses(lib, bad):
    assert lib.dmtp_sample_rows(C.byref(sample(**bad)), None) == EINVAL


def test_output_rows_of_one_address_are_refused(lib):
    for bad in (dict(o_row=0, rows=2), dict(o_seq=0)):
        assert lib.dmtp_paged_attention(C.byref(cache()), C.byref(query(**bad)), PTR, 1 << 40, None,
                                        None) == EINVAL
    assert lib.dmtp_paged_write(C.byref(cache()), C.byref(rows(qo_row=0)), None, None) == EINVAL


def test_binding_refuses_numbers_and_shapes_that_do_not_fit(lib):
    from mtp_block_draft_gb300 import add_rmsnorm_e4m3, sample_rows
    table = torch.zeros((2, 4), dtype=torch.int32)
    k = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16)
    c = DmtpPagedCache(k, k, table)
    seq = torch.zeros(3, dtype=torch.int32)
    kv, q = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    x = torch.zeros((2, 64))
    for call in (lambda: c.attention(q, seq[:2], window=1 << 31), lambda: c.attention(q, seq[:2], scale=1e39),
                 lambda: c.attention(q[0], seq[:2]), lambda: c.attention(q, seq[:2], out=q[0]),
                 lambda: c.write(kv, kv, seq, seq, rope_theta=1e39), lambda: c.write(kv[0], kv, seq, seq),
                 lambda: c.write(kv, kv, seq, seq, q=kv[0]), lambda: c.write(kv[:2], kv, seq, seq),
                 lambda: c.attention_workspace(0, 4), lambda: c.attention_workspace(1 << 40, 4),
                 lambda: add_rmsnorm_e4m3(x, None, torch.ones(64), eps=1e39),
                 lambda: add_rmsnorm_e4m3(x, x[0], torch.ones(64)), lambda: add_rmsnorm_e4m3(x[0], x[0], x[0]),
                 lambda: sample_rows(x[0], x[0, :1]), lambda: sample_rows(x, x[0])):
        with pytest.raises(DmtpError):
            call()


def test_binding_refuses_tensors_of_the_wrong_kind(lib):
    table = torch.zeros((2, 4), dtype=torch.int32)
    k = torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16)
    for bad in (dict(v=k.float()), dict(v=k[:, :, :8]), dict(table=table.long()),
                dict(k_scale=torch.ones(8, 2, 16)), dict(dtype=torch.float32)):
        kw = dict(k=k, v=k, table=table)
        kw.update(bad)
        with pytest.raises(DmtpError):
            DmtpPagedCache(**kw)
    q8 = torch.zeros((8, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(DmtpError):
        DmtpPagedCache(q8, q8, table)
    t = k.transpose(1, 2)
    with pytest.raises(DmtpError):
        DmtpPagedCache(t, t, table)
    # tensors on the host are refused by every call, not dereferenced by a kernel
    c = DmtpPagedCache(k, k, table)
    seq = torch.zeros(3, dtype=torch.int32)
    kv = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    for call in (lambda: c.write(kv, kv, seq, seq), lambda: c.read(seq, seq),
                 lambda: c.attention(q, seq[:2]), lambda: c.write(kv.float(), kv, seq, seq),
                 lambda: c.write(kv, kv, seq.long(), seq), lambda: c.attention(q[:1], seq[:1]),
                 lambda: c.attention(q.float(), seq[:2]), lambda: c.read(seq[::2], seq)):
        with pytest.raises(DmtpError):
            call()
