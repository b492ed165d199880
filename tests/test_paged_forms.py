"""The paged cache's other forms: argument checks on the host (no GPU). Every refused call below is
refused before any CUDA call, so the pointers are plain integers; each starts from a set of valid
arguments and spoils one of them."""
import ctypes as C

import pytest
import torch

from mtp_block_draft_gb300 import DmtpError, DmtpPagedCache, DmtpRope, binding, build
from test_decode_ops import BAD_CACHE, EINVAL, ENOMEM, PTR, cache, lib, query, rows  # noqa: F401

BF, I32 = torch.bfloat16, torch.int32


def rope(**kw):
    r = binding.dmtp_rope()
    v = dict(theta=1e4, factor=8.0, orig_len=4096.0, low=1.0, high=32.0, dims=128, interleaved=0, scaling=3,
             amplitude=1.0)
    v.update(kw)
    for k, x in v.items():
        setattr(r, k, x)
    return r


def scores(**kw):
    s = binding.dmtp_paged_scores()
    s.cap, s.slopes = kw.get("cap", 30.0), kw.get("slopes", PTR)
    return s


def prompt(**kw):
    a = binding.dmtp_paged_prompt()
    v = dict(q=PTR, out=PTR, q_row=4096, q_head=128, o_row=4096, o_head=128, row_start=PTR, kv_len=PTR, first=PTR,
             end=PTR, n_rows=100, n_heads=32, window=0, scale=0.1)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


def e2m1(**kw):
    return cache(**{**dict(e4m3=4, page_stride=4 * 64 * 128 * 9 // 16), **kw})


@pytest.mark.parametrize("bad", BAD_CACHE, ids=str)
def test_every_call_refuses_a_bad_cache(lib, bad):  # noqa: F811
    c = cache(**bad)
    n = C.c_size_t()
    assert lib.dmtp_paged_write_rope(C.byref(c), C.byref(rows(rope_theta=0.0)), C.byref(rope()), None, None) == EINVAL
    assert lib.dmtp_paged_attention_scores(C.byref(c), C.byref(query()), C.byref(scores()), PTR, 1 << 40, None, None) == EINVAL
    assert lib.dmtp_paged_prompt_workspace(C.byref(c), C.byref(prompt()), C.byref(n)) == EINVAL
    assert lib.dmtp_paged_prompt_attention(C.byref(c), C.byref(prompt()), PTR, 1 << 40, None, None) == EINVAL


@pytest.mark.parametrize("bad", [dict(page_stride=4 * 64 * 128 * 9 // 16 - 16), dict(page_stride=4 * 64 * 128 * 9 // 16 + 8),
                                 dict(k_scale=None), dict(v_scale=None), dict(e4m3=3), dict(e4m3=5),
                                 dict(scale_stride=255), dict(head_dim=120)], ids=str)
def test_a_bad_e2m1_cache_is_refused(lib, bad):  # noqa: F811
    c = e2m1(**bad)
    n = C.c_size_t()
    assert lib.dmtp_paged_write(C.byref(c), C.byref(rows()), None, None) == EINVAL
    assert lib.dmtp_paged_read(C.byref(c), PTR, PTR, 5, PTR, PTR, None, None) == EINVAL
    assert lib.dmtp_paged_attention_workspace(C.byref(c), C.byref(query()), C.byref(n)) == EINVAL
    assert lib.dmtp_paged_prompt_workspace(C.byref(c), C.byref(prompt()), C.byref(n)) == EINVAL
    assert lib.dmtp_paged_attention_workspace(C.byref(e2m1()), C.byref(query()), C.byref(n)) == 0


@pytest.mark.parametrize("bad", [dict(dims=0), dict(dims=8), dict(dims=120), dict(dims=144), dict(dims=-16),
                                 dict(interleaved=2), dict(interleaved=-1), dict(scaling=4), dict(scaling=-1),
                                 dict(theta=0.5), dict(theta=float("inf")), dict(theta=float("nan")), dict(theta=1.0),
                                 dict(factor=0.5), dict(factor=float("nan")), dict(factor=float("inf")),
                                 dict(low=0.0), dict(low=32.0), dict(high=float("inf")), dict(low=float("nan")),
                                 dict(orig_len=0.0), dict(orig_len=float("nan")),
                                 dict(amplitude=float("inf")), dict(amplitude=float("nan"))], ids=str)
def test_write_rope_refuses(lib, bad):  # noqa: F811
    for c in (cache(), e2m1()):
        assert lib.dmtp_paged_write_rope(C.byref(c), C.byref(rows(rope_theta=0.0)), C.byref(rope(**bad)), None, None) == EINVAL


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(n_rows=-1),
                                 dict(k=PTR + 4), dict(q_out=None), dict(k_row=510), dict(v_head=126), dict(k_head=124),
                                 dict(qo_head=64), dict(n_heads=0), dict(rope_theta=1e4), dict(rope_theta=-1.0),
                                 dict(seq=PTR + 1), dict(k_row=-512), dict(qo_row=0)], ids=str)
def test_write_rope_refuses_rows(lib, bad):  # noqa: F811
    r = rows(**{**dict(rope_theta=0.0), **bad})
    assert lib.dmtp_paged_write_rope(C.byref(cache()), C.byref(r), C.byref(rope()), None, None) == EINVAL
    assert lib.dmtp_paged_write_rope(C.byref(cache()), None, C.byref(rope()), None, None) == EINVAL
    assert lib.dmtp_paged_write_rope(C.byref(cache()), C.byref(rows(rope_theta=0.0)), C.byref(rope()), PTR + 1, None) == EINVAL
    assert lib.dmtp_paged_write_rope(C.byref(cache()), C.byref(rows(n_rows=0, rope_theta=0.0)), C.byref(rope()), None, None) == 0


@pytest.mark.parametrize("bad", [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-31),
                                 dict(cap=2e30), dict(slopes=PTR + 2)], ids=str)
def test_scores_are_refused(lib, bad):  # noqa: F811
    assert lib.dmtp_paged_attention_scores(C.byref(cache()), C.byref(query()), C.byref(scores(**bad)), PTR, 1 << 40,
                                           None, None) == EINVAL
    assert lib.dmtp_paged_prompt_attention(C.byref(cache()), C.byref(prompt(scores=scores(**bad))), PTR, 1 << 40, None,
                                           None) == EINVAL


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(row_start=None), dict(kv_len=None),
                                 dict(q=PTR + 8), dict(out=PTR + 8), dict(row_start=PTR + 2), dict(first=PTR + 1),
                                 dict(end=PTR + 2), dict(kv_len=PTR + 2), dict(n_rows=-1), dict(n_rows=(1 << 24) + 1),
                                 dict(n_rows=1 << 24, n_heads=256), dict(n_heads=0), dict(n_heads=30),
                                 dict(n_heads=5000), dict(window=-1), dict(scale=float("nan")), dict(scale=2e30),
                                 dict(q_row=4100), dict(q_head=-128), dict(o_row=0), dict(o_head=64)], ids=str)
def test_prompt_attention_refuses(lib, bad):  # noqa: F811
    assert lib.dmtp_paged_prompt_attention(C.byref(cache()), C.byref(prompt(**bad)), PTR, 1 << 40, None, None) == EINVAL


def test_prompt_workspaces(lib):  # noqa: F811
    n, c = C.c_size_t(), cache(max_blocks=512, table_stride=512)
    few = prompt(n_rows=3)
    assert lib.dmtp_paged_prompt_workspace(C.byref(c), C.byref(few), None) == EINVAL
    assert lib.dmtp_paged_prompt_workspace(C.byref(c), None, C.byref(n)) == EINVAL
    assert lib.dmtp_paged_prompt_workspace(C.byref(c), C.byref(few), C.byref(n)) == 0
    assert n.value > 0 and n.value % 256 == 0
    call = lambda w, size: lib.dmtp_paged_prompt_attention(C.byref(c), C.byref(few), w, size, None, None)  # noqa: E731
    assert call(None, 0) == EINVAL and call(PTR + 128, n.value) == EINVAL and call(PTR, n.value - 1) == ENOMEM
    assert lib.dmtp_paged_prompt_attention(C.byref(c), C.byref(few), PTR, n.value, PTR + 2, None) == EINVAL
    assert lib.dmtp_paged_prompt_attention(C.byref(c), C.byref(prompt(n_rows=0)), None, 0, None, None) == 0
    assert lib.dmtp_paged_prompt_workspace(C.byref(cache()), C.byref(prompt(n_rows=20000)), C.byref(n)) == 0
    assert n.value == 0


# ---- the binding ----------------------------------------------------------------------

def new_cache(**kw):
    k = torch.zeros((8, 2, 16, 64), dtype=BF)
    return DmtpPagedCache(**{"k": k, "v": k.clone(), "table": torch.zeros((2, 4), dtype=I32), **kw})


@pytest.mark.parametrize("bad", [3, 0.7, [1, 2, 3], "k"], ids=lambda x: type(x).__name__)
def test_what_is_no_tensor_is_an_argument_error(bad):
    build.build()
    c = new_cache()
    q, ln, st = torch.zeros((5, 4, 64), dtype=BF), torch.zeros(2, dtype=I32), torch.zeros(3, dtype=I32)
    seq, kv = torch.zeros(3, dtype=I32), torch.zeros((3, 2, 64), dtype=BF)
    for i, call in enumerate([lambda: c.prompt_attention(bad, st, ln), lambda: c.prompt_attention(q, bad, ln),
                              lambda: c.prompt_attention(q, st, bad), lambda: c.prompt_attention(q, st, ln, first=bad),
                              lambda: c.prompt_attention(q, st, ln, end=bad), lambda: c.prompt_attention(q, st, ln, slopes=bad),
                              lambda: c.prompt_attention(q, st, ln, out=bad), lambda: c.prompt_attention(q, st, ln, workspace=bad),
                              lambda: c.attention(q[None, :1].expand(2, 1, 4, 64), ln, slopes=bad),
                              lambda: c.write(kv, kv, seq, seq, rope=bad), lambda: DmtpRope(scaling=bad),
                              lambda: DmtpRope(dims=[bad]), lambda: DmtpRope(theta=[bad])]):
        try:
            call()
        except DmtpError as e:
            assert e.code == -1, i
        else:
            pytest.fail(f"call {i} was taken")


def test_shapes_and_numbers_that_do_not_fit():
    build.build()
    c = new_cache()
    q, ln, st = torch.zeros((5, 4, 64), dtype=BF), torch.zeros(2, dtype=I32), torch.zeros(3, dtype=I32)
    n5 = torch.zeros(5, dtype=I32)
    for call in (lambda: c.prompt_attention(q[0], st, ln), lambda: c.prompt_attention(q.float(), st, ln),
                 lambda: c.prompt_attention(q[..., ::2], st, ln), lambda: c.prompt_attention(q, ln, ln),
                 lambda: c.prompt_attention(q, st, st), lambda: c.prompt_attention(q, st.long(), ln),
                 lambda: c.prompt_attention(q, st, ln, first=n5[:4]), lambda: c.prompt_attention(q, st, ln, end=n5.float()),
                 lambda: c.prompt_attention(q, st, ln, slopes=torch.zeros(3)), lambda: c.prompt_attention(q[:, :3], st, ln),
                 lambda: c.prompt_attention(q, st, ln, out=q[:4]), lambda: c.prompt_attention(q, st, ln, cap=-1.0),
                 lambda: c.prompt_attention(q, st, ln, window=1 << 31), lambda: c.prompt_attention(q, st, ln, cap="a"),
                 lambda: c.prompt_attention(q, st, ln, scale=1e39), lambda: c.prompt_workspace(-1, 4),
                 lambda: c.prompt_workspace(5, 3), lambda: DmtpRope(theta="a"), lambda: DmtpRope(dims=1 << 40),
                 lambda: c.prompt_attention(q, st, ln),      # tensors on the host
                 lambda: c.prompt_attention(q.expand(5, 4, 64), st, ln, workspace=torch.zeros(4))):
        with pytest.raises(DmtpError):
            call()


def test_e2m1_caches_of_the_binding():
    build.build()
    t = torch.zeros((2, 4), dtype=I32)
    c = DmtpPagedCache.alloc(8, 16, 2, 64, t, e2m1=True)
    assert c.head_dim == 64 and c.n_kv_heads == 2 and c.c.e4m3 == 4 and c.c.page_stride == 16 * 2 * 36 and c.dtype is BF
    k, s = c.k, c.k_scale
    pool = torch.zeros((8, 2, 16 * 2 * 36), dtype=torch.uint8)       # two layers, page by page
    assert DmtpPagedCache(pool[:, 0], pool[:, 1], t, s, s.clone(), dtype=torch.float32).c.page_stride == 2 * 16 * 2 * 36
    for bad in (dict(k=k[:, :-1]), dict(k=k[:, :-8], v=k[:, :-8]), dict(v=k.float()), dict(k_scale=None), dict(v_scale=None),
                dict(k_scale=s[:4]), dict(k_scale=s.double()), dict(k=k[:, ::2], v=k[:, ::2]), dict(dtype=torch.float16),
                dict(k=k[None], v=k[None]), dict(k=k[0], v=k[0]), dict(k_scale=s[0])):
        with pytest.raises(DmtpError):
            DmtpPagedCache(**{**dict(k=k, v=k.clone(), table=t, k_scale=s, v_scale=s.clone()), **bad})
    for kw in (dict(head_dim=72), dict(e4m3=True)):
        with pytest.raises(DmtpError):
            DmtpPagedCache.alloc(**{**dict(n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, table=t, e2m1=True), **kw})
