"""The decode-step operators' binding on the host: what is refused, what is taken (no GPU)."""
import numpy as np
import pytest
import torch

from mtp_block_draft_gb300 import DmtpError, DmtpPagedCache, add_rmsnorm_e4m3, build, sample_rows

BF, FP, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


def new_cache(**kw):
    k = torch.zeros((8, 2, 16, 64), dtype=BF)
    return DmtpPagedCache(**{"k": k, "v": k.clone(), "table": torch.zeros((2, 4), dtype=I32), **kw})


NO_TENSORS = [None, 3, 0.7, [1, 2, 3], "k", np.zeros(3, np.float32)]


@pytest.mark.parametrize("bad", NO_TENSORS, ids=lambda x: type(x).__name__)
def test_what_is_no_tensor_is_an_argument_error(bad):
    """Every argument that is to be a tensor, given as something else (None where it may not be)."""
    c = new_cache()
    seq, kv = torch.zeros(3, dtype=I32), torch.zeros((3, 2, 64), dtype=BF)
    q, ln = torch.zeros((2, 1, 4, 64), dtype=BF), torch.zeros(2, dtype=I32)
    x, g, z, u = torch.zeros((2, 64)), torch.ones(64), torch.zeros((2, 9)), torch.zeros(2)
    k = c.k
    calls = [lambda: c.write(bad, kv, seq, seq), lambda: c.write(kv, bad, seq, seq), lambda: c.write(kv, kv, bad, seq),
             lambda: c.write(kv, kv, seq, bad), lambda: c.read(bad, seq), lambda: c.read(seq, bad),
             lambda: c.attention(bad, ln), lambda: c.attention(q, bad),
             lambda: add_rmsnorm_e4m3(bad, None, g), lambda: add_rmsnorm_e4m3(x, None, bad),
             lambda: sample_rows(bad, u), lambda: sample_rows(z, bad),
             lambda: DmtpPagedCache(bad, k, c.table), lambda: DmtpPagedCache(k, bad, c.table),
             lambda: DmtpPagedCache(k, k, bad), lambda: DmtpPagedCache.alloc(8, 16, 2, 64, bad)]
    if bad is not None:
        calls += [lambda: c.write(kv, kv, seq, seq, q=bad), lambda: c.write(kv, kv, seq, seq, q=kv, q_out=bad),
                  lambda: c.read(seq, seq, k_out=bad), lambda: c.read(seq, seq, v_out=bad),
                  lambda: c.attention(q, ln, out=bad), lambda: c.attention(q, ln, workspace=bad),
                  lambda: add_rmsnorm_e4m3(x, bad, g), lambda: add_rmsnorm_e4m3(x, None, g, x_out=bad),
                  lambda: add_rmsnorm_e4m3(x, None, g, q=bad), lambda: add_rmsnorm_e4m3(x, None, g, scale=bad),
                  lambda: new_cache(k_scale=bad), lambda: new_cache(v_scale=bad)]
        calls += [lambda n=n: sample_rows(z, u, **{n: bad})
                  for n in ("temperature", "top_k", "top_p", "min_p", "ids", "kept")]
    for i, call in enumerate(calls):
        try:
            call()
        except DmtpError as e:
            assert e.code == -1, i
        else:
            pytest.fail(f"call {i} was taken")


def test_tensors_of_other_ranks_are_argument_errors():
    c = new_cache()
    kv, one = torch.zeros((1, 2, 64), dtype=BF), torch.zeros((), dtype=I32)
    for call in (lambda: c.write(kv, kv, one, one), lambda: c.read(one, one), lambda: c.read(one[None, None], one),
                 lambda: sample_rows(torch.zeros(()), torch.zeros(())), lambda: add_rmsnorm_e4m3(one, None, one)):
        with pytest.raises(DmtpError):
            call()


def single_dimensions():
    """Dense pages whose dimensions of one element have strides of their own."""
    one_head = torch.zeros((8, 16, 1, 64), dtype=BF).transpose(1, 2)
    one_row = torch.zeros((8, 1, 4, 64), dtype=BF).transpose(1, 2)
    big = torch.zeros((3, 2, 16, 64), dtype=BF)
    return [(one_head, one_head.contiguous()), (one_head.contiguous(), one_head), (one_row, one_row.clone()),
            (big[:1], big.clone()[::2][:1])]


@pytest.mark.parametrize("i", range(4))
def test_strides_of_single_elements_do_not_count(i):
    k, v = single_dimensions()[i]
    c = DmtpPagedCache(k, v, torch.zeros((1, 2), dtype=I32))
    n, h, ps, hd = k.shape
    assert c.c.page_stride == (k.stride(0) if n > 1 else h * ps * hd)
    k8, v8 = (t.to(FP).to(torch.float8_e4m3fn).as_strided(t.shape, t.stride()) for t in (k.contiguous(), v.contiguous()))
    ks = torch.ones((n, ps, h)).transpose(1, 2) if h == 1 else torch.ones((n, h, ps))
    DmtpPagedCache(k8, v8, torch.zeros((1, 2), dtype=I32), ks, torch.ones((n, h, ps)))


def test_pages_that_are_not_dense_or_differ_are_refused():
    t = torch.zeros((1, 2), dtype=I32)
    k = torch.zeros((8, 4, 16, 64), dtype=BF)
    wide = torch.zeros((8, 4, 16, 128), dtype=BF)
    for a, b in ((k[:, :, ::2], k[:, :, ::2]), (wide[..., :64], wide[..., :64]), (k[:, ::2], k[:, ::2]),
                 (k[::2], k[:4]), (k[:, :2], k[:, :2].contiguous())):
        with pytest.raises(DmtpError):
            DmtpPagedCache(a, b, t)
    DmtpPagedCache(k[:, :2], k[:, 2:], t)      # two layers of a pool, page by page
