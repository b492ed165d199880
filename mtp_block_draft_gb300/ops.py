"""Binding of the decode-step operators of include/dmtp_ops.h on PyTorch tensors.

Argument checks and marshalling only: every call enqueues the library's kernels on the
current stream of the tensors' device. Argument errors raise DmtpError(DMTP_EINVAL) before
anything is launched; what only the device can see (an index out of range) is collected in
the cache's error word, which check() reads.
"""
from __future__ import annotations

import ctypes as C

from .binding import (DmtpError, _check, dmtp_norm_args, dmtp_paged_kv, dmtp_paged_query,
                      dmtp_paged_rows, dmtp_sample_args, load_library)

_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _need(ok, what: str):
    if not ok:
        raise DmtpError(-1, what)


def _dtype(t) -> int:
    """dtype code of a float tensor: 0 fp32, 1 bf16."""
    torch = _t()
    if t.dtype is torch.bfloat16:
        return 1
    _need(t.dtype is torch.float32, f"dtype {t.dtype}")
    return 0


class _on:
    """The stream handle of the current stream of `device`, with `device` current."""

    def __init__(self, device):
        torch = _t()
        _need(device.type == "cuda", "tensors must be on a CUDA device")
        self.index = device.index if device.index is not None else torch.cuda.current_device()

    def __enter__(self):
        torch = _t()
        self.prev = torch.cuda.current_device()
        if self.prev != self.index:
            torch.cuda.set_device(self.index)
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.prev != self.index:
            _t().cuda.set_device(self.prev)
        return False


def _same_device(device, *tensors):
    for t in tensors:
        _need(t is None or t.device == device, "tensors on different devices")


def _int32(t, n: int, what: str):
    _need(t.dtype is _t().int32 and t.dim() == 1 and t.shape[0] == n and
          (n <= 1 or t.stride(0) == 1), f"{what}: a dense int32 tensor of {n} is wanted")


class DmtpPagedCache:
    """A paged K/V cache of one layer over the caller's tensors.

    k, v: [n_pages, n_kv_heads, page_size, head_dim], bf16 or fp32, or float8_e4m3fn with
    k_scale and v_scale [n_pages, n_kv_heads, page_size] fp32; the pages may be strided (a
    pool that holds several layers), the rest is dense. table: int32 [n_seqs, max_blocks],
    the page of each block of each sequence. dtype: the type of the rows given and returned
    (bf16 or fp32; of a cache that is not E4M3, its own). The tensors may be updated between
    calls; they are the ones given here, not copies."""

    def __init__(self, k, v, table, k_scale=None, v_scale=None, dtype=None):
        torch = _t()
        e8 = k.dtype is torch.float8_e4m3fn
        _need(k.dim() == 4 and v.shape == k.shape and v.dtype is k.dtype and
              v.stride() == k.stride(), "k and v: the same 4-d shape, strides and dtype")
        n, h, ps, hd = k.shape
        _need(k.stride()[1:] == (ps * hd, hd, 1), "pages must be dense")
        if e8:
            self.dtype = torch.bfloat16 if dtype is None else dtype
            _need(k_scale is not None and v_scale is not None, "an E4M3 cache has scales")
            for s in (k_scale, v_scale):
                _need(s.shape == (n, h, ps) and s.dtype is torch.float32 and
                      s.stride()[1:] == (ps, 1) and s.stride(0) == k_scale.stride(0),
                      "scales: fp32 [n_pages, n_kv_heads, page_size], pages dense")
        else:
            self.dtype = k.dtype
            _need(k_scale is None and v_scale is None, "scales are of an E4M3 cache")
            _need(dtype is None or dtype is k.dtype, "rows have the cache's own dtype")
        _need(self.dtype in (torch.bfloat16, torch.float32), f"dtype {self.dtype}")
        _need(table.dtype is torch.int32 and table.dim() == 2 and
              (table.shape[1] <= 1 or table.stride(1) == 1), "table: int32 [n_seqs, max_blocks]")
        _same_device(k.device, v, table, k_scale, v_scale)
        self.lib = load_library()
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.device = k.device
        self.n_kv_heads, self.head_dim = h, hd
        self.n_seqs, self.max_blocks = table.shape
        c = self.c = dmtp_paged_kv()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        if e8:
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.scale_stride = k_scale.stride(0) if n > 1 else h * ps
        c.table = table.data_ptr()
        c.page_stride = k.stride(0) if n > 1 else h * ps * hd
        c.table_stride = table.stride(0) if self.n_seqs > 1 else self.max_blocks
        c.n_pages, c.page_size, c.n_kv_heads, c.head_dim = n, ps, h, hd
        c.n_seqs, c.max_blocks = self.n_seqs, self.max_blocks
        c.dtype, c.e4m3 = int(self.dtype is torch.bfloat16), int(e8)
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._err = self.err.data_ptr()
        self._c = C.byref(c)
        self._ws_bytes = {}

    @classmethod
    def alloc(cls, n_pages, page_size, n_kv_heads, head_dim, table, dtype=None, e4m3=False):
        """A cache of its own zeroed pages on the table's device."""
        torch = _t()
        dtype = torch.bfloat16 if dtype is None else dtype
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        kw = {"device": table.device}
        if not e4m3:
            return cls(torch.zeros(shape, dtype=dtype, **kw), torch.zeros(shape, dtype=dtype, **kw),
                       table)
        k, v = (torch.zeros(shape, dtype=torch.uint8, **kw).view(torch.float8_e4m3fn)
                for _ in range(2))
        ks, vs = (torch.ones(shape[:3], dtype=torch.float32, **kw) for _ in range(2))
        return cls(k, v, table, ks, vs, dtype=dtype)

    def _rows(self, t, n, heads, what):
        _need(t.dtype is self.dtype and t.dim() == 3 and t.shape[0] == n and
              t.shape[2] == self.head_dim and (heads is None or t.shape[1] == heads) and
              t.stride(2) == 1 and t.device == self.device,
              f"{what}: [{n}, heads, {self.head_dim}] of the cache's dtype and device")
        s0, s1, _ = t.stride()
        return s0, (s1 if t.shape[1] > 1 else self.head_dim)

    def write(self, k, v, seq, pos, q=None, q_out=None, rope_theta: float = 0.0):
        """dmtp_paged_write: rows k, v [n, n_kv_heads, head_dim] to positions pos of
        sequences seq (int32 [n]; seq < 0: skipped), rotated first if rope_theta > 0. With q
        [n, n_heads, head_dim] returns the rotated queries (q_out, or a new tensor)."""
        n = k.shape[0]
        r = dmtp_paged_rows()
        r.k_row, r.k_head = self._rows(k, n, self.n_kv_heads, "k")
        r.v_row, r.v_head = self._rows(v, n, self.n_kv_heads, "v")
        _int32(seq, n, "seq")
        _int32(pos, n, "pos")
        r.k, r.v, r.seq, r.pos = k.data_ptr(), v.data_ptr(), seq.data_ptr(), pos.data_ptr()
        r.n_rows = n
        r.rope_theta = rope_theta
        if q is not None:
            r.n_heads = q.shape[1]
            r.q_row, r.q_head = self._rows(q, n, None, "q")
            if q_out is None:
                q_out = _t().empty(q.shape, dtype=q.dtype, device=q.device)
            r.qo_row, r.qo_head = self._rows(q_out, n, q.shape[1], "q_out")
            r.q, r.q_out = q.data_ptr(), q_out.data_ptr()
        _same_device(self.device, seq, pos)
        with _on(self.device) as st:
            _check(self.lib.dmtp_paged_write(self._c, C.byref(r), self._err, st),
                   "dmtp_paged_write")
        return q_out

    def read(self, seq, pos, k_out=None, v_out=None):
        """dmtp_paged_read: positions pos of sequences seq (int32 [n]) as dense rows
        [n, n_kv_heads, head_dim]; returns (k, v)."""
        n = seq.shape[0]
        shape = (n, self.n_kv_heads, self.head_dim)
        k_out, v_out = (_t().empty(shape, dtype=self.dtype, device=self.device) if t is None else t
                        for t in (k_out, v_out))
        _int32(seq, n, "seq")
        _int32(pos, n, "pos")
        for t in (k_out, v_out):
            _need(t.shape == shape and t.dtype is self.dtype and t.is_contiguous(),
                  f"k_out, v_out: dense {shape} of the cache's dtype")
        _same_device(self.device, seq, pos, k_out, v_out)
        with _on(self.device) as st:
            _check(self.lib.dmtp_paged_read(self._c, seq.data_ptr(), pos.data_ptr(), n,
                                            k_out.data_ptr(), v_out.data_ptr(), self._err, st),
                   "dmtp_paged_read")
        return k_out, v_out

    def attention(self, q, kv_len, scale=None, window: int = 0, out=None, workspace=None):
        """dmtp_paged_attention: q [n_seqs, rows, n_heads, head_dim], the newest rows of each
        sequence; kv_len int32 [n_seqs], its length with them. scale: 1/sqrt(head_dim) if
        None; window > 0: a row sees that many positions. workspace: a uint8 tensor of
        attention_workspace() bytes that no overlapping call uses; None: taken from PyTorch's
        allocator for this call."""
        torch = _t()
        B, rows, heads, hd = q.shape
        _need(B == self.n_seqs and hd == self.head_dim and q.dtype is self.dtype,
              f"q: [{self.n_seqs}, rows, n_heads, {self.head_dim}] of the cache's dtype")
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _need(out.shape == q.shape and out.dtype is q.dtype, "out: the shape and dtype of q")
        _int32(kv_len, B, "kv_len")
        a = dmtp_paged_query()
        a.q, a.out, a.kv_len = q.data_ptr(), out.data_ptr(), kv_len.data_ptr()
        _need(q.stride(3) == 1 and out.stride(3) == 1, "head_dim must be dense")
        # (the stride of a dimension of one element says nothing)
        a.q_seq, a.q_row, a.q_head = (s if d > 1 else hd for s, d in zip(q.stride(), q.shape[:3]))
        a.o_seq, a.o_row, a.o_head = (s if d > 1 else hd for s, d in zip(out.stride(), q.shape[:3]))
        a.rows, a.n_heads, a.window = rows, heads, window
        a.scale = hd ** -0.5 if scale is None else scale
        _same_device(self.device, q, out, kv_len, workspace)
        key = (rows, heads)
        n = self._ws_bytes.get(key)
        if n is None:
            size = C.c_size_t()
            _check(self.lib.dmtp_paged_attention_workspace(self._c, C.byref(a), C.byref(size)),
                   "dmtp_paged_attention_workspace")
            n = self._ws_bytes[key] = size.value
        with _on(self.device) as st:
            if workspace is None:
                workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
            _check(self.lib.dmtp_paged_attention(self._c, C.byref(a), workspace.data_ptr(),
                                                 workspace.numel(), self._err, st),
                   "dmtp_paged_attention")
        return out

    def attention_workspace(self, rows: int, n_heads: int) -> int:
        """Bytes of workspace that attention() needs for q of these rows and heads."""
        a = dmtp_paged_query()
        a.rows, a.n_heads, a.scale = rows, n_heads, 1.0
        size = C.c_size_t()
        _check(self.lib.dmtp_paged_attention_workspace(self._c, C.byref(a), C.byref(size)),
               "dmtp_paged_attention_workspace")
        return size.value

    def check(self):
        """Wait for the device and raise DmtpError(DMTP_EDEVICE) if any call since the last
        check met an index out of range; the word is then cleared."""
        word = int(self.err.item())
        if word:
            self.err.zero_()
            raise DmtpError(-5, "paged cache", word)


def add_rmsnorm_e4m3(x, y, gain, eps: float = 1e-6, x_out=None, q=None, scale=None):
    """dmtp_add_rmsnorm_e4m3: x_out = x + y, and E4M3 rows of RMSNorm(x + y) * gain. x, y
    [rows, d] bf16 or fp32 (y None: no addition); x_out may be x (None: a new tensor, or x
    where y is None). Returns (x_out, q float8_e4m3fn [rows, d], scale fp32 [rows])."""
    torch = _t()
    _need(x.dim() == 2 and x.stride(1) == 1, "x: [rows, d], dense rows")
    rows, d = x.shape
    a = dmtp_norm_args()
    a.rows, a.d, a.eps = rows, d, eps
    a.x, a.x_dtype = x.data_ptr(), _dtype(x)
    a.x_row = x.stride(0) if rows > 1 else d
    if y is not None:
        _need(y.shape == x.shape and y.stride(1) == 1, "y: the shape of x, dense rows")
        a.y, a.y_dtype = y.data_ptr(), _dtype(y)
        a.y_row = y.stride(0) if rows > 1 else d
        if x_out is None:
            x_out = torch.empty((rows, d), dtype=x.dtype, device=x.device)
    if x_out is not None:
        _need(x_out.shape == x.shape and x_out.dtype is x.dtype and x_out.stride(1) == 1,
              "x_out: the shape and dtype of x, dense rows")
        a.x_out = x_out.data_ptr()
        a.xo_row = x_out.stride(0) if rows > 1 else d
    if q is None:
        q = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    _need(q.shape == x.shape and q.dtype is torch.float8_e4m3fn and q.stride(1) == 1,
          "q: float8_e4m3fn of the shape of x, dense rows")
    _need(scale.shape == (rows,) and scale.dtype is torch.float32 and
          (rows <= 1 or scale.stride(0) == 1), "scale: dense fp32 [rows]")
    _need(gain.shape == (d,) and (d <= 1 or gain.stride(0) == 1), "gain: dense [d]")
    _same_device(x.device, y, gain, x_out, q, scale)
    a.gain, a.gain_dtype = gain.data_ptr(), _dtype(gain)
    a.q, a.q_row = q.data_ptr(), q.stride(0) if rows > 1 else d
    a.scale = scale.data_ptr()
    with _on(x.device) as st:
        _check(load_library().dmtp_add_rmsnorm_e4m3(C.byref(a), st), "dmtp_add_rmsnorm_e4m3")
    return (x if x_out is None else x_out), q, scale


def sample_rows(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, ids=None,
                kept=None):
    """dmtp_sample_rows: one token id per row of logits [rows, vocab] (bf16 or fp32), drawn
    with the uniform numbers u (fp32 [rows]) under temperature, top_k (int32), top_p and
    min_p (fp32 [rows] each, None: off). Returns ids (int32 [rows]; -1 where nothing may be
    chosen); kept (int32 [rows], optional) receives how many tokens passed the filters."""
    torch = _t()
    _need(logits.dim() == 2 and (logits.shape[1] <= 1 or logits.stride(1) == 1),
          "logits: [rows, vocab], dense rows")
    rows, V = logits.shape
    if ids is None:
        ids = torch.empty(rows, dtype=torch.int32, device=logits.device)
    a = dmtp_sample_args()
    a.logits, a.dtype, a.rows, a.vocab = logits.data_ptr(), _dtype(logits), rows, V
    a.ld = logits.stride(0) if rows > 1 else V
    for name, t, dt in (("u", u, torch.float32), ("temperature", temperature, torch.float32),
                        ("top_k", top_k, torch.int32), ("top_p", top_p, torch.float32),
                        ("min_p", min_p, torch.float32), ("ids", ids, torch.int32),
                        ("kept", kept, torch.int32)):
        if t is None:
            continue
        _need(t.dtype is dt and t.shape == (rows,) and (rows <= 1 or t.stride(0) == 1),
              f"{name}: dense {dt} [rows]")
        setattr(a, name, t.data_ptr())
    _same_device(logits.device, u, temperature, top_k, top_p, min_p, ids, kept)
    with _on(logits.device) as st:
        _check(load_library().dmtp_sample_rows(C.byref(a), st), "dmtp_sample_rows")
    return ids
