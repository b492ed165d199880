"""Binding of the decode-step operators of include/dmtp_ops.h on PyTorch tensors.

Argument checks and marshalling only: every call enqueues the library's kernels on the
current stream of the tensors' device. Argument errors raise DmtpError(DMTP_EINVAL) before
anything is launched; what only the device can see (an index out of range) is collected in
the cache's error word, which check() reads. The operators are for inference: results carry no
gradient, whatever the inputs require.
"""
from __future__ import annotations

import ctypes as C
import struct
import threading

from .binding import (DmtpError, _check, dmtp_norm_args, dmtp_paged_kv, dmtp_paged_query,
                      dmtp_paged_rows, dmtp_sample_args, load_library)

# The argument structs as bytes: one pack() is several times quicker than setting a ctypes
# struct's fields, and a decode step makes these calls once per layer.
_ROWS = struct.Struct("@4P8q2P2if4x")
_QUERY = struct.Struct("@2P6qP3if")
_NORM = struct.Struct("@6P4q5if")
_SAMPLE = struct.Struct("@Pq3i4x7P")
for _s, _c in ((_ROWS, dmtp_paged_rows), (_QUERY, dmtp_paged_query), (_NORM, dmtp_norm_args),
               (_SAMPLE, dmtp_sample_args)):
    assert _s.size == C.sizeof(_c)


class _Calls:
    """The library's entry points taking packed arguments, and what they need of torch."""

    def __init__(self):
        import torch
        lib = load_library()
        P, B = C.c_void_p, C.c_char_p
        for name, args in (("dmtp_paged_write", [B, B, P, P]),
                           ("dmtp_paged_read", [B, P, P, C.c_int, P, P, P, P]),
                           ("dmtp_paged_attention_workspace", [B, B, P]),
                           ("dmtp_paged_attention", [B, B, P, C.c_size_t, P, P]),
                           ("dmtp_add_rmsnorm_e4m3", [B, P]), ("dmtp_sample_rows", [B, P])):
            f = lib[name]  # a function object of its own: the ctypes prototypes stay as they are
            f.argtypes, f.restype = args, C.c_int
            setattr(self, name[5:], f)
        self.torch = torch
        self.bf16, self.fp32, self.int32 = torch.bfloat16, torch.float32, torch.int32
        self.f8 = torch.float8_e4m3fn
        self.stream = torch._C._cuda_getCurrentRawStream
        self.device = torch._C._cuda_getDevice


# What the checks below run into with an argument that is no tensor, or has too few dimensions.
_NO_TENSOR = (AttributeError, IndexError, TypeError)

_calls = None


def _c() -> _Calls:
    global _calls
    if _calls is None:
        _calls = _Calls()
    return _calls


def _bad(what: str):
    raise DmtpError(-1, what)


def _pack(s, *args) -> bytes:
    """The packed struct; a number that its field cannot hold is an argument error."""
    try:
        return s.pack(*args)
    except (struct.error, OverflowError) as e:
        _bad(str(e))


def _dtype(c, t) -> int:
    """dtype code of a float tensor: 0 fp32, 1 bf16."""
    d = getattr(t, "dtype", type(t))
    if d is c.bf16:
        return 1
    if d is not c.fp32:
        _bad(f"dtype {d}")
    return 0


def _vector(t, dtype, n: int, dev: int, what: str) -> int:
    """Address of a dense vector of n elements."""
    try:
        if t.dtype is dtype and t.shape == (n,) and t.get_device() == dev and (
                n <= 1 or t.stride() == (1,)):
            return t.data_ptr()
    except _NO_TENSOR:
        pass
    _bad(f"{what}: a dense {dtype} tensor of {n} on the same device is wanted")


def _run(c, f, dev: int, what: str, *args):
    """f(*args, stream) on the current stream of CUDA device dev, with dev current."""
    if dev < 0:
        _bad("tensors must be on a CUDA device")
    if c.device() == dev:
        r = f(*args, c.stream(dev))
    else:
        with c.torch.cuda.device(dev):
            r = f(*args, c.stream(dev))
    if r:
        raise DmtpError(r, what)


def _dense_pages(t) -> bool:
    """All but the first dimension dense (the stride of a dimension of one element says nothing)."""
    want = 1
    for size, stride in zip(t.shape[:0:-1], t.stride()[:0:-1]):
        if size > 1 and stride != want:
            return False
        want *= size
    return True


class DmtpPagedCache:
    """A paged K/V cache of one layer over the caller's tensors.

    k, v: [n_pages, n_kv_heads, page_size, head_dim], bf16 or fp32, or float8_e4m3fn with
    k_scale and v_scale [n_pages, n_kv_heads, page_size] fp32; the pages may be strided (a
    pool that holds several layers), k's and v's alike, the rest is dense. table: int32
    [n_seqs, max_blocks], the page of each block of each sequence. dtype: the type of the rows
    given and returned (bf16 or fp32; of a cache that is not E4M3, its own). The tensors may be
    updated between calls; they are the ones given here, not copies. A cache is made outside
    stream captures; its calls may come from any stream and thread."""

    def __init__(self, k, v, table, k_scale=None, v_scale=None, dtype=None):
        c = _c()
        torch = c.torch

        def need(ok, what):
            if not ok:
                _bad(what)

        need(all(isinstance(t, torch.Tensor) for t in (k, v, table)) and
             all(t is None or isinstance(t, torch.Tensor) for t in (k_scale, v_scale)),
             "k, v, table and scales are tensors")
        e8 = k.dtype is c.f8
        need(k.dim() == 4 and v.shape == k.shape and v.dtype is k.dtype,
             "k and v: the same 4-d shape and dtype")
        n, h, ps, hd = k.shape
        need(_dense_pages(k) and _dense_pages(v) and (n <= 1 or v.stride(0) == k.stride(0)),
             "pages must be dense, and k's and v's as far apart")
        if e8:
            self.dtype = c.bf16 if dtype is None else dtype
            need(k_scale is not None and v_scale is not None, "an E4M3 cache has scales")
            for s in (k_scale, v_scale):
                need(s.shape == (n, h, ps) and s.dtype is c.fp32 and
                     _dense_pages(s) and (n <= 1 or s.stride(0) == k_scale.stride(0)),
                     "scales: fp32 [n_pages, n_kv_heads, page_size], pages dense")
        else:
            self.dtype = k.dtype
            need(k_scale is None and v_scale is None, "scales are of an E4M3 cache")
            need(dtype is None or dtype is k.dtype, "rows have the cache's own dtype")
        need(self.dtype in (c.bf16, c.fp32), f"dtype {self.dtype}")
        need(table.dtype is c.int32 and table.dim() == 2 and
             (table.shape[1] <= 1 or table.stride(1) == 1), "table: int32 [n_seqs, max_blocks]")
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.device = k.device
        self._dev = k.get_device()
        need(all(t is None or t.get_device() == self._dev for t in (v, table, k_scale, v_scale)),
             "tensors on different devices")
        self.n_kv_heads, self.head_dim = h, hd
        self.n_seqs, self.max_blocks = table.shape
        p = self.c = dmtp_paged_kv()
        p.k, p.v = k.data_ptr(), v.data_ptr()
        if e8:
            p.k_scale, p.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            p.scale_stride = k_scale.stride(0) if n > 1 else h * ps
        p.table = table.data_ptr()
        p.page_stride = k.stride(0) if n > 1 else h * ps * hd
        p.table_stride = table.stride(0) if self.n_seqs > 1 else self.max_blocks
        p.n_pages, p.page_size, p.n_kv_heads, p.head_dim = n, ps, h, hd
        p.n_seqs, p.max_blocks = self.n_seqs, self.max_blocks
        p.dtype, p.e4m3 = int(self.dtype is c.bf16), int(e8)
        self.err = torch.zeros(1, dtype=c.int32, device=k.device)
        if self._dev >= 0 and not torch.cuda.is_current_stream_capturing():
            # calls may come on any stream: the word is 0 before the first of them sets a bit
            torch.cuda.current_stream(k.device).synchronize()
        self._lock = threading.Lock()
        self._word = torch.zeros(1, dtype=torch.int64, device=k.device)  # index of the word in err
        self._err = self.err.data_ptr()
        self._c = bytes(p)
        self._scale = hd ** -0.5
        self._ws_bytes = {}

    @classmethod
    def alloc(cls, n_pages, page_size, n_kv_heads, head_dim, table, dtype=None, e4m3=False):
        """A cache of its own zeroed pages on the table's device."""
        torch = _c().torch
        if not isinstance(table, torch.Tensor):
            _bad("table: int32 [n_seqs, max_blocks]")
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
        """Row and head strides of t [n, heads, head_dim]."""
        try:
            if t.dtype is self.dtype and t.shape == (n, heads, self.head_dim) and \
                    t.get_device() == self._dev:
                s0, s1, s2 = t.stride()
                if s2 == 1:
                    return (s0 if n > 1 else heads * self.head_dim), (s1 if heads > 1 else self.head_dim)
        except _NO_TENSOR:
            pass
        _bad(f"{what}: [{n}, {heads}, {self.head_dim}], head_dim dense, of the cache's dtype and device")

    def write(self, k, v, seq, pos, q=None, q_out=None, rope_theta: float = 0.0):
        """dmtp_paged_write: rows k, v [n, n_kv_heads, head_dim] to positions pos of
        sequences seq (int32 [n]; seq < 0: skipped), rotated first if rope_theta > 0. With q
        [n, n_heads, head_dim] returns the rotated queries (q_out, or a new tensor)."""
        c, dev = _c(), self._dev
        qp = qop = qr = qh = qor = qoh = heads = 0
        try:
            n, h = seq.shape[0], self.n_kv_heads
            if q is not None:
                heads = q.shape[1]
                if q_out is None:
                    q_out = c.torch.empty(q.shape, dtype=q.dtype, device=q.device)
        except _NO_TENSOR:
            _bad("seq: int32 [n]; q: [n, n_heads, head_dim]")
        kr, kh = self._rows(k, n, h, "k")
        vr, vh = self._rows(v, n, h, "v")
        if q is not None:
            qr, qh = self._rows(q, n, heads, "q")
            qor, qoh = self._rows(q_out, n, heads, "q_out")
            qp, qop = q.data_ptr(), q_out.data_ptr()
        _run(c, c.paged_write, dev, "dmtp_paged_write", self._c,
             _pack(_ROWS, qp, k.data_ptr(), v.data_ptr(), qop, qr, qh, kr, kh, vr, vh, qor, qoh,
                   _vector(seq, c.int32, n, dev, "seq"),
                   _vector(pos, c.int32, n, dev, "pos"), n, heads, rope_theta), self._err)
        return q_out

    def read(self, seq, pos, k_out=None, v_out=None):
        """dmtp_paged_read: positions pos of sequences seq (int32 [n]) as dense rows
        [n, n_kv_heads, head_dim]; returns (k, v)."""
        c, dev = _c(), self._dev
        try:
            n = seq.shape[0]
            shape = (n, self.n_kv_heads, self.head_dim)
            if k_out is None:
                k_out = c.torch.empty(shape, dtype=self.dtype, device=self.device)
            if v_out is None:
                v_out = c.torch.empty(shape, dtype=self.dtype, device=self.device)
            for t in (k_out, v_out):
                if t.shape != shape or t.dtype is not self.dtype or not t.is_contiguous() or \
                        t.get_device() != dev:
                    _bad(f"k_out, v_out: dense {shape} of the cache's dtype and device")
        except _NO_TENSOR:
            _bad("seq: int32 [n]; k_out, v_out: [n, n_kv_heads, head_dim]")
        _run(c, c.paged_read, dev, "dmtp_paged_read", self._c,
             _vector(seq, c.int32, n, dev, "seq"), _vector(pos, c.int32, n, dev, "pos"), n,
             k_out.data_ptr(), v_out.data_ptr(), self._err)
        return k_out, v_out

    def attention(self, q, kv_len, scale=None, window: int = 0, out=None, workspace=None):
        """dmtp_paged_attention: q [n_seqs, rows, n_heads, head_dim], the newest rows of each
        sequence; kv_len int32 [n_seqs], its length with them. scale: 1/sqrt(head_dim) if
        None; window > 0: a row sees that many positions. workspace: a uint8 tensor of
        attention_workspace() bytes that no overlapping call uses; None: taken from PyTorch's
        allocator for this call."""
        c, dev = _c(), self._dev
        try:
            shape = q.shape
            if len(shape) != 4:
                _bad("q: [n_seqs, rows, n_heads, head_dim]")
            B, rows, heads, hd = shape
            if out is None:
                out = c.torch.empty(shape, dtype=q.dtype, device=q.device)
            if B != self.n_seqs or hd != self.head_dim or q.dtype is not self.dtype or \
                    q.get_device() != dev:
                _bad(f"q: [{self.n_seqs}, rows, n_heads, {self.head_dim}] of the cache's dtype and device")
            if out.shape != shape or out.dtype is not self.dtype or out.get_device() != dev:
                _bad("out: the shape, dtype and device of q")
            qb, qr, qh, q1 = q.stride()
            ob, orow, oh, o1 = out.stride()
        except _NO_TENSOR:
            _bad("q, out: [n_seqs, rows, n_heads, head_dim]")
        if q1 != 1 or o1 != 1:
            _bad("head_dim must be dense")
        if B == 1:  # (the stride of a dimension of one element says nothing)
            qb = ob = hd
        if rows == 1:
            qr = orow = hd
        if heads == 1:
            qh = oh = hd
        a = _pack(_QUERY, q.data_ptr(), out.data_ptr(), qb, qr, qh, ob, orow, oh,
                        _vector(kv_len, c.int32, B, dev, "kv_len"), rows, heads, window,
                        self._scale if scale is None else scale)
        n = self._ws_bytes.get((rows, heads))
        if n is None:
            n = self._ws_bytes[rows, heads] = self.attention_workspace(rows, heads)
        if workspace is not None:
            try:
                ok = workspace.dtype is c.torch.uint8 and workspace.get_device() == dev and \
                    workspace.is_contiguous()
            except _NO_TENSOR:
                ok = False
            if not ok:
                _bad("workspace: a dense uint8 tensor on the cache's device")
            n = workspace.numel()
        elif n and dev >= 0:  # on the stream that the kernels are enqueued on
            workspace = c.torch.empty(n, dtype=c.torch.uint8, device=self.device)
        _run(c, c.paged_attention, dev, "dmtp_paged_attention", self._c, a,
             workspace.data_ptr() if workspace is not None else None, n, self._err)
        return out

    def attention_workspace(self, rows: int, n_heads: int) -> int:
        """Bytes of workspace that attention() needs for q of these rows and heads."""
        a = _pack(_QUERY, 0, 0, 0, 0, 0, 0, 0, 0, 0, rows, n_heads, 0, 1.0)
        size = C.c_size_t()
        _check(_c().paged_attention_workspace(self._c, a, C.byref(size)),
               "dmtp_paged_attention_workspace")
        return size.value

    def check(self):
        """Wait for the device and raise DmtpError(DMTP_EDEVICE) if any call since the last
        check met an index out of range; the bits that it reports are then cleared."""
        torch = _c().torch
        with self._lock:
            torch.cuda.synchronize(self.device)
            word = int(self.err.item())
            if word:
                # taken off by an atomic addition: a bit that a call on another stream sets after
                # the word was read stays for the next check
                self.err.index_add_(0, self._word, torch.full_like(self.err, -word))
        if word:
            raise DmtpError(-5, "paged cache", word)


def _matrix(t, shape, dtype, dev: int, what: str) -> int:
    """Row pitch of a matrix with dense rows."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            s0, s1 = t.stride()
            if s1 == 1 or shape[1] == 1:
                return s0 if shape[0] > 1 else shape[1]
    except _NO_TENSOR:
        pass
    _bad(f"{what}: {dtype} {tuple(shape)} with dense rows on the same device")


def add_rmsnorm_e4m3(x, y, gain, eps: float = 1e-6, x_out=None, q=None, scale=None):
    """dmtp_add_rmsnorm_e4m3: x_out = x + y, and E4M3 rows of RMSNorm(x + y) * gain. x, y
    [rows, d] bf16 or fp32 (y None: no addition); x_out may be x (None: a new tensor, or x
    where y is None). Returns (x_out, q float8_e4m3fn [rows, d], scale fp32 [rows])."""
    c = _c()
    try:
        dev, shape = x.get_device(), x.shape
    except _NO_TENSOR:
        _bad("x: [rows, d]")
    if len(shape) != 2:
        _bad("x: [rows, d]")
    rows, d = shape
    x_dt, y_dt, g_dt = _dtype(c, x), 0, _dtype(c, gain)
    xr = _matrix(x, shape, x.dtype, dev, "x")
    yp = yr = xop = xor = 0
    if y is not None:
        y_dt = _dtype(c, y)
        yr, yp = _matrix(y, shape, y.dtype, dev, "y"), y.data_ptr()
        if x_out is None:
            x_out = c.torch.empty(shape, dtype=x.dtype, device=x.device)
    if x_out is not None:
        xor, xop = _matrix(x_out, shape, x.dtype, dev, "x_out"), x_out.data_ptr()
    if q is None:
        q = c.torch.empty(shape, dtype=c.f8, device=x.device)
    if scale is None:
        scale = c.torch.empty(rows, dtype=c.fp32, device=x.device)
    qr = _matrix(q, shape, c.f8, dev, "q")
    _run(c, c.add_rmsnorm_e4m3, dev, "dmtp_add_rmsnorm_e4m3",
         _pack(_NORM, x.data_ptr(), yp, _vector(gain, gain.dtype, d, dev, "gain"), xop, q.data_ptr(),
                    _vector(scale, c.fp32, rows, dev, "scale"), xr, yr, xor, qr, rows, d, x_dt,
                    y_dt, g_dt, eps))
    return (x if x_out is None else x_out), q, scale


def sample_rows(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, ids=None,
                kept=None):
    """dmtp_sample_rows: one token id per row of logits [rows, vocab] (bf16 or fp32), drawn
    with the uniform numbers u (fp32 [rows]) under temperature, top_k (int32), top_p and
    min_p (fp32 [rows] each, None: off). Returns ids (int32 [rows]; -1 where nothing may be
    chosen); kept (int32 [rows], optional) receives how many tokens passed the filters."""
    c = _c()
    try:
        dev, shape = logits.get_device(), logits.shape
    except _NO_TENSOR:
        _bad("logits: [rows, vocab]")
    if len(shape) != 2:
        _bad("logits: [rows, vocab]")
    rows, V = shape
    dt = _dtype(c, logits)
    ld = _matrix(logits, shape, logits.dtype, dev, "logits")
    if ids is None:
        ids = c.torch.empty(rows, dtype=c.int32, device=logits.device)
    f, i = c.fp32, c.int32
    _run(c, c.sample_rows, dev, "dmtp_sample_rows",
         _pack(_SAMPLE, logits.data_ptr(), ld, rows, V, dt, _vector(u, f, rows, dev, "u"),
                      0 if temperature is None else _vector(temperature, f, rows, dev, "temperature"),
                      0 if top_k is None else _vector(top_k, i, rows, dev, "top_k"),
                      0 if top_p is None else _vector(top_p, f, rows, dev, "top_p"),
                      0 if min_p is None else _vector(min_p, f, rows, dev, "min_p"),
                      _vector(ids, i, rows, dev, "ids"),
                      0 if kept is None else _vector(kept, i, rows, dev, "kept")))
    return ids
