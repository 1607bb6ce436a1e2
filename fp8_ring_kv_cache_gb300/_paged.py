"""Several-axes rotary positions and the paged FP8 cache (include/rc.h).

The tensors are the caller's; the objects here only hold them and the C
structures that describe them, so they are made once and used for many calls:

    rope = rc.RopeAxes((24, 20, 20))                      # pairs of time, height, width
    rc.rc_rope_axes(q, positions, rope, out=q)            # positions: int32 [axes][n]
    cache = rc.PagedKVCache.empty(pages=4096, kv_heads=8, head_dim=128, page_tokens=64)
    batch = rc.PagedBatch(page_table, kv_len, q_start, tokens=n, max_new=m, max_kv=l)
    cache.write(batch, k, v, positions, rope)
    cache.attend(batch, q, out, lse=lse)                  # out: bf16
    cache.accumulate(batch, q, lse, scores)               # scores += attention weight
    cache.evict(batch, scores, keep=4096, recent=256, dst_table=..., kept=..., kv_len_out=...)
    cache.sync()                                          # raises RcError on bad metadata

Every call is stream-ordered on torch's current stream of the tensors' device
(or ``stream=``), allocates nothing but the result of ``rc_rope_axes`` without
``out=``, and runs on that device whichever is current.
A cache that is constructed here (its workspace, and the pages of ``empty``) is
ready for calls on any stream; the tensors that a caller passes have to be ready on
the call's stream, and to live until it is through with them.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _check, lib

RC_ROPE_SHARED_FREQS = 1
RC_BF16, RC_F32 = 0, 1
RC_PAGED_WORKSPACE_BYTES = 64 << 20


class rc_rope_plan(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("axes", ctypes.c_int), ("turns", ctypes.c_uint64 * 64),
                ("axis", ctypes.c_uint8 * 64)]


class rc_paged_view(ctypes.Structure):
    _fields_ = [("kcodes", ctypes.c_void_p), ("vcodes", ctypes.c_void_p), ("kscale", ctypes.c_void_p),
                ("vscale", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_tokens", ctypes.c_int)]


class rc_paged_batch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("seqs", ctypes.c_int), ("table_pages", ctypes.c_int), ("tokens", ctypes.c_int),
                ("max_new", ctypes.c_int), ("max_kv", ctypes.c_int)]


_P, _I, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
for _name, _args in {
    "rc_rope_plan_init": [_P, _I, _I, _P, ctypes.c_double, ctypes.c_uint],
    "rc_rope_axes": [_P, _P, _I64, _P, _I64, _I, _I64, _I, _P, _I64, _I, _P],
    "rc_paged_write": [_P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P],
    "rc_paged_attend": [_P, _P, _P, _I64, _I, _P, _I64, _P, _I, _P],
    "rc_paged_accumulate": [_P, _P, _P, _I64, _I, _P, _P, _P, _I64, _I, _P],
    "rc_paged_evict": [_P, _P, _P, _I64, _I, _I, _P, _I, _P, _P, _P, _P],
    "rc_paged_status": [_P, _P],
    "rc_paged_set_wait_limit": [ctypes.c_uint64],
}.items():
    getattr(lib, _name).argtypes = _args
    getattr(lib, _name).restype = _I


def _refuse(t, dtype, shape, what: str, device):
    """Raise what is wrong with t, the first of: type, place, dtype, shape, device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what} is on {t.device}, not on {device}")


# (a call's checks are most of its time on the host: the usual case asks each thing
# once; `device` is always a CUDA device)
def _tensor(t, dtype, shape, what: str, device) -> int:
    """Address of a CUDA tensor of this type and shape, contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device):
        _refuse(t, dtype, shape, what, device)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, dtype, n, heads, dim, what: str, device) -> tuple[int, int]:
    """Address and token stride of a [n][heads][dim] tensor whose tokens may lie apart."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n, heads, dim) and t.device == device):
        _refuse(t, dtype, (n, heads, dim), what, device)
    s0, s1, s2 = t.stride()
    if n and ((s2 != 1 and dim > 1) or (s1 != dim and heads > 1)):
        raise ValueError(f"{what}: a token's heads must be contiguous")
    return t.data_ptr(), s0 if n > 1 else heads * dim


def _rows_meet(a: int, sa: int, b: int, sb: int, n: int, width: int) -> bool:
    """Whether n rows of `width` bytes, sa bytes apart from address a, share a byte with those sb apart from b."""
    d = b - a
    if n < 1 or d >= (n - 1) * sa + width or -d >= (n - 1) * sb + width:
        return False
    if n == 1 or sa == sb:  # row j of b begins d + (j - i) s behind row i of a: the largest j - i that is not too far
        k = min((width - 1 - d) // sa, n - 1)
        return k > -n and d + k * sa + width > 0
    for i in range(n):
        j = min((i * sa - d + width - 1) // sb, n - 1)
        if j >= 0 and j * sb + width > i * sa - d:
            return True
    return False


def _positions(t, axes, n, what: str, device) -> tuple[int, int]:
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == (axes, n) and t.device == device):
        _refuse(t, torch.int32, (axes, n), what, device)
    s0, s1 = t.stride()
    if n > 1 and s1 != 1:
        raise ValueError(f"{what}: an axis' positions must be contiguous")
    return t.data_ptr(), s0 if axes > 1 else n


# the raw handle of a device's current stream, and the current device, without the
# wrapper objects of torch.cuda (a fifth of a short call's time on the host)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _call(device, stream, what: str, fn, *args) -> None:
    """Call fn(*args, stream) with `device` current."""
    index = device.index
    if stream is None:
        sp = _raw_stream(index)
    else:
        sp = stream if isinstance(stream, int) else stream.cuda_stream
    if _current_device() == index:
        st = fn(*args, sp)
    else:
        with torch.cuda.device(device):
            st = fn(*args, sp)
    if st:
        _check(st, what)


def _filled(device) -> None:
    """Wait for the fills that were just issued on the device's current stream: the first call on what they fill may be
    on any stream.  (Inside a capture they are part of the graph, and there is nothing to wait for.)"""
    with torch.cuda.device(device):
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()


def _stream(stream, device):
    return torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream


def _empty_on(stream, shape, dtype, device):
    """A new tensor for a call on `stream`.  Its memory comes from that stream's pool, so that neither work still to be
    done on what lay there before nor the use of the block after this tensor is dropped can meet the call's kernel; and
    it is not reused before what the current stream does with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    own, current = _stream(stream, device), torch.cuda.current_stream(device)
    with torch.cuda.stream(own):
        t = torch.empty(shape, dtype=dtype, device=device)
    if own.cuda_stream != current.cuda_stream:
        t.record_stream(current)
    return t


class RopeAxes:
    """The plan of several-axes rotary positions: `sections` pairs of each axis (their sum is head_dim / 2)."""

    def __init__(self, sections, base: float = 10000.0, shared_freqs: bool = False):
        self.sections = tuple(int(s) for s in sections)
        self.axes, self.head_dim = len(self.sections), 2 * sum(self.sections)
        self.plan = rc_rope_plan()
        arr = (ctypes.c_int * max(1, self.axes))(*self.sections)
        _check(lib.rc_rope_plan_init(ctypes.addressof(self.plan), self.head_dim, self.axes, arr, float(base),
                                     RC_ROPE_SHARED_FREQS if shared_freqs else 0), "rc_rope_plan_init")
        self._ptr = ctypes.addressof(self.plan)


class _Turn(torch.autograd.Function):
    """The turn with its gradient, the turn back."""

    @staticmethod
    def forward(ctx, x, positions, rope, inverse):
        ctx.rope, ctx.inverse = rope, inverse
        ctx.save_for_backward(positions)
        return rc_rope_axes(x.detach(), positions, rope, inverse=inverse)

    @staticmethod
    def backward(ctx, dy):
        dy = dy.contiguous()  # (a broadcast gradient has no strides that the kernel takes)
        if dy.data_ptr() % 16:
            dy = dy.clone()
        return rc_rope_axes(dy, ctx.saved_tensors[0], ctx.rope, inverse=not ctx.inverse), None, None, None


def rc_rope_axes(x, positions, rope: RopeAxes, out=None, inverse: bool = False, stream=None):
    """x [n][heads][head_dim] (bf16 or fp32) turned at positions (int32 [axes][n]); inverse turns back, which is also
    the gradient: dx = rc_rope_axes(dy, positions, rope, inverse=True).  out defaults to a new tensor (of the call's
    stream, kept from reuse for the current one too) and may be x.  Autograd records the call if x requires a gradient;
    as with torch's own functions, not with out=, which is refused then."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [n][heads][head_dim] tensor")
    if not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    n, heads, dim = x.shape
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    if dim != rope.head_dim:
        raise ValueError(f"x has head_dim {dim}, the plan {rope.head_dim}")
    if torch.is_grad_enabled() and (x.requires_grad or getattr(out, "requires_grad", False)):
        if out is not None:
            raise RuntimeError("rc_rope_axes: out= is not differentiable, but x or out requires a gradient")
        if stream is None:
            return _Turn.apply(x, positions, rope, inverse)
        own, current = _stream(stream, x.device), torch.cuda.current_stream(x.device)
        with torch.cuda.stream(own):  # (autograd runs the gradient on the stream of the turn)
            y = _Turn.apply(x, positions, rope, inverse)
        y.record_stream(current)
        return y
    xp, xs = _rows(x, x.dtype, n, heads, dim, "x", x.device)
    if out is None:
        out = _empty_on(stream, (n, heads, dim), x.dtype, x.device)
    op, os_ = _rows(out, x.dtype, n, heads, dim, "out", x.device)
    pp, ps = _positions(positions, rope.axes, n, "positions", x.device)
    if out is not x and (xp != op or xs != os_):
        size = x.element_size()
        row = heads * dim
        if op < xp + ((n - 1) * xs + row) * size and xp < op + ((n - 1) * os_ + row) * size and \
                _rows_meet(xp, xs * size, op, os_ * size, n, row * size):
            raise ValueError("out overlaps x without being x")
    _call(x.device, stream, "rc_rope_axes", lib.rc_rope_axes, rope._ptr, xp, xs, op, os_,
          RC_BF16 if x.dtype == torch.bfloat16 else RC_F32, n, heads, pp, ps, 1 if inverse else 0)
    return out


class PagedBatch:
    """The sequences of a call: page_table int32 [seqs][table_pages], kv_len int32 [seqs], q_start int32 [seqs + 1]
    (None for evict alone) on the device; tokens, max_new, max_kv the bounds that include/rc.h describes."""

    def __init__(self, page_table, kv_len, q_start=None, *, tokens: int = 0, max_new: int = 0, max_kv: int = 0):
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a [seqs][table_pages] tensor")
        self.seqs, self.table_pages = page_table.shape
        self.device = page_table.device
        if not page_table.is_cuda:
            raise TypeError("page_table must be a CUDA tensor")
        c = rc_paged_batch()
        c.page_table = _tensor(page_table, torch.int32, (self.seqs, self.table_pages), "page_table", self.device)
        c.kv_len = _tensor(kv_len, torch.int32, (self.seqs,), "kv_len", self.device)
        if q_start is not None:
            c.q_start = _tensor(q_start, torch.int32, (self.seqs + 1,), "q_start", self.device)
        c.seqs, c.table_pages, c.tokens, c.max_new, c.max_kv = self.seqs, self.table_pages, tokens, max_new, max_kv
        self.tokens, self.max_new, self.max_kv = int(tokens), int(max_new), int(max_kv)
        self.page_table, self.kv_len, self.q_start = page_table, kv_len, q_start
        self._c, self._ptr = c, ctypes.addressof(c)


class PagedKVCache:
    """One layer's pages (uint8 tensors kcodes [pages][kv_heads][P][head_dim], vcodes [pages][kv_heads][head_dim][P],
    kscale and vscale [pages][kv_heads][P]) and the workspace of the calls on them.  The calls fill tensors that the
    caller passes; autograd records none of them."""

    def __init__(self, kcodes, vcodes, kscale, vscale, workspace=None):
        if not isinstance(kcodes, torch.Tensor) or kcodes.dim() != 4:
            raise ValueError("kcodes must be a [pages][kv_heads][page_tokens][head_dim] tensor")
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = kcodes.shape
        n, h, p, d = kcodes.shape
        self.device = kcodes.device
        if not kcodes.is_cuda:
            raise TypeError("kcodes must be a CUDA tensor")
        c = rc_paged_view()
        c.kcodes = _tensor(kcodes, torch.uint8, (n, h, p, d), "kcodes", self.device)
        c.vcodes = _tensor(vcodes, torch.uint8, (n, h, d, p), "vcodes", self.device)
        c.kscale = _tensor(kscale, torch.uint8, (n, h, p), "kscale", self.device)
        c.vscale = _tensor(vscale, torch.uint8, (n, h, p), "vscale", self.device)
        own_workspace = workspace is None
        if own_workspace:
            workspace = torch.zeros(RC_PAGED_WORKSPACE_BYTES, dtype=torch.uint8, device=self.device)
        c.workspace = _tensor(workspace, torch.uint8, (RC_PAGED_WORKSPACE_BYTES,), "workspace", self.device)
        c.pages, c.kv_heads, c.head_dim, c.page_tokens = n, h, d, p
        self.kcodes, self.vcodes, self.kscale, self.vscale, self.workspace = kcodes, vcodes, kscale, vscale, workspace
        self._c, self._ptr = c, ctypes.addressof(c)
        if own_workspace:
            _filled(self.device)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda",
              workspace=None) -> "PagedKVCache":
        """New zeroed pages.  Caches whose calls are issued on one stream (a model's layers) can share a workspace:
        pass the first one's `workspace`; each has one of its own (RC_PAGED_WORKSPACE_BYTES, 64 MB) otherwise."""
        def new(*shape):
            return torch.zeros(shape, dtype=torch.uint8, device=device)
        cache = cls(new(pages, kv_heads, page_tokens, head_dim), new(pages, kv_heads, head_dim, page_tokens),
                    new(pages, kv_heads, page_tokens), new(pages, kv_heads, page_tokens), workspace)
        if workspace is not None:
            _filled(cache.device)
        return cache

    def _batch(self, batch: PagedBatch):
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        return batch._ptr

    def write(self, batch: PagedBatch, K, V, positions, rope: RopeAxes, stream=None) -> None:
        n, h, d = batch.tokens, self.kv_heads, self.head_dim
        if rope.head_dim != d:
            raise ValueError(f"the plan has head_dim {rope.head_dim}, the cache {d}")
        kp, ks = _rows(K, torch.bfloat16, n, h, d, "K", self.device)
        vp, vs = _rows(V, torch.bfloat16, n, h, d, "V", self.device)
        pp, ps = _positions(positions, rope.axes, n, "positions", self.device)
        _call(self.device, stream, "rc_paged_write", lib.rc_paged_write, self._ptr, self._batch(batch), kp, ks, vp, vs, pp,
              ps, rope._ptr)

    def attend(self, batch: PagedBatch, Q, out, lse=None, causal: bool = True, stream=None) -> None:
        n, d = batch.tokens, self.head_dim
        if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
            raise ValueError("Q must be a [tokens][heads][head_dim] tensor")
        heads = Q.shape[1]
        qp, qs = _rows(Q, torch.bfloat16, n, heads, d, "Q", self.device)
        op, os_ = _rows(out, torch.bfloat16, n, heads, d, "out", self.device)
        lp = None if lse is None else _tensor(lse, torch.float32, (n, heads), "lse", self.device)
        _call(self.device, stream, "rc_paged_attend", lib.rc_paged_attend, self._ptr, self._batch(batch), qp, qs, heads, op,
              os_, lp, 1 if causal else 0)

    def accumulate(self, batch: PagedBatch, Q, lse, scores, out=None, causal: bool = True, stream=None) -> None:
        """out (default: scores, in place) = scores + the attention weight of this call's queries per cached token;
        scores, out: fp32 [seqs][kv_heads][>= max_kv]."""
        n, d = batch.tokens, self.head_dim
        if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
            raise ValueError("Q must be a [tokens][heads][head_dim] tensor")
        heads = Q.shape[1]
        qp, qs = _rows(Q, torch.bfloat16, n, heads, d, "Q", self.device)
        lp = _tensor(lse, torch.float32, (n, heads), "lse", self.device)
        sp, stride = self._scores(batch, scores, "scores")
        op = sp if out is None else _tensor(out, torch.float32, scores.shape, "out", self.device)
        _call(self.device, stream, "rc_paged_accumulate", lib.rc_paged_accumulate, self._ptr, self._batch(batch), qp, qs,
              heads, lp, sp, op, stride, 1 if causal else 0)

    def _scores(self, batch, scores, what):
        if not isinstance(scores, torch.Tensor) or scores.dim() != 3 or scores.shape[2] < batch.max_kv:
            raise ValueError(f"{what} must be a [seqs][kv_heads][>= max_kv] tensor")
        width = scores.shape[2]
        return _tensor(scores, torch.float32, (batch.seqs, self.kv_heads, width), what, self.device), width

    def evict(self, batch: PagedBatch, scores, *, keep: int, recent: int, dst_table, kept, kv_len_out, scores_out=None,
              stream=None) -> None:
        """Copy the kept tokens of each sequence and head to the pages of dst_table (include/rc.h: rc_paged_evict)."""
        sp, stride = self._scores(batch, scores, "scores")
        if not isinstance(dst_table, torch.Tensor) or dst_table.dim() != 2:
            raise ValueError("dst_table must be a [seqs][dst_pages] tensor")
        dst_pages = dst_table.shape[1]
        keep = int(keep)
        shape = (batch.seqs, self.kv_heads, keep)
        tp = _tensor(dst_table, torch.int32, (batch.seqs, dst_pages), "dst_table", self.device)
        kp = _tensor(kept, torch.int32, shape, "kept", self.device)
        lp = _tensor(kv_len_out, torch.int32, (batch.seqs,), "kv_len_out", self.device)
        op = None if scores_out is None else _tensor(scores_out, torch.float32, shape, "scores_out", self.device)
        _call(self.device, stream, "rc_paged_evict", lib.rc_paged_evict, self._ptr, self._batch(batch), sp, stride, keep,
              int(recent), tp, dst_pages, kp, lp, op)

    def sync(self, stream=None) -> None:
        """Wait for the stream; raises RcError if a call on this cache found bad metadata or failed."""
        _call(self.device, stream, "rc_paged_status", lib.rc_paged_status, self._ptr)


def rc_paged_set_wait_limit(ns: int) -> None:
    _check(lib.rc_paged_set_wait_limit(int(ns)), "rc_paged_set_wait_limit")
