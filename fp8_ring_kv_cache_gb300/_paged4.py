"""Rotary positions in other forms and the paged cache in 4 bits (include/rc.h).

    form = rc.RopeForm(128, layout="halves", scaling="parts", factor=16, context=4096, gain=1.25)
    rc.rc_rope_turn(q, positions, form, out=q)            # positions: int32 [axes][n]
    cache = rc.PagedKVCache4.empty(pages=4096, kv_heads=8, head_dim=128, page_tokens=64)
    batch = rc.PagedBatch(page_table, kv_len, q_start, tokens=n, max_new=m, max_kv=l)
    cache.write(batch, k, v, positions, form)             # E2M1 codes, a scale per 16 dims
    cache.attend(batch, q, out, lse=lse)                  # out: bf16
    cache.sync()                                          # raises RcError on bad metadata

Streams, devices and the lives of tensors are as in ``_paged.py``.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _check, lib
from ._paged import (RC_PAGED_WORKSPACE_BYTES, RC_ROPE_SHARED_FREQS, PagedBatch, _call, _filled, _positions, _rows,
                     _tensor, _turned)

RC_ROPE_MAX_AXES, RC_ROPE_MAX_HEAD_DIM = 4, 256
_LAYOUTS = {"pairs": 0, "halves": 1}
_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}


class rc_rope_spec(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("first", ctypes.c_int), ("dims", ctypes.c_int), ("layout", ctypes.c_int),
                ("axes", ctypes.c_int), ("sections", ctypes.c_int * RC_ROPE_MAX_AXES), ("flags", ctypes.c_uint),
                ("base", ctypes.c_double), ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("context", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double), ("gain", ctypes.c_float)]


class rc_rope_form(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("first", ctypes.c_int), ("dims", ctypes.c_int), ("layout", ctypes.c_int),
                ("axes", ctypes.c_int), ("gain", ctypes.c_float), ("turns", ctypes.c_uint64 * (RC_ROPE_MAX_HEAD_DIM // 2)),
                ("axis", ctypes.c_uint8 * (RC_ROPE_MAX_HEAD_DIM // 2))]


class rc_paged4_view(ctypes.Structure):
    _fields_ = [("kcodes", ctypes.c_void_p), ("vcodes", ctypes.c_void_p), ("kscale", ctypes.c_void_p),
                ("vscale", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("page_tokens", ctypes.c_int)]


_P, _I, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
for _name, _args in {
    "rc_rope_form_init": [_P, _P],
    "rc_rope_turn": [_P, _P, _I64, _P, _I64, _I, _I64, _I, _P, _I64, _I, _P],
    "rc_paged4_write": [_P, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P],
    "rc_paged4_attend": [_P, _P, _P, _I64, _I, _P, _I64, _P, _I, _P],
    "rc_paged4_status": [_P, _P],
}.items():
    getattr(lib, _name).argtypes = _args
    getattr(lib, _name).restype = _I


class RopeForm:
    """A form of rotary positions: dims first .. first + dims - 1 of a head turn (dims: the rest of the head, or twice the
    sum of `sections`), as neighbouring "pairs" or as "halves" of that part; sections: pairs of each axis (one axis by
    default).  scaling: None, "linear", "base" or "parts", by `factor`; "parts" also reads context, low and high, the
    turns in `context` positions between which a frequency goes over from stretched to kept, evenly over the turns (a model
    that was trained with the same evenly over the pairs' numbers, or with factors of its own for each pair, has other
    frequencies, which this class does not make).  gain multiplies what turns."""

    def __init__(self, head_dim: int, sections=None, dims=None, first: int = 0, layout: str = "pairs", base: float = 10000.0,
                 shared_freqs: bool = False, scaling=None, factor: float = 1.0, context: float = 0.0, low: float = 1.0,
                 high: float = 32.0, gain: float = 1.0):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {list(_SCALINGS)}, got {scaling!r}")
        first = int(first)
        if dims is None:
            dims = 2 * sum(int(w) for w in sections) if sections is not None else head_dim - first
        sections = (int(dims) // 2,) if sections is None else tuple(int(w) for w in sections)
        if not 1 <= len(sections) <= RC_ROPE_MAX_AXES:
            raise ValueError(f"1 to {RC_ROPE_MAX_AXES} axes, got {len(sections)}")
        self.head_dim, self.first, self.dims, self.layout = int(head_dim), first, int(dims), layout
        self.sections, self.axes = sections, len(sections)
        spec = rc_rope_spec(head_dim=self.head_dim, first=first, dims=self.dims, layout=_LAYOUTS[layout], axes=self.axes,
                            flags=RC_ROPE_SHARED_FREQS if shared_freqs else 0, base=float(base), scaling=_SCALINGS[scaling],
                            factor=float(factor), context=float(context), low=float(low), high=float(high), gain=float(gain))
        spec.sections[:self.axes] = sections
        self.form = rc_rope_form()
        _check(lib.rc_rope_form_init(ctypes.addressof(self.form), ctypes.addressof(spec)), "rc_rope_form_init")
        self.gain = self.form.gain
        self._ptr = ctypes.addressof(self.form)

    def __setstate__(self, state):  # (a deep copy, or one from another process, has numbers of its own)
        self.__dict__.update(state)
        self._ptr = ctypes.addressof(self.form)


def rc_rope_turn(x, positions, form: RopeForm, out=None, back: bool = False, stream=None):
    """x [n][heads][head_dim] (bf16 or fp32) turned at positions (int32 [axes][n]) in the form's manner, times its gain;
    back turns back with the same gain, which is the gradient: dx = rc_rope_turn(dy, positions, form, back=True).  out,
    streams and autograd as for rc_rope_axes."""
    return _turned(x, positions, form, out, back, stream, "rc_rope_turn", lib.rc_rope_turn, rc_rope_turn)


class PagedKVCache4:
    """One layer's pages in 4 bits (uint8 tensors kcodes [pages][kv_heads][P][head_dim / 2], vcodes
    [pages][kv_heads][head_dim][P / 2], kscale and vscale [pages][kv_heads][head_dim / 16][P]) and the workspace of the
    calls on them.  The calls fill tensors that the caller passes; autograd records none of them."""

    def __init__(self, kcodes, vcodes, kscale, vscale, workspace=None):
        if not isinstance(kcodes, torch.Tensor) or kcodes.dim() != 4:
            raise ValueError("kcodes must be a [pages][kv_heads][page_tokens][head_dim / 2] tensor")
        n, h, p, d = kcodes.shape
        d *= 2
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = n, h, p, d
        self.device = kcodes.device
        if not kcodes.is_cuda:
            raise TypeError("kcodes must be a CUDA tensor")
        c = rc_paged4_view()
        c.kcodes = _tensor(kcodes, torch.uint8, (n, h, p, d // 2), "kcodes", self.device)
        c.vcodes = _tensor(vcodes, torch.uint8, (n, h, d, p // 2), "vcodes", self.device)
        c.kscale = _tensor(kscale, torch.uint8, (n, h, d // 16, p), "kscale", self.device)
        c.vscale = _tensor(vscale, torch.uint8, (n, h, d // 16, p), "vscale", self.device)
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
              workspace=None) -> "PagedKVCache4":
        """New zeroed pages.  Caches whose calls are issued on one stream (a model's layers, FP8 ones among them) can share
        a workspace: pass the first one's `workspace`; each has one of its own (RC_PAGED_WORKSPACE_BYTES, 64 MB) otherwise."""
        def new(*shape):
            return torch.zeros(shape, dtype=torch.uint8, device=device)
        cache = cls(new(pages, kv_heads, page_tokens, head_dim // 2), new(pages, kv_heads, head_dim, page_tokens // 2),
                    new(pages, kv_heads, head_dim // 16, page_tokens), new(pages, kv_heads, head_dim // 16, page_tokens), workspace)
        if workspace is not None:
            _filled(cache.device)
        return cache

    def _batch(self, batch: PagedBatch):
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        return batch._ptr

    def write(self, batch: PagedBatch, K, V, positions=None, form: RopeForm | None = None, stream=None) -> None:
        """The batch's new tokens into their pages; form None: K is stored as it comes."""
        n, h, d = batch.tokens, self.kv_heads, self.head_dim
        kp, ks = _rows(K, torch.bfloat16, n, h, d, "K", self.device)
        vp, vs = _rows(V, torch.bfloat16, n, h, d, "V", self.device)
        pp, ps, fp = None, 0, None
        if form is not None:
            if form.head_dim != d:
                raise ValueError(f"the form has head_dim {form.head_dim}, the cache {d}")
            pp, ps = _positions(positions, form.axes, n, "positions", self.device)
            fp = form._ptr
        elif positions is not None:
            raise ValueError("positions without a form")
        _call(self.device, stream, "rc_paged4_write", lib.rc_paged4_write, self._ptr, self._batch(batch), kp, ks, vp, vs, pp,
              ps, fp)

    def attend(self, batch: PagedBatch, Q, out, lse=None, causal: bool = True, stream=None) -> None:
        n, d = batch.tokens, self.head_dim
        if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
            raise ValueError("Q must be a [tokens][heads][head_dim] tensor")
        heads = Q.shape[1]
        qp, qs = _rows(Q, torch.bfloat16, n, heads, d, "Q", self.device)
        op, os_ = _rows(out, torch.bfloat16, n, heads, d, "out", self.device)
        lp = None if lse is None else _tensor(lse, torch.float32, (n, heads), "lse", self.device)
        _call(self.device, stream, "rc_paged4_attend", lib.rc_paged4_attend, self._ptr, self._batch(batch), qp, qs, heads, op,
              os_, lp, 1 if causal else 0)

    def sync(self, stream=None) -> None:
        """Wait for the stream; raises RcError if a call on this cache found bad metadata or failed."""
        _call(self.device, stream, "rc_paged4_status", lib.rc_paged4_status, self._ptr)
