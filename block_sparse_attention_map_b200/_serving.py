"""Positions and the paged cache: rotary positions with several axes (forward,
backward, and into a cache), attention of drafted tokens over a paged key/value
cache, and eviction from it by accumulated attention weight.

Argument marshalling only, like the rest of the binding: every step runs in the
library's CUDA kernels (include/bsa.h), on the current stream of the tensors'
device.  Wrong arguments raise ValueError here or BsaError from the library."""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import BsaError, _check, c_f32, c_i32, c_i64, c_vp, lib

DTYPE = {torch.bfloat16: 0, torch.float16: 1}
LAYOUT = {"interleaved": 0, "halves": 1}
MAX_TREE = 64


class RopeSpec(ctypes.Structure):
    _fields_ = [("n_axes", c_i32), ("n_pairs", c_i32), ("layout", c_i32), ("inverse", c_i32),
                ("inv_freq", c_vp), ("axis", c_vp), ("pos", c_vp), ("pos_stride", c_i64 * 2)]


class Tokens(ctypes.Structure):
    _fields_ = [("B", c_i32), ("T", c_i32), ("H", c_i32), ("H_kv", c_i32), ("D", c_i32), ("dtype", c_i32),
                ("q_stride", c_i64 * 3), ("k_stride", c_i64 * 3), ("v_stride", c_i64 * 3),
                ("qo_stride", c_i64 * 3), ("ko_stride", c_i64 * 3), ("scale", c_f32), ("reserved", c_i32),
                ("n_new", c_vp), ("tree", c_vp)]


class Cache(ctypes.Structure):
    _fields_ = [("n_pages", c_i32), ("page_size", c_i32), ("H_kv", c_i32), ("D", c_i32), ("dtype", c_i32),
                ("B", c_i32), ("max_pages", c_i32), ("reserved", c_i32), ("k", c_vp), ("v", c_vp),
                ("k_stride", c_i64 * 3), ("v_stride", c_i64 * 3), ("page_table", c_vp), ("table_stride", c_i64),
                ("length", c_vp)]


class EvictSpec(ctypes.Structure):
    _fields_ = [("budget", c_i32), ("sinks", c_i32), ("recent", c_i32), ("reserved", c_i32), ("next_pos", c_vp),
                ("score_in", c_vp), ("pos_in", c_vp), ("score_out", c_vp), ("pos_out", c_vp), ("length_out", c_vp)]


_P = ctypes.POINTER
_SIGNATURES = {
    "bsa_rope": [_P(Tokens), _P(RopeSpec), c_vp, c_vp, c_vp, c_vp, c_vp],
    "bsa_cache_workspace_size": [_P(Cache), c_i32, _P(ctypes.c_size_t)],
    "bsa_cache_append": [_P(Cache), _P(Tokens), _P(RopeSpec), c_vp, c_vp, c_vp, c_vp, c_vp, ctypes.c_size_t, c_vp],
    "bsa_cache_attend": [_P(Cache), _P(Tokens), c_vp, c_vp, c_vp, c_vp, ctypes.c_size_t, c_vp],
    "bsa_cache_weigh": [_P(Cache), _P(Tokens), c_vp, c_vp, c_vp, c_vp, c_vp, ctypes.c_size_t, c_vp],
    "bsa_cache_evict": [_P(Cache), _P(EvictSpec), c_vp, ctypes.c_size_t, c_vp],
}
_FNS: dict = {}


def _fn(name):
    f = _FNS.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.restype, f.argtypes = c_i32, _SIGNATURES[name]
        _FNS[name] = f
    return f


def _call(name, device, *args):
    """One library call on the current stream of ``device``, with it current."""
    fn = _fn(name)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc != 0:
        raise BsaError(rc, name)


def _rows(t, name, device, dtype=None):
    """The strides of a [B, S, H, D] tensor of the operators' types on ``device``."""
    if t.dim() != 4 or t.device != device or (t.dtype not in DTYPE if dtype is None else t.dtype != dtype):
        raise ValueError(f"{name}: expected a [B, S, H, D] {dtype or 'bf16 or fp16'} tensor on {device}")
    s = t.stride()
    if s[3] != 1 and t.shape[3] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    if 0 in s[:3] and any(st == 0 and n > 1 for st, n in zip(s[:3], t.shape)):
        raise ValueError(f"{name}: a broadcast dimension (stride 0) is not taken")
    if t.numel() == 0 or 0 in s[:3]:
        return (0, 0, 0) if t.is_contiguous() else tuple(max(x, 8) for x in s[:3])
    return s[:3]


def _flat(t, name, device, dtype, shape):
    """A contiguous tensor of exactly this type and shape on ``device``; its address."""
    if t.dtype != dtype or t.device != device or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape} on {device}")
    return t.data_ptr()


def _rope_spec(B, T, D, device, pos, inv_freq, axis, layout, inverse):
    if layout not in LAYOUT:
        raise ValueError(f"layout: one of {sorted(LAYOUT)}")
    if pos.dim() != 3 or pos.shape[1:] != (B, T) or pos.dtype != torch.int32 or pos.device != device or \
            (T > 1 and pos.stride(2) != 1):
        raise ValueError(f"pos: expected int32 [n_axes, {B}, {T}] on {device}, contiguous in the tokens")
    n = inv_freq.numel()
    r = RopeSpec(pos.shape[0], n, LAYOUT[layout], 1 if inverse else 0)
    r.inv_freq = _flat(inv_freq, "inv_freq", device, torch.float64, (n,))
    r.axis = _flat(axis, "axis", device, torch.int32, (n,))
    r.pos = pos.data_ptr()
    if not pos.is_contiguous():
        r.pos_stride[:] = pos.stride()[:2]
        if r.pos_stride[0] == 0 and r.pos_stride[1] == 0:  # one row of positions for all
            raise ValueError("pos: give every axis and sequence its row (a fully broadcast pos is not taken)")
    return r


def _overlap(a, b):
    """Whether two tensors' spans of memory meet."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    end = lambda t: t.data_ptr() + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    return a.data_ptr() < end(b) and b.data_ptr() < end(a)


def _out_like(x, out, name):
    """The output of a rotation of ``x``: new, ``x`` itself, or apart from it."""
    if out is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out.shape != x.shape:
        raise ValueError(f"{name}: expected the input's shape {tuple(x.shape)}")
    if not (out.data_ptr() == x.data_ptr() and out.stride() == x.stride()) and _overlap(x, out):
        raise ValueError(f"{name}: overlaps its input without being it")
    return out


def _rotate(q, k, pos, inv_freq, axis, layout, inverse, q_out, k_out):
    x = q if q is not None else k
    if x is None:
        raise ValueError("give q, k or both")
    if not x.is_cuda or x.dim() != 4:
        raise ValueError("q and k are [B, S, H, D] CUDA tensors")
    device, dtype = x.device, x.dtype
    B, S, _, D = x.shape
    t = Tokens(B, S, q.shape[2] if q is not None else k.shape[2], k.shape[2] if k is not None else 0, D, DTYPE.get(dtype, -1))
    if q is not None and k is not None and (k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != D):
        raise ValueError("q and k must share B, S and D")
    ptr = [None] * 4
    if q is not None:
        q_out = _out_like(q, q_out, "q_out")
        t.q_stride[:] = _rows(q, "q", device)
        t.qo_stride[:] = _rows(q_out, "q_out", device, dtype)
        ptr[:2] = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        k_out = _out_like(k, k_out, "k_out")
        t.k_stride[:] = _rows(k, "k", device, dtype)
        t.ko_stride[:] = _rows(k_out, "k_out", device, dtype)
        ptr[2:] = k.data_ptr(), k_out.data_ptr()
        if q is None:
            t.H = t.H_kv
    r = _rope_spec(B, S, D, device, pos, inv_freq, axis, layout, inverse)
    _call("bsa_rope", device, t, r, *ptr)
    return q_out, k_out


def rope(q, k, pos, inv_freq, axis, layout="interleaved", q_out=None, k_out=None):
    """Rotary positions with several axes: (q_out, k_out), q [B, S, H, D] and k
    [B, S, H_kv, D] (either may be None) turned pair by pair by the angle
    ``pos[axis[p], b, t] * inv_freq[p]``.

    ``pos`` int32 [n_axes, B, S], ``inv_freq`` float64 [n_pairs] (radians per
    position), ``axis`` int32 [n_pairs].  ``layout``: pair p is the elements
    (2p, 2p+1) ("interleaved") or (p, p + n_pairs) ("halves"); elements past
    2 n_pairs are copied.  ``q_out=q`` rotates in place."""
    return _rotate(q, k, pos, inv_freq, axis, layout, False, q_out, k_out)


def rope_bwd(dq, dk, pos, inv_freq, axis, layout="interleaved", q_out=None, k_out=None):
    """The gradient of :func:`rope`: the incoming gradients of its outputs turned
    back by the same angles (the outputs go to ``q_out`` and ``k_out``)."""
    return _rotate(dq, dk, pos, inv_freq, axis, layout, True, q_out, k_out)


def tree_words(parents):
    """Tree words (int64 [B, T], bit j of word t: token t sees token j) from each
    token's parent (int [B, T]; -1: it follows the cache; a parent comes before
    its children).  A token sees its ancestors and itself."""
    B, T = parents.shape
    if T > MAX_TREE:
        raise ValueError(f"at most {MAX_TREE} tokens")
    host = parents.tolist()
    words = [[0] * T for _ in range(B)]
    for b in range(B):
        for t in range(T):
            p = host[b][t]
            if not -1 <= p < t:
                raise ValueError(f"parents[{b}, {t}] = {p}: a parent comes before its children")
            words[b][t] = (words[b][p] if p >= 0 else 0) | 1 << t
    signed = [[w - (1 << 64) if w >> 63 else w for w in row] for row in words]
    return torch.tensor(signed, dtype=torch.int64, device=parents.device).view(B, T)


class PagedCache:
    """A paged key/value cache and the calls around it.

    ``k``, ``v`` [n_pages, page_size, H_kv, D] (bf16 or fp16, the head dimension
    contiguous), ``page_table`` int32 [B, max_pages], ``length`` int32 [B]: the
    slots in use.  Slot s of sequence b is row s mod page_size of page
    page_table[b, s // page_size].  The tensors are kept, not copied: change
    ``length`` in place as tokens are accepted.  Only :meth:`append` and
    :meth:`evict` write the cache, in place.

    The calls of one PagedCache share a workspace, so they belong on one stream
    at a time; use one PagedCache (over the same tensors) per concurrent stream
    or captured graph."""

    def __init__(self, k, v, page_table, length):
        if not k.is_cuda or k.dim() != 4 or k.dtype not in DTYPE:
            raise ValueError("k and v are [n_pages, page_size, H_kv, D] bf16 or fp16 CUDA tensors")
        if v.shape != k.shape:
            raise ValueError("v must have k's shape")
        self.device, self.dtype = k.device, k.dtype
        self.k, self.v, self.page_table, self.length = k, v, page_table, length
        self.n_pages, self.page_size, self.H_kv, self.D = k.shape
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != self.device or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table: expected int32 [B, max_pages] on the cache's device, contiguous rows")
        self.B, self.max_pages = page_table.shape
        self.capacity = self.max_pages * self.page_size
        c = self._c = Cache(self.n_pages, self.page_size, self.H_kv, self.D, DTYPE[self.dtype], self.B, self.max_pages)
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.k_stride[:] = _rows(k, "k", self.device)
        c.v_stride[:] = _rows(v, "v", self.device, self.dtype)
        c.page_table = page_table.data_ptr()
        c.table_stride = page_table.stride(0) if self.B > 1 else 0
        c.length = _flat(length, "length", self.device, torch.int32, (self.B,))
        self._ws = None
        self._workspace(0)

    def _workspace(self, budget):
        """The workspace, grown to what a call needs (the status word is kept)."""
        n = ctypes.c_size_t(0)
        _check(_fn("bsa_cache_workspace_size")(self._c, budget, ctypes.byref(n)), "bsa_cache_workspace_size")
        if self._ws is None or self._ws.numel() < n.value:
            new = torch.empty(n.value, dtype=torch.uint8, device=self.device)
            if self._ws is None:
                new[:256].zero_()
            else:
                new[:256].copy_(self._ws[:256])
            self._ws = new
        return self._ws

    def _tokens(self, B, T, H, n_new, tree, scale):
        t = Tokens(B, T, H, self.H_kv, self.D, self._c.dtype)
        if scale is not None:
            t.scale = scale
        if B != self.B:
            raise ValueError(f"expected {self.B} sequences")
        if n_new is not None:
            t.n_new = _flat(n_new, "n_new", self.device, torch.int32, (B,))
        if tree is not None:
            t.tree = _flat(tree, "tree", self.device, torch.int64, (B, T))
        return t

    def append(self, k, v, q=None, rope=None, n_new=None, q_out=None):
        """The new tokens' k and v [B, T, H_kv, D] into the slots from
        ``length`` on (``length`` itself stays).  ``rope`` = (pos, inv_freq,
        axis, layout) rotates k on its way and q [B, T, H, D], which is returned
        (in ``q_out``).  ``n_new`` int32 [B]: only the first n_new[b] tokens of a
        sequence are stored."""
        if k.dim() != 4 or k.shape[2:] != (self.H_kv, self.D) or v.shape != k.shape:
            raise ValueError(f"k and v: expected [B, T, {self.H_kv}, {self.D}]")
        B, T = k.shape[:2]
        H = self.H_kv if q is None else q.shape[2]
        t = self._tokens(B, T, H, n_new, None, None)
        t.k_stride[:] = _rows(k, "k", self.device, self.dtype)
        t.v_stride[:] = _rows(v, "v", self.device, self.dtype)
        qp = qop = None
        if q is not None:
            if q.shape[:2] != (B, T) or q.shape[3] != self.D:
                raise ValueError("q must be [B, T, H, D] of the same tokens")
            q_out = _out_like(q, q_out, "q_out")
            t.q_stride[:] = _rows(q, "q", self.device, self.dtype)
            t.qo_stride[:] = _rows(q_out, "q_out", self.device, self.dtype)
            qp, qop = q.data_ptr(), q_out.data_ptr()
        r = None if rope is None else _rope_spec(B, T, self.D, self.device, *rope, inverse=False)
        _call("bsa_cache_append", self.device, self._c, t, r, qp, qop, k.data_ptr(), v.data_ptr(),
              self._ws.data_ptr(), self._ws.numel())
        return q_out

    def attend(self, q, tree=None, n_new=None, scale=None, out=None, lse=None):
        """(out, lse) of T <= 64 new tokens' queries [B, T, H, D] over the cache,
        which already holds the new tokens' keys (:meth:`append`).  Token t sees
        the slots below ``length`` and the new tokens of its word in ``tree``
        (int64 [B, T], :func:`tree_words`; None: a chain).  Rows at or past
        ``n_new`` are written as 0 / -inf."""
        if q.dim() != 4 or q.shape[3] != self.D:
            raise ValueError(f"q: expected [B, T, H, {self.D}]")
        B, T, H, _ = q.shape
        t = self._tokens(B, T, H, n_new, tree, scale)
        t.q_stride[:] = _rows(q, "q", self.device, self.dtype)
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else out
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
        t.qo_stride[:] = _rows(out, "out", self.device, self.dtype)
        if lse is None:
            lse = torch.empty(B, H, T, dtype=torch.float32, device=self.device)
        _call("bsa_cache_attend", self.device, self._c, t, q.data_ptr(), out.data_ptr(),
              _flat(lse, "lse", self.device, torch.float32, (B, H, T)), self._ws.data_ptr(), self._ws.numel())
        return out, lse

    def weigh(self, q, lse, scores, tree=None, n_new=None, scale=None, out=None):
        """Adds to ``scores`` (fp32 [B, H_kv, capacity]) the attention weight each
        slot took from these queries: exp(scale q.k - lse), summed over tokens and
        the query heads of the key head's group.  q, tree, n_new and scale as
        given to :meth:`attend`, lse as it returned.  In place, or into ``out``."""
        if q.dim() != 4 or q.shape[3] != self.D:
            raise ValueError(f"q: expected [B, T, H, {self.D}]")
        B, T, H, _ = q.shape
        t = self._tokens(B, T, H, n_new, tree, scale)
        t.q_stride[:] = _rows(q, "q", self.device, self.dtype)
        out = scores if out is None else out
        shape = (B, self.H_kv, self.capacity)
        _call("bsa_cache_weigh", self.device, self._c, t, q.data_ptr(),
              _flat(lse, "lse", self.device, torch.float32, (B, H, T)),
              _flat(scores, "scores", self.device, torch.float32, shape),
              _flat(out, "out", self.device, torch.float32, shape), self._ws.data_ptr(), self._ws.numel())
        return out

    def evict(self, scores, pos, next_pos, budget, sinks=0, recent=0, scores_out=None, pos_out=None,
              length_out=None):
        """Each head with more than ``budget`` slots keeps that many: the positions
        below ``sinks`` and from ``next_pos - recent`` on, then the highest
        ``scores``.  ``scores`` fp32 and ``pos`` int32 [B, H_kv, capacity],
        ``next_pos`` int32 [B].  Kept slots past the budget move into the dropped
        ones below it (K, V, score and pos); slots from the budget on get score 0
        and pos -1.  scores, pos and ``length`` change in place unless outputs
        are given, which are returned."""
        shape = (self.B, self.H_kv, self.capacity)
        scores_out = scores if scores_out is None else scores_out
        pos_out = pos if pos_out is None else pos_out
        length_out = self.length if length_out is None else length_out
        e = EvictSpec(int(budget), int(sinks), int(recent))
        e.next_pos = _flat(next_pos, "next_pos", self.device, torch.int32, (self.B,))
        e.score_in = _flat(scores, "scores", self.device, torch.float32, shape)
        e.pos_in = _flat(pos, "pos", self.device, torch.int32, shape)
        e.score_out = _flat(scores_out, "scores_out", self.device, torch.float32, shape)
        e.pos_out = _flat(pos_out, "pos_out", self.device, torch.int32, shape)
        e.length_out = _flat(length_out, "length_out", self.device, torch.int32, (self.B,))
        ws = self._workspace(max(e.budget, 0))
        _call("bsa_cache_evict", self.device, self._c, e, ws.data_ptr(), ws.numel())
        return scores_out, pos_out, length_out

    def status(self, clear=False):
        """The sticky device status of this cache's calls (0: ok; synchronises)."""
        return int(lib().bsa_get_device_status(self._ws.data_ptr(), self._ws.numel(),
                                               torch.cuda.current_stream(self.device).cuda_stream,
                                               1 if clear else 0))
