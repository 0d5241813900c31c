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


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(index):
    """The handle of the current stream of device ``index``."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _call(name, index, *args):
    """One library call on the current stream of device ``index``, with it current."""
    fn = _FNS.get(name) or _fn(name)
    if index == torch.cuda.current_device():
        rc = fn(*args, _stream_of(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream_of(index))
    if rc != 0:
        raise BsaError(rc, name)


def _strides(shape, stride, name):
    """The (batch, token, head) strides of a [B, S, H, D] tensor for the library."""
    if stride[3] != 1 and shape[3] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    if 0 in shape:
        return (0, 0, 0)
    for st, n in zip(stride[:3], shape):
        if st == 0 and n > 1:
            raise ValueError(f"{name}: a broadcast dimension (stride 0) is not taken")
    # the stride of a dimension of one says nothing; the library wants a valid one
    return tuple(st if n > 1 else 8 * -(-max(st, shape[3]) // 8) for st, n in zip(stride[:3], shape))


def _rows(t, name, index, dtype):
    """Checks a [B, S, H, D] tensor of this type on device ``index``."""
    if t.dim() != 4 or t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{name}: expected a [B, S, H, D] {dtype} tensor on cuda:{index}")


def _flat(t, name, index, dtype, shape):
    """A contiguous tensor of exactly this type and shape on device ``index``; its address."""
    if t.dtype != dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


# Argument blocks by layout (shapes, strides, options; no addresses): filled and
# checked once, then copied for each call.
_LAYOUTS: dict = {}


def _layout(key, make):
    x = _LAYOUTS.get(key)
    if x is None:
        x = make()
        if len(_LAYOUTS) >= 4096:
            _LAYOUTS.clear()
        _LAYOUTS[key] = x
    return x


def _span(shape, stride):
    """Elements from a tensor's first to one past its last."""
    return 0 if 0 in shape else 1 + sum((n - 1) * s for n, s in zip(shape, stride))


def _rope_layout(B, T, shape, stride, n, layout, inverse):
    """The rotation's argument block, but for its addresses."""
    if layout not in LAYOUT:
        raise ValueError(f"layout: one of {sorted(LAYOUT)}")
    if len(shape) != 3 or shape[1:] != (B, T) or (T > 1 and stride[2] != 1):
        raise ValueError(f"pos: expected [n_axes, {B}, {T}], contiguous in the tokens")
    r = RopeSpec(shape[0], n, LAYOUT[layout], 1 if inverse else 0)
    r.pos_stride[:] = stride[:2]
    if stride[0] == 0 and stride[1] == 0 and shape[0] * B > 1:
        raise ValueError("pos: give every axis or sequence its row (a fully broadcast pos is not taken)")
    return r


def _rope_spec(B, T, index, pos, inv_freq, axis, layout, inverse):
    ps, pt, n = pos.shape, pos.stride(), inv_freq.numel()
    proto = _layout(("r", B, T, ps, pt, n, layout, inverse), lambda: _rope_layout(B, T, ps, pt, n, layout, inverse))
    if pos.dtype != torch.int32 or pos.get_device() != index:
        raise ValueError(f"pos: expected an int32 tensor on cuda:{index}")
    r = RopeSpec.from_buffer_copy(proto)
    r.inv_freq = _flat(inv_freq, "inv_freq", index, torch.float64, (n,))
    r.axis = _flat(axis, "axis", index, torch.int32, (n,))
    r.pos = pos.data_ptr()
    return r


def _check_apart(x, xs, out, os, span_x, span_out, name):
    """``out`` is ``x`` itself or shares no memory with it."""
    a, b, e = x.data_ptr(), out.data_ptr(), x.element_size()
    if a < b + span_out * e and b < a + span_x * e and not (a == b and xs == os):
        raise ValueError(f"{name}: overlaps its input without being it")


def _pair_layout(xs, xt, os, ot, name):
    """Strides and spans of a rotation's input and output."""
    if os != xs:
        raise ValueError(f"{name}_out: expected the input's shape {tuple(xs)}")
    return _strides(xs, xt, name), _strides(os, ot, name + "_out"), _span(xs, xt), _span(os, ot)


def _pair(x, out, name, index, dtype):
    """A rotation's input and output (new where None), checked: (out, their layout)."""
    _rows(x, name, index, dtype)
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=x.device)
    _rows(out, name + "_out", index, dtype)
    xs, xt, os, ot = x.shape, x.stride(), out.shape, out.stride()
    lay = _layout(("p", xs, xt, os, ot), lambda: _pair_layout(xs, xt, os, ot, name))
    _check_apart(x, xt, out, ot, lay[2], lay[3], name + "_out")
    return out, lay


def _rotate(q, k, pos, inv_freq, axis, layout, inverse, q_out, k_out):
    x = q if q is not None else k
    if x is None:
        raise ValueError("give q, k or both")
    dtype = DTYPE.get(x.dtype)
    if not x.is_cuda or x.dim() != 4 or dtype is None:
        raise ValueError("q and k are [B, S, H, D] bf16 or fp16 CUDA tensors")
    index = x.get_device()
    B, S, H, D = x.shape
    t = Tokens(B, S, H, 0, D, dtype)
    qp = qop = kp = kop = None
    if q is not None:
        q_out, lay = _pair(q, q_out, "q", index, x.dtype)
        t.q_stride[:], t.qo_stride[:] = lay[0], lay[1]
        qp, qop = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        k_out, lay = _pair(k, k_out, "k", index, x.dtype)
        ks = k.shape
        if ks[0] != B or ks[1] != S or ks[3] != D:
            raise ValueError("q and k must share B, S and D")
        t.H_kv = ks[2]
        t.k_stride[:], t.ko_stride[:] = lay[0], lay[1]
        kp, kop = k.data_ptr(), k_out.data_ptr()
    r = _rope_spec(B, S, index, pos, inv_freq, axis, layout, inverse)
    _call("bsa_rope", index, t, r, qp, qop, kp, kop)
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
        self.device, self.dtype, self._index = k.device, k.dtype, k.get_device()
        _rows(v, "v", self._index, self.dtype)
        self.k, self.v, self.page_table, self.length = k, v, page_table, length
        self.n_pages, self.page_size, self.H_kv, self.D = k.shape
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.get_device() != self._index or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table: expected int32 [B, max_pages] on the cache's device, contiguous rows")
        self.B, self.max_pages = page_table.shape
        self.capacity = self.max_pages * self.page_size
        c = self._c = Cache(self.n_pages, self.page_size, self.H_kv, self.D, DTYPE[self.dtype], self.B, self.max_pages)
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.k_stride[:] = _strides(k.shape, k.stride(), "k")
        c.v_stride[:] = _strides(v.shape, v.stride(), "v")
        c.page_table = page_table.data_ptr()
        c.table_stride = page_table.stride(0) if self.B > 1 else 0
        c.length = _flat(length, "length", self._index, torch.int32, (self.B,))
        self._ws = None
        self._workspace(0)

    def _workspace(self, budget):
        """The workspace, grown to what an eviction to ``budget`` needs (the status word is kept)."""
        n = ctypes.c_size_t(0)
        _check(_fn("bsa_cache_workspace_size")(self._c, budget, ctypes.byref(n)), "bsa_cache_workspace_size")
        if self._ws is None or self._ws_bytes < n.value:
            new = torch.empty(n.value, dtype=torch.uint8, device=self.device)
            if self._ws is None:
                new[:256].zero_()
            else:
                new[:256].copy_(self._ws[:256])
            self._ws, self._ws_ptr, self._ws_bytes = new, new.data_ptr(), n.value

    def _token_layout(self, shape, stride, out_shape, out_stride, scale):
        if len(shape) != 4 or shape[3] != self.D:
            raise ValueError(f"q: expected [B, T, H, {self.D}]")
        if shape[0] != self.B:
            raise ValueError(f"expected {self.B} sequences")
        if out_shape != shape:
            raise ValueError("out must have q's shape")
        t = Tokens(shape[0], shape[1], shape[2], self.H_kv, self.D, self._c.dtype)
        t.q_stride[:] = _strides(shape, stride, "q")
        t.qo_stride[:] = _strides(out_shape, out_stride, "out")
        if scale is not None:
            t.scale = scale
        return t

    def _queries(self, q, out, tree, n_new, scale):
        """The argument block of q [B, T, H, D] and its options, checked."""
        shape, stride, out_shape, out_stride = q.shape, q.stride(), out.shape, out.stride()
        t = Tokens.from_buffer_copy(_layout(
            ("t", shape, stride, out_shape, out_stride, scale, self.B, self.H_kv, self.D, self._c.dtype),
            lambda: self._token_layout(shape, stride, out_shape, out_stride, scale)))
        if q.dtype != self.dtype or q.get_device() != self._index:
            raise ValueError(f"q: expected a {self.dtype} tensor on cuda:{self._index}")
        self._options(t, shape[0], shape[1], tree, n_new)
        return t

    def _options(self, t, B, T, tree, n_new):
        if n_new is not None:
            t.n_new = _flat(n_new, "n_new", self._index, torch.int32, (B,))
        if tree is not None:
            t.tree = _flat(tree, "tree", self._index, torch.int64, (B, T))

    def append(self, k, v, q=None, rope=None, n_new=None, q_out=None):
        """The new tokens' k and v [B, T, H_kv, D] into the slots from
        ``length`` on (``length`` itself stays).  ``rope`` = (pos, inv_freq,
        axis, layout) rotates k on its way and q [B, T, H, D], which is returned
        (in ``q_out``).  ``n_new`` int32 [B]: only the first n_new[b] tokens of a
        sequence are stored."""
        _rows(k, "k", self._index, self.dtype)
        _rows(v, "v", self._index, self.dtype)
        ks, vs = k.shape, v.shape
        if ks[2] != self.H_kv or ks[3] != self.D or vs != ks or ks[0] != self.B:
            raise ValueError(f"k and v: expected [{self.B}, T, {self.H_kv}, {self.D}]")
        kt, vt = k.stride(), v.stride()
        B, T = ks[0], ks[1]
        t = Tokens(B, T, self.H_kv, self.H_kv, self.D, self._c.dtype)
        t.k_stride[:], t.v_stride[:] = _layout(("kv", ks, kt, vt), lambda: (_strides(ks, kt, "k"), _strides(vs, vt, "v")))
        self._options(t, B, T, None, n_new)
        qp = qop = None
        if q is not None:
            q_out, lay = _pair(q, q_out, "q", self._index, self.dtype)
            qs = q.shape
            if qs[0] != B or qs[1] != T or qs[3] != self.D:
                raise ValueError("q must be [B, T, H, D] of the same tokens")
            t.H = qs[2]
            t.q_stride[:], t.qo_stride[:] = lay[0], lay[1]
            qp, qop = q.data_ptr(), q_out.data_ptr()
        r = None
        if rope is not None:
            pos, inv_freq, axis, layout = rope
            r = _rope_spec(B, T, self._index, pos, inv_freq, axis, layout, False)
        _call("bsa_cache_append", self._index, self._c, t, r, qp, qop, k.data_ptr(), v.data_ptr(), self._ws_ptr,
              self._ws_bytes)
        return q_out

    def attend(self, q, tree=None, n_new=None, scale=None, out=None, lse=None):
        """(out, lse) of T <= 64 new tokens' queries [B, T, H, D] over the cache,
        which already holds the new tokens' keys (:meth:`append`).  Token t sees
        the slots below ``length`` and the new tokens of its word in ``tree``
        (int64 [B, T], :func:`tree_words`; None: a chain).  Rows at or past
        ``n_new`` are written as 0 / -inf."""
        if out is None:
            out = torch.empty(q.shape, dtype=self.dtype, device=self.device)
        t = self._queries(q, out, tree, n_new, scale)
        if out.dtype != self.dtype or out.get_device() != self._index:
            raise ValueError(f"out: expected a {self.dtype} tensor on cuda:{self._index}")
        B, T, H, _ = q.shape
        if lse is None:
            lse = torch.empty(B, H, T, dtype=torch.float32, device=self.device)
        _call("bsa_cache_attend", self._index, self._c, t, q.data_ptr(), out.data_ptr(),
              _flat(lse, "lse", self._index, torch.float32, (B, H, T)), self._ws_ptr, self._ws_bytes)
        return out, lse

    def weigh(self, q, lse, scores, tree=None, n_new=None, scale=None, out=None):
        """Adds to ``scores`` (fp32 [B, H_kv, capacity]) the attention weight each
        slot took from these queries: exp(scale q.k - lse), summed over tokens and
        the query heads of the key head's group.  q, tree, n_new and scale as
        given to :meth:`attend`, lse as it returned.  In place, or into ``out``."""
        t = self._queries(q, q, tree, n_new, scale)
        B, T, H, _ = q.shape
        shape = (B, self.H_kv, self.capacity)
        score_in = _flat(scores, "scores", self._index, torch.float32, shape)
        score_out = score_in if out is None else _flat(out, "out", self._index, torch.float32, shape)
        _call("bsa_cache_weigh", self._index, self._c, t, q.data_ptr(),
              _flat(lse, "lse", self._index, torch.float32, (B, H, T)), score_in, score_out, self._ws_ptr, self._ws_bytes)
        return scores if out is None else out

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
        index = self._index
        e.next_pos = _flat(next_pos, "next_pos", index, torch.int32, (self.B,))
        e.score_in = _flat(scores, "scores", index, torch.float32, shape)
        e.pos_in = _flat(pos, "pos", index, torch.int32, shape)
        e.score_out = e.score_in if scores_out is scores else _flat(scores_out, "scores_out", index, torch.float32, shape)
        e.pos_out = e.pos_in if pos_out is pos else _flat(pos_out, "pos_out", index, torch.int32, shape)
        e.length_out = _flat(length_out, "length_out", index, torch.int32, (self.B,))
        if e.budget > 0:
            self._workspace(e.budget)
        _call("bsa_cache_evict", index, self._c, e, self._ws_ptr, self._ws_bytes)
        return scores_out, pos_out, length_out

    def status(self, clear=False):
        """The sticky device status of this cache's calls (0: ok; synchronises)."""
        with torch.cuda.device(self._index):
            return int(lib().bsa_get_device_status(self._ws_ptr, self._ws_bytes, _stream_of(self._index), 1 if clear else 0))
