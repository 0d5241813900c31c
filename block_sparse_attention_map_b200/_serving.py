"""Positions and the paged cache: rotary positions with several axes (forward,
backward, and into a cache), attention of drafted tokens over a paged key/value
cache, and eviction from it by accumulated attention weight.

Argument marshalling only, like the rest of the binding: every step runs in the
library's CUDA kernels (include/bsa.h), on the current stream of the tensors'
device.  Wrong arguments raise ValueError here or BsaError from the library."""

from __future__ import annotations

import ctypes
import math
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


def _call(name, index, stream, *args):
    """One library call on this stream of device ``index``, with the device current."""
    fn = _FNS.get(name) or _fn(name)
    if index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        raise BsaError(rc, name)


def _int32(x, name):
    """An int that the library's int32 holds (ctypes would drop the bits above)."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


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
        # zeros would mean contiguous to the library; an axis or sequence there is one of may have any stride
        if shape[0] > 1 and B > 1:
            raise ValueError("pos: give every axis or every sequence its own rows (one row for all is not taken)")
        r.pos_stride[0 if shape[0] == 1 else 1] = 1
    return r


def _check_tables(pos, inv_freq, axis, index):
    """The rotation's tensors, but for the shape of ``pos``."""
    if pos.dtype != torch.int32 or pos.get_device() != index:
        raise ValueError(f"pos: expected an int32 tensor on cuda:{index}")
    if inv_freq.dtype != torch.float64 or inv_freq.get_device() != index or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq: expected a contiguous float64 tensor on cuda:{index}")
    if axis.dtype != torch.int32 or axis.get_device() != index or not axis.is_contiguous():
        raise ValueError(f"axis: expected a contiguous int32 tensor on cuda:{index}")


def _rope_args(proto, pos, inv_freq, axis):
    r = RopeSpec.from_buffer_copy(proto)
    r.inv_freq, r.axis, r.pos = inv_freq.data_ptr(), axis.data_ptr(), pos.data_ptr()
    return r


def _apart_rules(xs, xt, ys, yt):
    """Where a tensor and another one of these shapes and strides share no element
    although their spans overlap (head ranges of one fused tensor, say): the outer
    strides of both are multiples of a period, the inner extents of both fit it, and
    within it they lie apart.  A (period, extent, other's extent) a way to split them."""
    if 0 in xs or 0 in ys:
        return ()
    x, y = ([(st, n) for st, n in zip(t, s) if n > 1] for s, t in ((xs, xt), (ys, yt)))
    rules = []
    for cut in sorted({st for st, _ in x + y if st > 1}):
        period = math.gcd(*(st for st, _ in x + y if st >= cut))
        ex, ey = (1 + sum((n - 1) * st for st, n in z if st < cut) for z in (x, y))
        if ex + ey <= period:
            rules.append((period, ex, ey))
    return tuple(rules)


def _overlap(a, span_a, b, span_b, rules):
    """Whether tensors at addresses ``a`` and ``b`` may share an element."""
    if a >= b + 2 * span_b or b >= a + 2 * span_a:
        return False
    for period, ea, eb in rules:
        at = (b - a) // 2 % period
        if ea <= at <= period - eb:
            return False
    return True


def _check_apart(a, b, same, span_x, span_out, rules, name):
    """An output at address ``b`` is its input at ``a`` itself (``same`` strides) or shares no element with it."""
    if not (a == b and same) and _overlap(a, span_x, b, span_out, rules):
        raise ValueError(f"{name}: overlaps an input without being it")


def _check_flat(a, b, nbytes, name):
    """As :func:`_check_apart` for two contiguous tensors of one size."""
    if a < b + nbytes and b < a + nbytes and a != b:
        raise ValueError(f"{name}: overlaps an input without being it")


def _pair_layout(xs, xt, os, ot, name):
    """A rotation's input and output: (strides, output's strides, whether they are alike, spans, when they are apart)."""
    if len(xs) != 4 or os != xs:
        raise ValueError(f"{name} and {name}_out: expected [B, S, H, D] tensors of one shape")
    same = all(a == b for a, b, n in zip(xt, ot, xs) if n > 1)
    return (_strides(xs, xt, name), _strides(os, ot, name + "_out"), same, _span(xs, xt), _span(os, ot),
            _apart_rules(xs, xt, os, ot))


def _rotate_layout(qs, qt, qos, qot, ks, kt, kos, kot, ps, pt, fs, axs, dtype, layout, inverse):
    """A rotation's argument blocks, but for the addresses, its inputs' and outputs' spans, and
    when k and q_out, q and k_out, and the outputs are apart."""
    xs = qs if qs is not None else ks
    if len(xs) != 4:
        raise ValueError("q and k are [B, S, H, D] tensors")
    B, S, H, D = xs
    t = Tokens(B, S, H, 0, D, dtype)
    q = k = None
    if qs is not None:
        q = _pair_layout(qs, qt, qos, qot, "q")
        t.q_stride[:], t.qo_stride[:] = q[0], q[1]
    if ks is not None:
        k = _pair_layout(ks, kt, kos, kot, "k")
        if ks[0] != B or ks[1] != S or ks[3] != D:
            raise ValueError("q and k must share B, S and D")
        t.H_kv = ks[2]
        t.k_stride[:], t.ko_stride[:] = k[0], k[1]
    if len(fs) != 1 or axs != fs:
        raise ValueError("inv_freq and axis: expected one entry a pair")
    cross = None
    if q is not None and k is not None:
        cross = _apart_rules(ks, kt, qos, qot), _apart_rules(qs, qt, kos, kot), _apart_rules(qos, qot, kos, kot)
    return t, _rope_layout(B, S, ps, pt, fs[0], layout, inverse), q and q[2:], k and k[2:], cross


def _rotate(q, k, pos, inv_freq, axis, layout, inverse, q_out, k_out):
    x = q if q is not None else k
    if x is None:
        raise ValueError("give q, k or both")
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("q_out without q, or k_out without k")
    kind, index = x.dtype, x.get_device()
    if index < 0 or kind not in DTYPE:
        raise ValueError("q and k are [B, S, H, D] bf16 or fp16 CUDA tensors")
    qs = qt = qos = qot = ks = kt = kos = kot = qp = qop = kp = kop = None
    for y in (q, k, q_out, k_out):
        if y is not None and (y.dtype != kind or y.get_device() != index):
            raise ValueError(f"q, k and their outputs: expected {kind} tensors on cuda:{index}")
    _check_tables(pos, inv_freq, axis, index)
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=kind, device=q.device)
        qs, qt, qos, qot = q.shape, q.stride(), q_out.shape, q_out.stride()
        qp, qop = q.data_ptr(), q_out.data_ptr()
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=kind, device=k.device)
        ks, kt, kos, kot = k.shape, k.stride(), k_out.shape, k_out.stride()
        kp, kop = k.data_ptr(), k_out.data_ptr()
    args = (qs, qt, qos, qot, ks, kt, kos, kot, pos.shape, pos.stride(), inv_freq.shape, axis.shape, DTYPE[kind], layout,
            inverse)
    t, r, qa, ka, cross = _layout(args, lambda: _rotate_layout(*args))
    if qa is not None:
        _check_apart(qp, qop, *qa, "q_out")
    if ka is not None:
        _check_apart(kp, kop, *ka, "k_out")
    if cross is not None:
        # (in place, q and k may lie side by side in one tensor, and so may the outputs)
        if _overlap(kp, ka[1], qop, qa[2], cross[0]):
            raise ValueError("q_out: overlaps k")
        if _overlap(qp, qa[1], kop, ka[2], cross[1]):
            raise ValueError("k_out: overlaps q")
        if _overlap(qop, qa[2], kop, ka[2], cross[2]):
            raise ValueError("q_out and k_out overlap")
    _call("bsa_rope", index, _stream_of(index), t, _rope_args(r, pos, inv_freq, axis), qp, qop, kp, kop)
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
    its children).  A token sees its ancestors and itself.  Made on the host: a call
    waits for ``parents`` and cannot be captured into a graph; a captured step takes
    the words as an input."""
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


def _append_layout(ks, kt, vs, vt, qs, qt, qos, qot, ps, pt, fs, axs, layout, B, H_kv, D, dtype):
    """An append's argument blocks, but for the addresses, the spans of q and its output, and the
    spans of k and v with when they are apart from that output."""
    if len(ks) != 4 or ks[0] != B or ks[2] != H_kv or ks[3] != D or vs != ks:
        raise ValueError(f"k and v: expected [{B}, T, {H_kv}, {D}]")
    T = ks[1]
    t = Tokens(B, T, H_kv, H_kv, D, dtype)
    t.k_stride[:], t.v_stride[:] = _strides(ks, kt, "k"), _strides(vs, vt, "v")
    q = r = None
    cross = None
    if qs is not None:
        q = _pair_layout(qs, qt, qos, qot, "q")
        cross = tuple((_span(s, st), _apart_rules(s, st, qos, qot)) for s, st in ((ks, kt), (vs, vt)))
        if qs[0] != B or qs[1] != T or qs[3] != D:
            raise ValueError("q must be [B, T, H, D] of the same tokens")
        t.H = qs[2]
        t.q_stride[:], t.qo_stride[:] = q[0], q[1]
    if ps is not None:
        if len(fs) != 1 or axs != fs:
            raise ValueError("inv_freq and axis: expected one entry a pair")
        r = _rope_layout(B, T, ps, pt, fs[0], layout, False)
    return t, r, q and q[2:], cross


class CacheWorkspace:
    """Scratch memory and the sticky status word of paged caches' calls.  Caches
    whose calls all follow one another on one stream (the layers of a model) may
    share one; it grows to what the largest call needs.  A captured graph goes on
    with the memory it was captured with, which the workspace keeps: keep the
    workspace (or a PagedCache that has it) as long as the graph."""

    def __init__(self, device):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("workspace: expected a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.bufs, self.ptr, self.nbytes = [], None, 0  # the last buffer is the one in use
        self.streams = set()                            # that it is in use on

    def grow(self, nbytes):
        """At least ``nbytes``."""
        if nbytes <= self.nbytes:
            return
        with torch.cuda.device(self.device):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the workspace cannot grow while a stream is captured: reserve() before the capture")
            nbytes = max(nbytes, 2 * self.nbytes)  # so that those that are kept are less than the one in use
            new = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            new[:256].zero_()
        self.bufs.append(new)
        self.ptr, self.nbytes, self.streams = new.data_ptr(), nbytes, {_stream_of(self.device.index)}

    def use(self, stream):
        """The current stream, of this handle, uses the memory from now on."""
        self.bufs[-1].record_stream(torch.cuda.current_stream(self.device))
        self.streams.add(stream)

    def status(self, clear):
        with torch.cuda.device(self.device):
            stream = _stream_of(self.device.index)
            found = [int(lib().bsa_get_device_status(x.data_ptr(), x.numel(), stream, 1 if clear else 0))
                     for x in reversed(self.bufs)]
        return next((x for x in found if x != 0), 0)


def _held(i, name):
    """A tensor whose address the library holds: another cannot take its place (``x.length += 1`` works in place)."""
    def keep(self, value):
        if value is not self._tensors[i]:
            raise ValueError(f"{name}: change the tensor in place, or make another PagedCache")
    return property(lambda self: self._tensors[i], keep)


class PagedCache:
    """A paged key/value cache and the calls around it.

    ``k``, ``v`` [n_pages, page_size, H_kv, D] (bf16 or fp16, the head dimension
    contiguous), ``page_table`` int32 [B, max_pages] (rows that hold the same pages
    are fine, a row broadcast over the sequences is not), ``length`` int32 [B]: the
    slots in use.  Slot s of sequence b is row s mod page_size of page
    page_table[b, s // page_size].  The tensors are kept, not copied: change
    ``length`` in place as tokens are accepted.  Only :meth:`append` and
    :meth:`evict` write the cache, in place.

    The calls of one PagedCache share a workspace (its own, or the ``workspace``
    given), so they belong on one stream at a time; use a PagedCache (over the
    same tensors) and workspace for each stream, and for each captured graph that
    may run beside another.  :meth:`reserve` before a capture that evicts."""

    def __init__(self, k, v, page_table, length, workspace: Optional[CacheWorkspace] = None):
        if not k.is_cuda or k.dim() != 4 or k.dtype not in DTYPE:
            raise ValueError("k and v are [n_pages, page_size, H_kv, D] bf16 or fp16 CUDA tensors")
        if v.shape != k.shape:
            raise ValueError("v must have k's shape")
        self.device, self.dtype, self._index = k.device, k.dtype, k.get_device()
        _rows(v, "v", self._index, self.dtype)
        self._tensors = k, v, page_table, length
        self.n_pages, self.page_size, self.H_kv, self.D = k.shape
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.get_device() != self._index or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table: expected int32 [B, max_pages] on the cache's device, contiguous rows")
        self.B, self.max_pages = page_table.shape
        if self.B > 1 and page_table.stride(0) < self.max_pages:
            # (0 would mean contiguous rows to the library, which would read past a broadcast row's end)
            raise ValueError("page_table: every sequence needs a row of its own memory (one row for all is not taken)")
        self.capacity = self.max_pages * self.page_size
        c = self._c = Cache(self.n_pages, self.page_size, self.H_kv, self.D, DTYPE[self.dtype], self.B, self.max_pages)
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.k_stride[:] = _strides(k.shape, k.stride(), "k")
        c.v_stride[:] = _strides(v.shape, v.stride(), "v")
        c.page_table = page_table.data_ptr()
        c.table_stride = page_table.stride(0) if self.B > 1 else 0
        c.length = _flat(length, "length", self._index, torch.int32, (self.B,))
        self.workspace = CacheWorkspace(self.device) if workspace is None else workspace
        if self.workspace.device != self.device:
            raise ValueError("workspace: on another device")
        self.reserve(0)

    k = _held(0, "k")
    v = _held(1, "v")
    page_table = _held(2, "page_table")
    length = _held(3, "length")

    def reserve(self, budget):
        """Grows the workspace to what evictions to ``budget`` or less need."""
        n = ctypes.c_size_t(0)
        budget = _int32(budget, "budget")
        _check(_fn("bsa_cache_workspace_size")(self._c, budget, ctypes.byref(n)), "bsa_cache_workspace_size")
        self.workspace.grow(n.value)

    def _run(self, name, *args):
        """A library call on the cache, on the current stream."""
        ws, stream = self.workspace, _stream_of(self._index)
        if stream not in ws.streams:
            ws.use(stream)
        _call(name, self._index, stream, self._c, *args, ws.ptr, ws.nbytes)

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
            if not 0.0 < t.scale < math.inf:  # (the library would take 1/sqrt(D))
                raise ValueError(f"scale: expected a positive finite number of 32 bits, got {scale}")
        return t, _span(shape, stride), _span(out_shape, out_stride), _apart_rules(shape, stride, out_shape, out_stride)

    def _queries(self, q, out, tree, n_new, scale):
        """The argument block of q [B, T, H, D] and its options, checked."""
        shape, stride, out_shape, out_stride = q.shape, q.stride(), out.shape, out.stride()
        proto, span_q, span_out, rules = _layout(
            ("t", shape, stride, out_shape, out_stride, scale, self.B, self.H_kv, self.D, self._c.dtype),
            lambda: self._token_layout(shape, stride, out_shape, out_stride, scale))
        t = Tokens.from_buffer_copy(proto)
        if out is not q:  # the rows of one token are written while others' are still to be read
            _check_apart(q.data_ptr(), out.data_ptr(), False, span_q, span_out, rules, "out")
        if q.dtype != self.dtype or q.get_device() != self._index:
            raise ValueError(f"q: expected a {self.dtype} tensor on cuda:{self._index}")
        if n_new is not None:
            t.n_new = _flat(n_new, "n_new", self._index, torch.int32, (self.B,))
        if tree is not None:
            t.tree = _flat(tree, "tree", self._index, torch.int64, shape[:2])
        return t

    def append(self, k, v, q=None, rope=None, n_new=None, q_out=None):
        """The new tokens' k and v [B, T, H_kv, D] into the slots from
        ``length`` on (``length`` itself stays).  ``rope`` = (pos, inv_freq,
        axis, layout) rotates k on its way and q [B, T, H, D], which is returned
        (in ``q_out``).  ``n_new`` int32 [B]: only the first n_new[b] tokens of a
        sequence are stored."""
        index, kind = self._index, self.dtype
        for y in (k, v, q, q_out):
            if y is not None and (y.dtype != kind or y.get_device() != index):
                raise ValueError(f"k, v, q and q_out: expected {kind} tensors on cuda:{index}")
        qs = qt = qos = qot = ps = pt = fs = axs = layout = qp = qop = r = None
        if q is None and q_out is not None:
            raise ValueError("q_out without q")
        if q is not None:
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=kind, device=self.device)
            qs, qt, qos, qot = q.shape, q.stride(), q_out.shape, q_out.stride()
            qp, qop = q.data_ptr(), q_out.data_ptr()
        if rope is not None:
            pos, inv_freq, axis, layout = rope
            _check_tables(pos, inv_freq, axis, index)
            ps, pt, fs, axs = pos.shape, pos.stride(), inv_freq.shape, axis.shape
        args = (k.shape, k.stride(), v.shape, v.stride(), qs, qt, qos, qot, ps, pt, fs, axs, layout, self.B, self.H_kv, self.D,
                self._c.dtype)
        proto, rp, qa, cross = _layout(args, lambda: _append_layout(*args))
        kp, vp = k.data_ptr(), v.data_ptr()
        t = Tokens.from_buffer_copy(proto)
        if n_new is not None:
            t.n_new = _flat(n_new, "n_new", index, torch.int32, (self.B,))
        if qa is not None:
            _check_apart(qp, qop, *qa, "q_out")
            for p, (span, rules), name in ((kp, cross[0], "k"), (vp, cross[1], "v")):
                if _overlap(p, span, qop, qa[2], rules):
                    raise ValueError(f"q_out: overlaps {name}")
        if rp is not None:
            r = _rope_args(rp, pos, inv_freq, axis)
        self._run("bsa_cache_append", t, r, qp, qop, kp, vp)
        return q_out

    def attend(self, q, tree=None, n_new=None, scale=None, out=None, lse=None):
        """(out, lse) of T <= 64 new tokens' queries [B, T, H, D] over the cache,
        which already holds the new tokens' keys (:meth:`append`); out does not
        overlap q.  Token t sees
        the slots below ``length`` and the new tokens of its word in ``tree``
        (int64 [B, T], :func:`tree_words`; None: a chain).  Rows at or past
        ``n_new`` are written as 0 / -inf.  ``scale`` > 0; None: 1/sqrt(D)."""
        if out is None:
            out = torch.empty(q.shape, dtype=self.dtype, device=self.device)
        elif out is q:
            raise ValueError("out: overlaps q")
        t = self._queries(q, out, tree, n_new, scale)
        if out.dtype != self.dtype or out.get_device() != self._index:
            raise ValueError(f"out: expected a {self.dtype} tensor on cuda:{self._index}")
        B, T, H, _ = q.shape
        if lse is None:
            lse = torch.empty(B, H, T, dtype=torch.float32, device=self.device)
        self._run("bsa_cache_attend", t, q.data_ptr(), out.data_ptr(), _flat(lse, "lse", self._index, torch.float32, (B, H, T)))
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
        score_out = score_in
        if out is not None:
            score_out = _flat(out, "out", self._index, torch.float32, shape)
            _check_flat(score_in, score_out, 4 * out.numel(), "out")
        self._run("bsa_cache_weigh", t, q.data_ptr(), _flat(lse, "lse", self._index, torch.float32, (B, H, T)), score_in,
                  score_out)
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
        e = EvictSpec(_int32(budget, "budget"), _int32(sinks, "sinks"), _int32(recent, "recent"))
        index = self._index
        e.next_pos = _flat(next_pos, "next_pos", index, torch.int32, (self.B,))
        e.score_in = _flat(scores, "scores", index, torch.float32, shape)
        e.pos_in = _flat(pos, "pos", index, torch.int32, shape)
        e.score_out = e.score_in if scores_out is scores else _flat(scores_out, "scores_out", index, torch.float32, shape)
        e.pos_out = e.pos_in if pos_out is pos else _flat(pos_out, "pos_out", index, torch.int32, shape)
        e.length_out = _flat(length_out, "length_out", index, torch.int32, (self.B,))
        nbytes = 4 * self.B * self.H_kv * self.capacity
        if nbytes > 0:  # (an address of 0 reads as None)
            if scores_out is not scores:
                _check_flat(e.score_in, e.score_out, nbytes, "scores_out")
            if pos_out is not pos:
                _check_flat(e.pos_in, e.pos_out, nbytes, "pos_out")
            if length_out is not self.length:
                _check_flat(self._c.length, e.length_out, 4 * self.B, "length_out")
                if abs(e.length_out - e.next_pos) < 4 * self.B:
                    raise ValueError("length_out: overlaps next_pos")
        try:
            self._run("bsa_cache_evict", e)
        except BsaError as x:
            if x.code != 3:  # too small a workspace, found before anything is launched
                raise
            self.reserve(e.budget)
            self._run("bsa_cache_evict", e)
        return scores_out, pos_out, length_out

    def status(self, clear=False):
        """The sticky device status of this cache's calls (0: ok; synchronises)."""
        return self.workspace.status(clear)
