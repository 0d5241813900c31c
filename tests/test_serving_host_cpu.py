"""What the binding of the positions and the paged cache checks before it calls
the library, without a GPU: CPU tensors stand in for CUDA ones, and the call
itself is recorded instead of made."""

import itertools
import random

import pytest
import torch

from block_sparse_attention_map_b200 import _binding as bd
from block_sparse_attention_map_b200 import _serving as sv


class OnCuda:
    """A CPU tensor that says it is on cuda:0."""

    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, at):
        return OnCuda(self.t[at])


class Workspace:
    device, ptr, nbytes, streams = torch.device("cuda", 0), 4096, 1 << 30, {0}

    def grow(self, nbytes):
        pass


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The names of the library calls that got past the checks."""
    import os
    if not os.path.exists(bd.LIB_PATH):
        from block_sparse_attention_map_b200 import build
        build.build()
    made = []
    monkeypatch.setattr(sv, "_call", lambda name, *args: made.append(name))
    monkeypatch.setattr(sv, "_stream_of", lambda index: 0)
    return made


def pages(n=8, page=16, H_kv=2, D=64):
    return OnCuda(torch.zeros(n, page, H_kv, D, dtype=torch.bfloat16))


def paged(table=None, B=3, **kw):
    k = pages(**kw)
    if table is None:
        table = torch.zeros(B, 4, dtype=torch.int32)
    length = OnCuda(torch.zeros(table.shape[0], dtype=torch.int32))
    return sv.PagedCache(k, pages(**kw), OnCuda(table), length, workspace=Workspace())


def test_a_page_table_whose_rows_share_memory_is_refused():
    """A stride of 0 between sequences would mean contiguous rows to the library,
    which would read the second sequence's pages past the table's end."""
    row = torch.zeros(4, dtype=torch.int32)
    for table in (row.expand(3, 4), row[:1].expand(3, 1), torch.zeros(9, dtype=torch.int32).as_strided((3, 4), (1, 1)),
                  torch.zeros(9, dtype=torch.int32).as_strided((2, 4), (3, 1))):
        with pytest.raises(ValueError, match="page_table"):
            paged(table)
    wide = torch.zeros(3, 9, dtype=torch.int32)
    for table, stride in ((torch.zeros(3, 4, dtype=torch.int32), 4), (wide[:, 2:6], 9), (row.expand(1, 4), 0),
                          (torch.zeros(3, 1, dtype=torch.int32), 1), (wide[:, :1], 9)):
        assert paged(table)._c.table_stride == stride


def spec(S, B=1):
    return (OnCuda(torch.zeros(1, B, S, dtype=torch.int32)), OnCuda(torch.zeros(32, dtype=torch.float64)),
            OnCuda(torch.zeros(32, dtype=torch.int32)))


def fused(heads, B=2, S=5):
    return OnCuda(torch.zeros(B, S, heads, 64, dtype=torch.bfloat16))


def test_a_rotation_in_place_over_the_others_memory_is_refused(calls):
    """q rotated in place while k is read from (part of) the same memory, or both
    outputs over one another: what is read or kept would go by the order of threads."""
    x, p = fused(6), spec(5, 2)
    head = slice(None), slice(None)
    q, k = x[(*head, slice(0, 3))], x[(*head, slice(2, 5))]
    apart = fused(3), fused(3)
    for args, kw in (((x, x), dict(q_out=x, k_out=fused(6))), ((x, x), dict(q_out=fused(6), k_out=x)),
                     ((q, k), dict(q_out=q, k_out=apart[0])), ((q, k), dict(q_out=q, k_out=k)),
                     ((q, k), dict(q_out=apart[0], k_out=k)), (apart, dict(q_out=q, k_out=k)),
                     (apart, dict(q_out=x[(*head, slice(0, 3))], k_out=x[(*head, slice(0, 3))]))):
        with pytest.raises(ValueError):
            sv.rope(*args, *p, **kw)
    assert calls == []
    k = x[(*head, slice(3, 6))]
    sv.rope(q, k, *p, q_out=q, k_out=k)
    sv.rope(*apart, *p, q_out=q, k_out=k)
    sv.rope(x, x, *p, q_out=fused(6), k_out=fused(6))  # read twice
    assert len(calls) == 3


def test_an_append_in_place_over_its_k_or_v_is_refused(calls):
    cache, x, p = paged(B=2), fused(6), spec(5, 2)
    at = lambda a: x[:, :, a:a + 2]  # noqa: E731
    for k, v in ((at(0), at(2)), (at(2), at(0)), (at(1), at(4)), (at(4), at(1))):
        with pytest.raises(ValueError):
            cache.append(k, v, q=at(0), rope=(*p, "halves"), q_out=at(0))
    assert calls == []
    cache.append(at(2), at(4), q=at(0), rope=(*p, "halves"), q_out=at(0))
    cache.append(at(2), at(2), q=at(0), rope=(*p, "halves"), q_out=at(0))
    assert len(calls) == 2


def test_overlap_is_found_for_any_strides():
    """Against the elements themselves: never apart where an element is shared, and
    apart for head, token and batch ranges of fused tensors in any order of dimensions."""
    rng = random.Random(0)
    shared = found = 0
    for _ in range(4000):
        views = []
        for _ in range(2):
            shape = [rng.choice([1, 1, 2, 3, 4]) for _ in range(3)] + [rng.choice([1, 4])]
            order, stride, at = rng.sample(range(3), 3), [0, 0, 0, 1], shape[3]
            for d in order:
                stride[d] = at * rng.choice([1, 1, 1, 2, 3])
                at = stride[d] * shape[d]
            views.append((shape, stride, rng.randrange(0, 60)))
        (xs, xt, x0), (ys, yt, y0) = views
        cells = [{o + sum(i * st for i, st in zip(ix, t)) for ix in itertools.product(*map(range, s))} for s, t, o in views]
        truth = bool(cells[0] & cells[1])
        got = sv._overlap(2 * x0 + 96, sv._span(xs, xt), 2 * y0 + 96, sv._span(ys, yt), sv._apart_rules(xs, xt, ys, yt))
        assert got or not truth, views
        shared, found = shared + truth, found + (not got)
    assert shared > 500 and found > 500
    big = torch.zeros(4, 6, 8, 64)
    for order in itertools.permutations(range(3)):
        x = big.permute(*order, 3)
        for d, n in enumerate(x.shape[:3]):
            a, b = x.narrow(d, 0, n // 2), x.narrow(d, n // 2, n - n // 2)
            for p, q in ((a, b), (b, a), (x.narrow(d, 0, 1), x.narrow(d, n - 1, 1))):
                rules = sv._apart_rules(p.shape, p.stride(), q.shape, q.stride())
                # (the elements of `big` as 16-bit ones)
                at = [2 * y.storage_offset() for y in (p, q)]
                assert not sv._overlap(at[0], sv._span(p.shape, p.stride()), at[1], sv._span(q.shape, q.stride()), rules)


def test_an_output_beside_its_input_in_one_tensor_is_taken(calls):
    x, p = fused(8), spec(5, 2)
    at = lambda a: x[:, :, a:a + 2]  # noqa: E731
    sv.rope(at(0), at(2), *p, q_out=at(4), k_out=at(6))
    cache = paged(B=2)
    cache.append(at(0), at(2), q=at(4), rope=(*p, "halves"), q_out=at(6))
    lse, tree = OnCuda(torch.zeros(2, 2, 5)), OnCuda(torch.zeros(2, 5, dtype=torch.int64))
    cache.attend(at(0), tree=tree, out=at(2), lse=lse)
    # in place through a view whose strides differ where there is one of a dimension
    one = OnCuda(torch.zeros(1, 5, 1, 64, dtype=torch.bfloat16))
    again = OnCuda(one.t.as_strided((1, 5, 1, 64), (64, 64, 128, 1)))
    sv.rope(one, None, *spec(5), q_out=again)
    assert calls == ["bsa_rope", "bsa_cache_append", "bsa_cache_attend", "bsa_rope"]
    for call in (lambda: sv.rope(at(0), None, *p, q_out=x[:, :, 1:3]), lambda: cache.attend(at(0), out=x[:, :, 1:3], lse=lse),
                 lambda: cache.attend(at(0), out=at(0), lse=lse), lambda: sv.rope(x[:, :4, :2], None, *spec(4, 2), q_out=x[:, 1:, :2])):
        with pytest.raises(ValueError):
            call()
    assert len(calls) == 4


@pytest.mark.parametrize("scale", [0, 0.0, -0.125, float("nan"), float("inf"), 1e-50, 1e39])
def test_a_scale_that_is_not_positive_and_finite_is_refused(scale, calls):
    """The library would take 1/sqrt(D) in its place (None says so here)."""
    cache, q = paged(B=2), fused(2, S=3)
    lse, scores = OnCuda(torch.zeros(2, 2, 3)), OnCuda(torch.zeros(2, 2, cache.capacity))
    with pytest.raises(ValueError, match="scale"):
        cache.attend(q, out=fused(2, S=3), lse=lse, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        cache.weigh(q, lse, scores, scale=scale)
    assert calls == []
    for good in (None, 0.125, 3, 1e-30):
        cache.attend(q, out=fused(2, S=3), lse=lse, scale=good)
        cache.weigh(q, lse, scores, scale=good)
    assert len(calls) == 8


def test_an_output_without_its_input_is_refused(calls):
    """It would come back as it was given, unwritten."""
    x, p, cache = fused(2), spec(5, 2), paged(B=2)
    for call in (lambda: sv.rope(x, None, *p, q_out=fused(2), k_out=fused(2)), lambda: sv.rope(None, x, *p, q_out=fused(2), k_out=fused(2)),
                 lambda: sv.rope_bwd(x, None, *p, q_out=fused(2), k_out=fused(2)), lambda: cache.append(x, x, q_out=fused(2))):
        with pytest.raises(ValueError, match="without"):
            call()
    assert calls == []
