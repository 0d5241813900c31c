"""Rotary positions with several axes against the fp64 oracle: forward, backward
and the form that appends to a paged cache."""

import numpy as np
import pytest
import torch

import block_sparse_attention_map_b200 as bsa
from oracle import serving as oracle
from tests.serving_common import DT, HALF_STEP, Setup, f64, gen, normal

pytestmark = pytest.mark.gpu


def tables(n_pairs, n_axes, theta=10000.0):
    freq = np.array([theta ** (-k / max(1, n_pairs)) for k in range(n_pairs)])
    axis = np.arange(n_pairs) % n_axes
    return (torch.from_numpy(freq).cuda(), torch.from_numpy(axis.astype(np.int32)).cuda())


def check_rotated(y, x, ref, dtype):
    """The result rounded once (half a step of it, and fp16's subnormal half step),
    after fp32 sines (2^-21: sincospi within 2 ulp, the angle's rounding 2^-26
    turns) and fp32 products of the pair (bounded by the row's largest |x|)."""
    x = f64(x)
    m = np.abs(x).max(-1, keepdims=True) * 2
    tol = HALF_STEP[dtype] * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -21 * m + (2.0 ** -25 if dtype == "fp16" else 0)
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), float((err - tol).max())


CASES = [  # B, S, H, H_kv, D, n_axes, n_pairs, layout, dtype
    (1, 1, 1, 1, 64, 1, 32, "interleaved", "bf16"),
    (2, 37, 4, 2, 128, 3, 64, "interleaved", "bf16"),
    (2, 37, 4, 1, 128, 3, 64, "halves", "fp16"),
    (3, 129, 5, 5, 64, 2, 24, "halves", "bf16"),
    (1, 300, 3, 3, 64, 2, 13, "interleaved", "fp16"),
    (1, 17, 40, 8, 128, 3, 56, "halves", "bf16"),
    (1, 65, 2, 2, 256, 8, 128, "halves", "bf16"),
    (1, 9, 2, 1, 80, 2, 40, "interleaved", "bf16"),
    (1, 5, 3, 3, 16, 1, 8, "halves", "fp16"),
    (1, 40000, 1, 1, 128, 3, 64, "interleaved", "bf16"),  # more tokens than one step of the grid
    (2, 3000, 45, 3, 64, 2, 32, "halves", "bf16"),
]


@pytest.mark.parametrize("B,S,H,H_kv,D,n_axes,n_pairs,layout,dtype", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_oracle(B, S, H, H_kv, D, n_axes, n_pairs, layout, dtype, inverse):
    g = gen(B * 1000 + S)
    q, k = normal(g, (B, S, H, D), dtype), normal(g, (B, S, H_kv, D), dtype)
    pos = torch.randint(-50, 100000, (n_axes, B, S), generator=g, device="cuda").to(torch.int32)
    freq, axis = tables(n_pairs, n_axes)
    call = bsa.rope_bwd if inverse else bsa.rope
    yq, yk = call(q, k, pos, freq, axis, layout)
    args = (pos.cpu().numpy(), freq.cpu().numpy(), axis.cpu().numpy(), layout, inverse)
    check_rotated(yq, q, oracle.rope(f64(q), *args), dtype)
    check_rotated(yk, k, oracle.rope(f64(k), *args), dtype)
    # one of the two alone, and in place: the same bits
    only, none = call(q, None, pos, freq, axis, layout)
    assert none is None and torch.equal(only, yq)
    none, only = call(None, k, pos, freq, axis, layout)
    assert none is None and torch.equal(only, yk)
    q2, k2 = q.clone(), k.clone()
    call(q2, k2, pos, freq, axis, layout, q_out=q2, k_out=k2)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)


def test_far_positions_keep_the_angle():
    """Positions up to the int32 range: the angle is the fp64 product's, whose own
    rounding is 2^-53 of the angle (2^31 rad: 2.4e-7 rad)."""
    g = gen(1)
    q = normal(g, (1, 6, 2, 64), "fp16")
    pos = torch.tensor([[[0, 1, 2 ** 20 + 1, 2 ** 31 - 1, -(2 ** 31), -12345]]], dtype=torch.int32, device="cuda")
    freq, axis = tables(32, 1)
    y, _ = bsa.rope(q, None, pos, freq, axis)
    check_rotated(y, q, oracle.rope(f64(q), pos.cpu().numpy(), freq.cpu().numpy(), axis.cpu().numpy(), "interleaved"), "fp16")


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_gradient_is_the_transpose_and_matches_differences(layout):
    """<R x, y> = <x, R^T y> with R^T the backward, and the loss sum(y * R x)'s
    directional difference (R is linear: exact but for rounding)."""
    g = gen(3)
    B, S, H, D = 2, 33, 3, 64
    x, y, dx = (normal(g, (B, S, H, D), "fp16") for _ in range(3))
    pos = torch.randint(0, 5000, (2, B, S), generator=g, device="cuda").to(torch.int32)
    freq, axis = tables(32, 2)
    rx, _ = bsa.rope(x, None, pos, freq, axis, layout)
    gy, _ = bsa.rope_bwd(y, None, pos, freq, axis, layout)
    lhs, rhs = (f64(rx) * f64(y)).sum(), (f64(x) * f64(gy)).sum()
    # each output element is off by at most 2^-11 of itself and 2^-20 of its row
    bound = 2.0 ** -10.9 * (np.abs(f64(rx) * f64(y)).sum() + np.abs(f64(x) * f64(gy)).sum())
    assert abs(lhs - rhs) <= bound
    moved = (x.float() + 0.5 * dx.float()).half()
    step = f64(moved) - f64(x)
    rm, _ = bsa.rope(moved, None, pos, freq, axis, layout)
    diff = ((f64(rm) - f64(rx)) * f64(y)).sum()
    bound = 2.0 ** -10.9 * (np.abs(f64(rx) * f64(y)).sum() + np.abs(f64(rm) * f64(y)).sum() + np.abs(f64(gy) * step).sum())
    assert abs(diff - (f64(gy) * step).sum()) <= bound
    # and R^T R = 1
    back, _ = bsa.rope_bwd(rx, None, pos, freq, axis, layout)
    m = np.abs(f64(x)).max(-1, keepdims=True)
    assert (np.abs(f64(back) - f64(x)) <= 2.0 ** -11 * 4 * m).all()


def test_strided_inputs_and_outputs():
    """Heads inside a fused projection, a transposed order, and a broadcast batch of positions."""
    g = gen(4)
    B, S, H, D = 2, 50, 4, 64
    fused = normal(g, (B, S, 3 * H, D), "bf16")
    q, k = fused[:, :, :H], fused[:, :, H:2 * H]
    pos = torch.arange(S, device="cuda", dtype=torch.int32).expand(2, B, S)
    freq, axis = tables(32, 2)
    with pytest.raises(ValueError):
        bsa.rope(q, k, pos, freq, axis, "halves")
    pos = torch.arange(2 * S, device="cuda", dtype=torch.int32).view(2, 1, S).expand(2, B, S)
    out = torch.zeros(B, H, S, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    before = fused.clone()
    yq, yk = bsa.rope(q, k, pos, freq, axis, "halves", q_out=out)
    args = (pos.cpu().numpy(), freq.cpu().numpy(), axis.cpu().numpy(), "halves")
    check_rotated(yq, q, oracle.rope(f64(q), *args), "bf16")
    check_rotated(yk, k, oracle.rope(f64(k), *args), "bf16")
    bsa.rope(q, k, pos, freq, axis, "halves", q_out=q, k_out=k)  # in place inside the fused tensor
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(fused[:, :, 2 * H:], before[:, :, 2 * H:])


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_copied_elements_keep_their_bits(layout):
    """Elements past the rotated ones, and pairs of no axis, are copied, infinities and NaN too."""
    x = torch.full((1, 3, 2, 64), float("inf"), dtype=torch.bfloat16, device="cuda")
    x[:, :, :, ::3] = float("nan")
    pos = torch.full((1, 1, 3), 7, dtype=torch.int32, device="cuda")
    freq, axis = tables(16, 1)
    axis[:8] = -1
    axis[8:16] = 5
    y, _ = bsa.rope(x, None, pos, freq, axis, layout)
    assert torch.equal(y.view(torch.int16), x.view(torch.int16))
    freq[3] = float("nan")
    axis[:] = 0
    x = normal(gen(0), (1, 3, 2, 64), "bf16")
    y, _ = bsa.rope(x, None, pos, freq, axis, layout)
    i, j = (6, 7) if layout == "interleaved" else (3, 19)
    assert torch.equal(y[..., i], x[..., i]) and torch.equal(y[..., j], x[..., j])


@pytest.mark.parametrize("layout,dtype,D,page", [("halves", "bf16", 128, 16), ("interleaved", "fp16", 64, 64), (None, "bf16", 64, 8)])
def test_append_writes_its_slots_and_nothing_else(layout, dtype, D, page):
    st = Setup([5, 0, 130, 16], 9, 4, 2, D, page, dtype, seed=5, n_new=[9, 3, 0, 1], spare=20)
    k, v = normal(st.g, (4, 9, 2, D), dtype), normal(st.g, (4, 9, 2, D), dtype)
    freq, axis = tables(D // 2, 3)
    pos = torch.randint(0, 9000, (3, 4, 9), generator=st.g, device="cuda").to(torch.int32)
    want_k, want_v = st.k.clone(), st.v.clone()
    rk = bsa.rope(None, k, pos, freq, axis, layout)[1] if layout else k
    for b in range(4):
        for t in range(st.new[b]):
            s = st.lengths[b] + t
            at = (int(st.table_np[b][s // page]), s % page)
            want_k[at], want_v[at] = rk[b, t], v[b, t]
    cache = st.cache()
    q = cache.append(k, v, q=st.q if layout else None, rope=(pos, freq, axis, layout) if layout else None, n_new=st.n_new)
    assert torch.equal(st.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(st.v.view(torch.int16), want_v.view(torch.int16))
    if layout:
        assert torch.equal(q, bsa.rope(st.q, None, pos, freq, axis, layout)[0])
    assert cache.status() == 0 and st.length.tolist() == st.lengths


def test_append_of_a_long_prompt():
    st = Setup([3, 40], 300, 2, 2, 64, 32, seed=7, n_new=[300, 211], spare=10, tree=None)
    k, v = normal(st.g, (2, 300, 2, 64), "bf16"), normal(st.g, (2, 300, 2, 64), "bf16")
    cache = st.cache()
    cache.append(k, v, n_new=st.n_new)
    assert cache.status() == 0
    for b in range(2):
        s = np.arange(st.lengths[b], st.lengths[b] + st.new[b])
        at = torch.from_numpy(st.table_np[b][s // 32].astype(np.int64)).cuda(), torch.from_numpy(s % 32).cuda()
        assert torch.equal(st.k[at], k[b, :st.new[b]]) and torch.equal(st.v[at], v[b, :st.new[b]])


def test_append_past_the_capacity_or_a_bad_page_writes_nothing_there():
    st = Setup([5, 30], 4, 2, 2, 64, 8, seed=6)
    per = st.table.shape[1]
    k, v = normal(st.g, (2, 4, 2, 64), "bf16"), normal(st.g, (2, 4, 2, 64), "bf16")
    before = st.k.clone(), st.v.clone()
    st.length[:] = torch.tensor([per * 8 - 1, 16])
    st.table[1, 2] = st.k.shape[0] + 7
    cache = st.cache()
    cache.append(k, v)
    assert cache.status(clear=True) == 11 and cache.status() == 0
    last = int(st.table_np[0][per - 1])
    want_k, want_v = before
    want_k[last, 7], want_v[last, 7] = k[0, 0], v[0, 0]
    assert torch.equal(st.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(st.v.view(torch.int16), want_v.view(torch.int16))


def test_refusals():
    g = gen(8)
    q = normal(g, (1, 4, 2, 64), "bf16")
    pos = torch.zeros(1, 1, 4, dtype=torch.int32, device="cuda")
    freq, axis = tables(32, 1)
    for bad in (dict(layout="pairs"), dict(pos=pos.long()), dict(pos=pos[:, :, :3]), dict(freq=freq.float()),
                dict(axis=axis[:5]), dict(pos=pos.cpu()), dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]),
                dict(q=q.expand(1, 4, 2, 64)[:, :, :1].expand(1, 4, 2, 64)), dict(q_out=q[:, :, :, :32]),
                dict(q=q[:, :3], q_out=q[:, 1:], pos=pos[:, :, :3].contiguous())):
        a = dict(q=q, pos=pos, freq=freq, axis=axis, layout="halves", q_out=None)
        a.update(bad)
        with pytest.raises(ValueError):
            bsa.rope(a["q"], None, a["pos"], a["freq"], a["axis"], a["layout"], q_out=a["q_out"])
    with pytest.raises(bsa.BsaError) as e:  # more pairs than the head holds
        bsa.rope(q, None, pos, *tables(40, 1))
    assert e.value.code == 1
    with pytest.raises(bsa.BsaError) as e:  # halves take their pairs in eights
        bsa.rope(q, None, pos, *tables(12, 1), layout="halves")
    assert e.value.code == 2
    with pytest.raises(bsa.BsaError) as e:  # a row off the 16-byte grid
        bsa.rope(torch.zeros(4 * 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:513].view(1, 4, 2, 64), None, pos, freq, axis)
    assert e.value.code == 2


def test_outputs_across_each_other_are_refused_and_packed_ones_are_not():
    g = gen(9)
    pos = torch.arange(5, device="cuda", dtype=torch.int32).view(1, 1, 5)
    freq, axis = tables(32, 1)
    qk = normal(g, (1, 5, 6, 64), "bf16")
    q, k = qk[:, :, :3], qk[:, :, 3:]
    want = bsa.rope(q, k, pos, freq, axis)
    a, b, c = torch.empty_like(want[0]), torch.empty_like(want[0]), q.contiguous()
    for kw in (dict(q=q, k=k, q_out=k, k_out=q), dict(q=q, k=k, q_out=a, k_out=a), dict(q=c, k=b, q_out=b, k_out=a),
               dict(q=c, k=b, q_out=a, k_out=c)):
        with pytest.raises(ValueError):
            bsa.rope(kw["q"], kw["k"], pos, freq, axis, q_out=kw["q_out"], k_out=kw["k_out"])
    packed = torch.empty_like(qk)
    bsa.rope(q, k, pos, freq, axis, q_out=packed[:, :, :3], k_out=packed[:, :, 3:])
    bsa.rope(q, k, pos, freq, axis, q_out=q, k_out=k)
    for got in (packed, qk):
        assert torch.equal(got[:, :, :3], want[0]) and torch.equal(got[:, :, 3:], want[1])


def test_positions_that_sequences_or_axes_share():
    g = gen(10)
    q = normal(g, (3, 5, 2, 64), "bf16")
    row = torch.randint(0, 9000, (5,), generator=g, device="cuda", dtype=torch.int32)
    freq, axis = tables(32, 1)
    want = bsa.rope(q, None, row.expand(1, 3, 5).contiguous(), freq, axis)[0]
    assert torch.equal(bsa.rope(q, None, row.expand(1, 3, 5), freq, axis)[0], want)
    f2, a2 = tables(32, 2)
    want = bsa.rope(q[:1], None, row.expand(2, 1, 5).contiguous(), f2, a2)[0]
    assert torch.equal(bsa.rope(q[:1], None, row.expand(2, 1, 5), f2, a2)[0], want)
    two = torch.stack([row, row + 7])
    for pos in (two[:, None].expand(2, 3, 5), two[None].expand(2, 2, 5)):
        x = q[:pos.shape[1]]
        assert torch.equal(bsa.rope(x, None, pos, f2, a2)[0], bsa.rope(x, None, pos.contiguous(), f2, a2)[0])
    with pytest.raises(ValueError):
        bsa.rope(q, None, row.expand(2, 3, 5), f2, a2)


def test_empty_calls_do_nothing():
    freq, axis = tables(32, 1)
    for B, S in ((0, 4), (2, 0)):
        q = torch.empty(B, S, 2, 64, dtype=torch.bfloat16, device="cuda")
        n = bsa.launch_count()
        y, _ = bsa.rope(q, None, torch.empty(1, B, S, dtype=torch.int32, device="cuda"), freq, axis)
        assert y.shape == q.shape and bsa.launch_count() == n


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_far_positions_of_fast_pairs_keep_the_angle(layout):
    """Frequencies from far below to far above a turn a position, at positions up to
    the int32 range, against angles reduced in 60 decimal digits (fp64's own product
    is off by up to 2^-8 rad here): as exact at 2^31 - 1 as at 1."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097493")
    g = gen(11)
    q = normal(g, (1, 9, 2, 64), "fp16")
    places = [0, 1, -1, 7, 2 ** 20 + 1, -(2 ** 24) - 3, 2 ** 31 - 1, -(2 ** 31), 1999999973]
    freqs = [1.0, 1e-9, -1e-9, 0.3, -0.7, 6.2, 6.283185307179586, 7.0, 100.0, -123.456, 9999.99, 1e4, 12345.678, -1e6 / 7, 2.0 ** 40 / 3, 1e15]
    freq = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    axis = torch.zeros(16, dtype=torch.int32, device="cuda")
    y, _ = bsa.rope(q, None, torch.tensor([[places]], dtype=torch.int32, device="cuda"), freq, axis, layout)
    back, _ = bsa.rope_bwd(y, None, torch.tensor([[places]], dtype=torch.int32, device="cuda"), freq, axis, layout)
    angle = np.array([[float(Decimal(p) * Decimal(f) % turn) for f in freqs] for p in places])[None, :, None]
    for x, got, s in ((f64(q), y, 1.0), (f64(y), back, -1.0)):
        ref = np.array(x)
        i, j = (slice(0, 32, 2), slice(1, 32, 2)) if layout == "interleaved" else (slice(0, 16), slice(16, 32))
        a, b = np.array(x[..., i]), np.array(x[..., j])
        ref[..., i], ref[..., j] = a * np.cos(angle) - s * b * np.sin(angle), s * a * np.sin(angle) + b * np.cos(angle)
        check_rotated(got, torch.from_numpy(x), ref, "fp16")
