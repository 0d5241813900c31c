"""The paged cache's attention, weighing and eviction against the fp64 oracle,
and a serving loop of them together."""

import math

import numpy as np
import pytest
import torch

import block_sparse_attention_map_b200 as bsa
from oracle import serving as oracle
from tests.serving_common import DT, HALF_STEP, Setup, attend_tolerance, exponent_tolerance, f64, gen, normal

pytestmark = pytest.mark.gpu


def words(st):
    return oracle.words_or_chain(None if st.tree is None else st.tree.tolist(), st.B, st.T)


def check_attend(st, out, lse):
    seq_k, seq_v = st.seqs(), st.seqs(st.v)
    O, L, mass = oracle.attend(f64(st.q), seq_k, seq_v, st.lengths, st.new, words(st), st.scale)
    n = max(a + b for a, b in zip(st.lengths, st.new))
    vmax = max((np.abs(np.nan_to_num(v)).max(initial=0.0) for v in seq_v), default=0.0)
    err = np.abs(f64(out) - O)
    tol = attend_tolerance(O, mass, n, vmax, st.dtype)
    assert (err <= tol).all(), (float(err.max()), float((err - tol).max()))
    got = f64(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(L))
    fin = np.isfinite(L)
    e = exponent_tolerance(f64(st.q), seq_k, st.scale)
    assert (np.abs(got[fin] - L[fin]) <= e + 1e-6).all(), float(np.abs(got[fin] - L[fin]).max())
    return L


ATTEND = [  # lengths, T, H, H_kv, D, page, dtype, n_new, tree
    ([0], 1, 1, 1, 64, 8, "bf16", None, None),
    ([1], 1, 4, 2, 128, 16, "fp16", None, "random"),
    ([127, 128, 129], 1, 4, 4, 64, 64, "bf16", None, None),
    ([255, 0, 256, 300], 1, 8, 2, 128, 128, "bf16", None, None),
    ([100, 3, 61, 250], 7, 6, 2, 128, 32, "fp16", [7, 1, 0, 5], "random"),
    ([511, 512, 513, 77], 16, 4, 1, 64, 256, "bf16", [16, 15, 16, 2], "random"),
    ([640, 9], 64, 5, 1, 128, 16, "bf16", None, "random"),
    ([200, 383], 64, 16, 2, 64, 8, "fp16", [63, 64], "random"),
    ([1000, 1500], 32, 8, 1, 128, 64, "bf16", None, None),
    ([70], 33, 7, 1, 128, 1024, "bf16", None, "random"),
    ([2500, 17, 900], 3, 40, 8, 128, 64, "bf16", [3, 3, 2], "random"),
    ([130, 2], 2, 128, 1, 64, 32, "bf16", None, "random"),
    ([600], 5, 100, 1, 128, 32, "fp16", None, "random"),
    ([20000], 2, 4, 1, 64, 64, "bf16", None, "random"),   # a run a tile or two: every SM has a piece of the same rows
    ([6000, 1], 40, 8, 1, 64, 128, "bf16", [40, 3], "random"),  # two row tiles and one, many pieces
]


@pytest.mark.parametrize("lengths,T,H,H_kv,D,page,dtype,n_new,tree", ATTEND)
def test_attend_matches_oracle(lengths, T, H, H_kv, D, page, dtype, n_new, tree):
    st = Setup(lengths, T, H, H_kv, D, page, dtype, seed=T + H, n_new=n_new, tree=tree)
    cache = st.cache()
    out, lse = cache.attend(st.q, st.tree, st.n_new)
    assert cache.status() == 0
    check_attend(st, out, lse)
    again, lse2 = cache.attend(st.q, st.tree, st.n_new)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lengths,T,H,H_kv,D,page,dtype,n_new,tree", ATTEND)
def test_weigh_matches_oracle(lengths, T, H, H_kv, D, page, dtype, n_new, tree):
    st = Setup(lengths, T, H, H_kv, D, page, dtype, seed=T + H, n_new=n_new, tree=tree)
    cache = st.cache()
    _, L, _ = oracle.attend(f64(st.q), st.seqs(), st.seqs(st.v), st.lengths, st.new, words(st), st.scale)
    lse = torch.from_numpy(L).float().cuda()
    scores = torch.rand(st.B, H_kv, cache.capacity, generator=st.g, device="cuda")
    out = torch.full_like(scores, 7.0)
    assert cache.weigh(st.q, lse, scores, st.tree, st.n_new, out=out) is out
    assert cache.status() == 0
    want = oracle.weigh(f64(scores), f64(st.q), st.seqs(), f64(lse), st.lengths, st.new, words(st), st.scale)
    e = exponent_tolerance(f64(st.q), st.seqs(), st.scale)
    for b in range(st.B):
        n = st.lengths[b] + st.new[b]
        w = want[b, :, :n]
        # each weight is off by the factor exp(+-e), and rows * 2^-23 of it in the sum; the score's own rounding 2^-23
        tol = (w - f64(scores)[b, :, :n]) * (2 * e + T * (H // H_kv) * 2.0 ** -23) + 2.0 ** -23 * w + 1e-12
        err = np.abs(f64(out)[b, :, :n] - w)
        assert (err <= tol).all(), float((err - tol).max())
        assert (out[b, :, n:] == 7.0).all()
    first = out.clone()
    cache.weigh(st.q, lse, scores, st.tree, st.n_new)  # in place
    for b in range(st.B):
        n = st.lengths[b] + st.new[b]
        assert torch.equal(scores[b, :, :n], first[b, :, :n])


@pytest.mark.parametrize("T,G", [(1, 4), (24, 4), (64, 8)])
def test_what_a_row_does_not_see_never_reaches_it(T, G):
    """A drafted token whose key and value are NaN, infinite or the type's lowest
    value: the rows that do not see it give the bits they give without it, and the
    rows that see it are not finite."""
    st = Setup([150, 90], T, 2 * G, 2, 128, 32, seed=9, tree="random")
    ref_out, ref_lse = st.cache().attend(st.q, st.tree)
    sees = np.array([[[(w >> j) & 1 for j in range(T)] for w in row] for row in words(st)], dtype=bool)
    for j in {0, T // 2, T - 1}:
        for bad in (math.nan, math.inf, -math.inf):
            k, v = st.k.clone(), st.v.clone()
            for b in range(2):
                s = st.lengths[b] + j
                at = (int(st.table_np[b][s // 32]), s % 32)
                v[at][:, ::3] = bad
                v[at][:, 1::3] = torch.finfo(torch.bfloat16).min
                k[at][:, 5] = bad
            out, lse = bsa.PagedCache(k, v, st.table, st.length).attend(st.q, st.tree)
            for b in range(2):
                for t in range(T):
                    if not sees[b, t, j]:
                        assert torch.equal(out[b, t], ref_out[b, t]) and torch.equal(lse[b, :, t], ref_lse[b, :, t])
            # the value alone, the key fine: the seen infinities and NaN come through
            out, _ = bsa.PagedCache(st.k, v, st.table, st.length).attend(st.q, st.tree)
            for b in range(2):
                for t in range(T):
                    if sees[b, t, j]:
                        got = out[b, t, :, ::3]
                        assert torch.isnan(got).all() if math.isnan(bad) else torch.equal(got, torch.full_like(got, bad))
                    else:
                        assert torch.equal(out[b, t], ref_out[b, t])


@pytest.mark.parametrize("T", [1, 5])
def test_many_sequences_of_any_length(T):
    """More sequences than a warp scans at once, most of them short or empty."""
    rng = np.random.default_rng(T)
    lengths = [int(rng.integers(0, 900)) if rng.random() < 0.3 else int(rng.integers(0, 3)) for _ in range(77)]
    new = [int(rng.integers(0, T + 1)) for _ in range(77)]
    st = Setup(lengths, T, 2, 1, 64, 16, seed=50 + T, n_new=new)
    cache = st.cache()
    out, lse = cache.attend(st.q, st.tree, st.n_new)
    L = check_attend(st, out, lse)
    scores = torch.zeros(77, 1, cache.capacity, device="cuda")
    cache.weigh(st.q, torch.from_numpy(L).float().cuda(), scores, st.tree, st.n_new)
    assert cache.status() == 0
    seen = np.isfinite(L).sum((1, 2))  # every row that sees something spreads a weight of 1
    assert np.allclose(scores.sum((1, 2)).cpu().numpy(), seen, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("B,T,H,H_kv,D,page,keys,dtype", [
    (16, 24, 16, 4, 128, 128, 9000, "bf16"),   # one row tile
    (2, 64, 40, 8, 128, 256, 30000, "bf16"),   # two row tiles and one
    (2, 64, 32, 4, 64, 64, 30000, "fp16"),     # two row tiles twice
    (12, 1, 16, 4, 128, 16, 7000, "fp16"),     # a few rows
    (24, 9, 8, 8, 64, 32, 3000, "bf16"),       # many pieces a CTA
])
def test_long_ragged_batches_again_and_again(B, T, H, H_kv, D, page, keys, dtype):
    """The whole GPU busy with sequences that end inside tiles, forty times without
    a wait between: every pass the same bits, and the values of the plain form."""
    rng = np.random.default_rng(keys)
    lengths = [int(keys - rng.integers(0, keys // 2)) for _ in range(B)]
    new = [max(1, T - int(rng.integers(0, 4))) for _ in range(B)]
    st = Setup(lengths, T, H, H_kv, D, page, dtype, seed=keys, n_new=new)
    caches = [st.cache() for _ in range(2)]
    runs = [caches[i % 2].attend(st.q, st.tree, st.n_new) for i in range(40)]
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    scores = torch.zeros(B, H_kv, caches[0].capacity, device="cuda")
    weights = [caches[0].weigh(st.q, runs[0][1], scores, st.tree, st.n_new, out=torch.zeros_like(scores)) for _ in range(20)]
    assert all(torch.equal(w, weights[0]) for w in weights[1:])
    assert caches[0].status() == 0 and caches[1].status() == 0
    u, G = HALF_STEP[dtype], H // H_kv
    for b in range(B):
        n, m = lengths[b], new[b]
        s = torch.arange(n + m, device="cuda")
        at = st.table[b].long()[s // page], s % page
        k, v, q = st.k[at].double(), st.v[at].double(), st.q[b, :m].double()
        bits = (st.tree[b, :m, None] >> torch.arange(m, device="cuda")) & 1
        seen = torch.cat((torch.ones(m, n, device="cuda"), bits), 1).bool()
        x = torch.einsum("tkgd,jkd->tkgj", q.view(m, H_kv, G, D), k) * st.scale
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        z = torch.logsumexp(x, -1)
        p = torch.exp(x - z[..., None])
        O = torch.einsum("tkgj,jkd->tkgd", p, v).reshape(m, H, D)
        # the rounded weights' errors are independent: 8 of their standard deviations (u / sqrt 3 of sqrt(sum (p v)^2))
        # and the common factor of the rounded sum, the result's own half step, and 2^-17 of the weights for fp32
        spread = torch.einsum("tkgj,jkd->tkgd", p * p, v * v).sqrt().reshape(m, H, D)
        norm = (p * p).sum(-1).sqrt().reshape(m, H, 1)
        tol = 8 * u / 3 ** 0.5 * (spread + norm * O.abs()) + u * O.abs() + 2.0 ** -17 * v.abs().max() + \
            ((n + m) * 2.0 ** -25 if dtype == "fp16" else 0)
        err = (runs[0][0][b, :m].double() - O).abs()
        assert (err <= tol).all(), (b, float((err - tol).max()))
        assert (runs[0][0][b, m:] == 0).all()
        w = (p * seen[:, None, None]).sum((0, 2)).T.float()
        got = weights[0][b, :, :n + m].T
        assert torch.allclose(got, w, rtol=2e-4, atol=1e-6)


def test_a_cache_past_32_bits():
    """Element offsets of K and V past 2^32: a few pages at the far end of a large cache."""
    st = Setup([700, 90], 3, 4, 2, 128, 64, seed=60, spare=30)
    n = (1 << 32) // (64 * 2 * 128) + 40
    k = torch.empty(n, 64, 2, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    used = st.k.shape[0]
    k[n - used:], v[n - used:] = st.k, st.v
    far = bsa.PagedCache(k, v, st.table + (n - used), st.length)
    near = st.cache()
    out, lse = far.attend(st.q, st.tree)
    want = near.attend(st.q, st.tree)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    sc = torch.rand(2, 2, near.capacity, generator=st.g, device="cuda")
    pos = torch.arange(near.capacity, dtype=torch.int32, device="cuda").expand(2, 2, -1).contiguous()
    far_sc, far_pos = sc.clone(), pos.clone()
    for c, s, p in ((near, sc, pos), (far, far_sc, far_pos)):
        c.weigh(st.q, lse, s, st.tree)
    assert torch.equal(sc, far_sc)
    nk, nv = normal(st.g, (2, 3, 2, 128), "bf16"), normal(st.g, (2, 3, 2, 128), "bf16")
    nxt = torch.tensor([5000, 5000], dtype=torch.int32, device="cuda")
    far.append(nk, nv)
    near.append(nk, nv)
    far_len = st.length.clone()
    near.evict(sc, pos, nxt, 300, length_out=torch.empty_like(far_len))
    far.evict(far_sc, far_pos, nxt, 300, length_out=far_len)
    assert torch.equal(sc, far_sc) and torch.equal(pos, far_pos) and far_len.tolist() == [300, 90]
    assert torch.equal(k[n - used:].view(torch.int16), st.k.view(torch.int16))
    assert torch.equal(v[n - used:].view(torch.int16), st.v.view(torch.int16))
    assert far.status() == 0


def test_words_that_leave_rows_empty_and_bits_past_the_new_tokens():
    st = Setup([0, 40, 0], 4, 4, 2, 64, 16, seed=10, n_new=[4, 3, 2], tree=None)
    w = torch.full((3, 4), -1, dtype=torch.int64, device="cuda")  # every bit: more than there are
    w[:, 1] = 0                                                   # sees no new token
    st.tree = w
    cache = st.cache()
    out, lse = cache.attend(st.q, w, st.n_new)
    L = check_attend(st, out, lse)
    assert np.isneginf(L[0, :, 1]).all() and (out[0, 1] == 0).all() and np.isfinite(L[1, :, 1]).all()
    scores = torch.zeros(3, 2, cache.capacity, device="cuda")
    cache.weigh(st.q, lse, scores, w, st.n_new)
    total = scores.sum((1, 2)).cpu().numpy()
    assert np.allclose(total, [3 * 4, 3 * 4, 1 * 4], rtol=1e-5)  # every row that sees something spreads a weight of 1


@pytest.mark.parametrize("T,H,H_kv,lengths", [(1, 2, 2, [300]), (16, 20, 2, [300, 40]), (64, 10, 2, [513, 0])])
def test_rows_whose_lse_is_minus_infinity_weigh_nothing_whatever_they_hold(T, H, H_kv, lengths):
    st = Setup(lengths, T, H, H_kv, 64, 16, seed=30 + T)
    cache = st.cache()
    _, lse = cache.attend(st.q, st.tree)
    off = torch.rand(lse.shape, generator=st.g, device="cuda") < 0.3
    off[0, -1] = True  # a whole head
    lse = lse.masked_fill(off, -math.inf)
    rows = off.transpose(1, 2)[..., None]
    plain, odd = st.q.masked_fill(rows, 0.0), st.q.masked_fill(rows, math.nan)
    odd[..., 1::2] = odd[..., 1::2].masked_fill(rows, math.inf)
    scores = torch.rand(st.B, H_kv, cache.capacity, generator=st.g, device="cuda")
    a, b = torch.empty_like(scores), torch.empty_like(scores)
    cache.weigh(plain, lse, scores, st.tree, out=a)
    cache.weigh(odd, lse, scores, st.tree, out=b)
    want = oracle.weigh(f64(scores), f64(plain), st.seqs(), f64(lse), st.lengths, st.new, words(st), st.scale)
    e = exponent_tolerance(f64(plain), st.seqs(), st.scale)
    for i in range(st.B):
        n = st.lengths[i] + st.new[i]
        assert torch.equal(a[i, :, :n], b[i, :, :n])
        w = want[i, :, :n]
        tol = (w - f64(scores)[i, :, :n]) * (2 * e + T * (H // H_kv) * 2.0 ** -23) + 2.0 ** -23 * w + 1e-12
        assert (np.abs(f64(b)[i, :, :n] - w) <= tol).all()


def test_strided_tensors_another_scale_and_a_shared_page():
    st = Setup([70, 75], 5, 4, 2, 64, 16, seed=11)
    big = torch.full((st.k.shape[0], 2, 2, 16, 192), math.nan, dtype=torch.bfloat16, device="cuda")
    big[:, 0, :, :, :64] = st.k.transpose(1, 2)
    big[:, 1, :, :, 64:128] = st.v.transpose(1, 2)
    k, v = big[:, 0, :, :, :64].transpose(1, 2), big[:, 1, :, :, 64:128].transpose(1, 2)
    table = torch.full((2, 40), 12345, dtype=torch.int32, device="cuda")[:, 3:3 + st.table.shape[1]]
    table.copy_(st.table)
    table[1, :4] = table[0, :4]  # a common prefix
    st.table_np[1, :4] = st.table_np[0, :4]
    q = torch.zeros(2, 5, 9, 64, dtype=torch.bfloat16, device="cuda")[:, :, 2:6]
    q.copy_(st.q)
    out = torch.full((2, 4, 5, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    st.scale = 0.3
    got, lse = bsa.PagedCache(k, v, table, st.length).attend(q, st.tree, scale=0.3, out=out.transpose(1, 2)[..., :64])
    check_attend(st, got, lse)
    assert (out[..., 64:] == 3.0).all()


def test_large_scores_rescale():
    """Scores that grow along the cache by far more than the exponent's range."""
    st = Setup([1000, 700], 2, 4, 2, 64, 64, seed=12)
    with torch.no_grad():
        st.k *= 8
        st.q *= 8
    for b in range(2):
        for s in range(st.lengths[b]):
            st.k[int(st.table_np[b][s // 64]), s % 64] *= 0.1 + 0.9 * s / 1000
    out, lse = st.cache().attend(st.q, st.tree)
    O, L, mass = oracle.attend(f64(st.q), st.seqs(), st.seqs(st.v), st.lengths, st.new, words(st), st.scale)
    e = exponent_tolerance(f64(st.q), st.seqs(), st.scale, np.abs(L).max())
    assert (np.abs(f64(lse) - L) <= e).all()
    tol = attend_tolerance(O, mass, 1002, 6.0, "bf16") + 2 * e * mass
    assert (np.abs(f64(out) - O) <= tol).all()


def test_bad_lengths_and_pages_are_reported_and_read_as_zeros():
    st = Setup([100, 40, 60], 2, 4, 2, 64, 16, seed=13)
    cap = st.table.shape[1] * 16
    cache = st.cache()
    ref, _ = cache.attend(st.q)
    st.table[1, 1] = -3
    out, lse = cache.attend(st.q)
    assert cache.status(clear=True) == 11
    assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    st.k[int(st.table_np[1][1])] = 0
    st.v[int(st.table_np[1][1])] = 0
    st.table[1, 1] = int(st.table_np[1][1])
    want, wlse = cache.attend(st.q)
    assert torch.equal(out, want) and torch.equal(lse, wlse) and cache.status() == 0
    st.length[2] = -5
    st.lengths[2] = 0
    out, _ = cache.attend(st.q)
    assert cache.status(clear=True) == 11 and torch.equal(out[0], ref[0])
    st.length[2] = cap + 9  # no room for the new tokens: every row of it is a row of none
    out, lse = cache.attend(st.q)
    assert cache.status(clear=True) == 11 and (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    n = torch.tensor([2, 3, -1], dtype=torch.int32, device="cuda")
    st.length[2] = 60
    out, lse = cache.attend(st.q, n_new=n)
    assert cache.status(clear=True) == 11 and torch.equal(out[0], ref[0]) and (out[2] == 0).all()


# ------------------------------------------------------------------ eviction

def evict_setup(lengths, H_kv, page, dtype="bf16", seed=0, D=64):
    st = Setup(lengths, 0, H_kv, H_kv, D, page, dtype, seed=seed)
    cap = st.table.shape[1] * page
    rng = np.random.default_rng(seed)
    score = np.round(rng.standard_normal((st.B, H_kv, cap)).astype(np.float32) ** 2 * 8) / 8  # many equal ones
    pos = np.stack([[rng.permutation(cap) for _ in range(H_kv)] for _ in range(st.B)]).astype(np.int32)
    return st, torch.from_numpy(score).cuda(), torch.from_numpy(pos).cuda()


def check_evict(st, before, score, pos, next_pos, budget, sinks, recent, score_out, pos_out, length_out, marks):
    k0, v0 = before
    for b in range(st.B):
        n = st.lengths[b]
        at = lambda s: (int(st.table_np[b][s // st.page]), s % st.page)  # noqa: E731
        for h in range(st.H_kv):
            src = oracle.evict_sources(score[b, h], pos[b, h], n, budget, sinks, recent, next_pos[b])
            for s, o in enumerate(src):
                assert torch.equal(st.k[at(s)][h].view(torch.int16), k0[at(o)][h].view(torch.int16)), (b, h, s, o)
                assert torch.equal(st.v[at(s)][h].view(torch.int16), v0[at(o)][h].view(torch.int16))
            want_s, want_p = marks[0][b, h].copy(), marks[1][b, h].copy()
            want_s[:n], want_p[:n] = 0.0, -1
            want_s[:len(src)], want_p[:len(src)] = score[b, h, src], pos[b, h, src]
            assert np.array_equal(score_out[b, h], want_s, equal_nan=True) and np.array_equal(pos_out[b, h], want_p)
            for s in range(len(src), n):  # what is dropped past the budget stays as it was
                assert torch.equal(st.k[at(s)][h].view(torch.int16), k0[at(s)][h].view(torch.int16))
        assert length_out[b] == min(n, budget)


EVICT = [  # lengths, H_kv, page, dtype, D, budget, sinks, recent
    ([0, 1, 5], 2, 8, "bf16", 64, 4, 1, 1),
    ([33, 32, 31, 64], 1, 16, "fp16", 128, 32, 2, 8),
    ([257, 1], 3, 64, "bf16", 128, 256, 4, 16),
    ([300, 1500, 1024], 2, 32, "bf16", 64, 100, 0, 0),
    ([1100, 1025], 2, 128, "bf16", 128, 1024, 4, 1000),
    ([90], 1, 8, "bf16", 64, 1, 0, 0),
    ([90], 1, 8, "bf16", 64, 10, 50, 50),
    ([5000, 2100], 1, 256, "bf16", 64, 2000, 4, 256),
]


@pytest.mark.parametrize("lengths,H_kv,page,dtype,D,budget,sinks,recent", EVICT)
def test_evict_matches_oracle(lengths, H_kv, page, dtype, D, budget, sinks, recent):
    st, score, pos = evict_setup(lengths, H_kv, page, dtype, seed=budget, D=D)
    next_pos = torch.tensor([score.shape[2]] * st.B, dtype=torch.int32, device="cuda")
    k0, v0 = st.k.clone(), st.v.clone()
    s0, p0 = score.cpu().numpy(), pos.cpu().numpy()
    cache = st.cache()
    so, po, lo = torch.full_like(score, 5.0), torch.full_like(pos, 9), torch.full_like(st.length, 77)
    marks = so.cpu().numpy(), po.cpu().numpy()
    got = cache.evict(score, pos, next_pos, budget, sinks, recent, so, po, lo)
    assert got[0] is so and got[1] is po and got[2] is lo
    assert cache.status() == 0 and st.length.tolist() == st.lengths
    assert np.array_equal(score.cpu().numpy(), s0) and np.array_equal(pos.cpu().numpy(), p0)
    check_evict(st, (k0, v0), s0, p0, next_pos.tolist(), budget, sinks, recent, so.cpu().numpy(), po.cpu().numpy(),
                lo.tolist(), marks)
    # in place, from the same start
    st.k.copy_(k0), st.v.copy_(v0)
    cache.evict(score, pos, next_pos, budget, sinks, recent)
    check_evict(st, (k0, v0), s0, p0, next_pos.tolist(), budget, sinks, recent, score.cpu().numpy(), pos.cpu().numpy(),
                st.length.tolist(), (s0, p0))


@pytest.mark.parametrize("keys,H_kv,D,budget", [
    (2000, 3, 64, 1700), (4000, 2, 64, 3999), (8000, 2, 128, 100), (12000, 2, 64, 6000), (30000, 2, 64, 17001),
    (50000, 5, 64, 20000), (50000, 3, 64, 49990), (150000, 1, 64, 70000), (900000, 1, 64, 400000),
    (30000, 2, 64, 29900), (50000, 1, 64, 49900), (90000, 3, 64, 30000), (90000, 3, 64, 300), (400000, 5, 64, 1000)])
def test_evict_of_every_size(keys, H_kv, D, budget):
    """One call of each way the selection is laid out (slots a CTA, cluster sizes, keys
    in registers, in shared memory and read again), against a stable sort."""
    g = gen(keys)
    page, B = 64, 2 if keys < 100000 else 1
    per = -(-keys // page)
    n_pages = B * per
    k = torch.randn(n_pages, page, H_kv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(n_pages, page, H_kv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(n_pages, generator=g, device="cuda").view(B, per).int()
    lengths = [keys - 7, keys - keys // 3][:B]
    length = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cache = bsa.PagedCache(k, v, table, length)
    score = (torch.randn(B, H_kv, cache.capacity, generator=g, device="cuda") * 50).round()  # many equal ones
    pos = torch.stack([torch.randperm(cache.capacity, generator=g, device="cuda") for _ in range(B * H_kv)]).int()
    pos = pos.view(B, H_kv, -1).contiguous()
    nxt = torch.full((B,), cache.capacity, dtype=torch.int32, device="cuda")
    k0, v0, s0, p0 = k.clone(), v.clone(), score.clone(), pos.clone()
    cache.evict(score, pos, nxt, budget, sinks=5, recent=budget // 3)
    assert cache.status() == 0 and length.tolist() == [min(n, budget) for n in lengths]
    slot = torch.arange(cache.capacity, device="cuda")
    for b in range(B):
        n, page_of = lengths[b], table[b].long()
        for h in range(H_kv):
            src = slot[:min(n, budget)].clone()
            if n > budget:
                p, s = p0[b, h, :n], s0[b, h, :n]
                must = (p < 5) | (p >= int(nxt[b]) - budget // 3)
                rank = torch.where(must, math.inf, s)
                keep = torch.sort(rank, descending=True, stable=True).indices[:budget]
                kept = torch.zeros(n, dtype=torch.bool, device="cuda")
                kept[keep] = True
                src[~kept[:budget]] = slot[budget:n][kept[budget:]]
            to, fr = slot[:src.numel()], src
            assert torch.equal(score[b, h, to], s0[b, h, fr]) and torch.equal(pos[b, h, to], p0[b, h, fr])
            assert (score[b, h, src.numel():n] == 0).all() and (pos[b, h, src.numel():n] == -1).all()
            assert torch.equal(score[b, h, n:], s0[b, h, n:])
            for x, x0 in ((k, k0), (v, v0)):
                assert torch.equal(x[page_of[to // page], to % page, h], x0[page_of[fr // page], fr % page, h])
                late = slot[src.numel():n]
                assert torch.equal(x[page_of[late // page], late % page, h], x0[page_of[late // page], late % page, h])


def test_evict_orders_odd_scores():
    """NaN counts as the lowest, -0 equals 0, infinities order, equal scores keep the lower slot."""
    st, score, pos = evict_setup([40], 1, 8, seed=3)
    odd = [math.nan, -math.inf, math.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38, math.nan]
    score[0, 0, :40] = torch.tensor(odd * 4)
    pos[0, 0, :40] = torch.arange(100, 140, dtype=torch.int32)
    s0, p0 = score.cpu().numpy(), pos.cpu().numpy()
    k0, v0 = st.k.clone(), st.v.clone()
    next_pos = torch.tensor([10000], dtype=torch.int32, device="cuda")
    for budget in (1, 6, 11, 13, 22, 29, 33, 39):
        st.k.copy_(k0), st.v.copy_(v0)
        so, po, lo = torch.zeros_like(score), torch.zeros_like(pos), torch.zeros_like(st.length)
        st.cache().evict(score, pos, next_pos, budget, scores_out=so, pos_out=po, length_out=lo)
        z = np.zeros_like(s0), np.zeros_like(p0)
        check_evict(st, (k0, v0), s0, p0, [10000], budget, 0, 0, so.cpu().numpy(), po.cpu().numpy(), lo.tolist(), z)


def test_evict_reports_a_bad_page_and_writes_only_good_ones():
    st, score, pos = evict_setup([64, 64], 2, 8, seed=4)
    score[:, :, :32], score[:, :, 32:] = 1.0, 2.0  # every kept key moves
    next_pos = torch.tensor([10000] * 2, dtype=torch.int32, device="cuda")
    st.table[0, 5] = -1
    st.table[1, 2] = st.k.shape[0]
    k0 = st.k.clone()
    cache = st.cache()
    cache.evict(score, pos, next_pos, 32)
    assert cache.status(clear=True) == 11 and st.length.tolist() == [32, 32]
    for b, skip in ((0, 8), (1, 16)):
        for s in range(32):
            to, fr = (int(st.table_np[b][s // 8]), s % 8), (int(st.table_np[b][4 + s // 8]), s % 8)
            want = k0[to] if skip <= s < skip + 8 else k0[fr]
            assert torch.equal(st.k[to].view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------------------ together

def serve(st, cache, scores, pos, next_pos, budget, g, steps, T):
    """Draft, rotate and append, attend, weigh, accept a prefix of the chain, evict."""
    B, H, H_kv, D = st.B, st.H, st.H_kv, st.D
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    axis = (torch.arange(D // 2, device="cuda") % 2).to(torch.int32)
    outs = []
    for step in range(steps):
        q, k, v = (normal(g, (B, T, n, D), st.dtype) for n in (H, H_kv, H_kv))
        p = (next_pos[None, :, None] + torch.arange(T, device="cuda", dtype=torch.int32)).expand(2, B, T).contiguous()
        qr = cache.append(k, v, q=q, rope=(p, freq, axis, "halves"))
        out, lse = cache.attend(qr)
        take = torch.tensor([1 + (step + b) % T for b in range(B)], dtype=torch.int32, device="cuda")
        cache.weigh(qr, lse, scores, n_new=take)
        slots = cache.length[:, None] + torch.arange(T, device="cuda")
        for h in range(H_kv):
            pos[:, h].scatter_(1, slots.long(), p[0])
        cache.length += take
        next_pos += take
        cache.evict(scores, pos, next_pos, budget, sinks=2, recent=T)
        outs.append((q, qr, k, v, out, lse, p, take))
    return outs


def test_a_serving_loop_over_a_full_cache():
    """Sixteen steps on a cache that evicts at every one, against an fp64 model of
    the same cache held as lists of keys per head."""
    B, H, H_kv, D, page, budget, T, steps = 2, 4, 2, 64, 16, 48, 3, 16
    st = Setup([40, 47], T, H, H_kv, D, page, "bf16", seed=20, spare=24)
    st.k.nan_to_num_(), st.v.nan_to_num_()
    cache = st.cache()
    scores = torch.zeros(B, H_kv, cache.capacity, device="cuda")
    pos = torch.arange(cache.capacity, device="cuda", dtype=torch.int32).expand(B, H_kv, -1).contiguous()
    next_pos = st.length.clone()
    model_k = [[list(st.seqs()[b][:st.lengths[b], h]) for h in range(H_kv)] for b in range(B)]
    model_v = [[list(st.seqs(st.v)[b][:st.lengths[b], h]) for h in range(H_kv)] for b in range(B)]
    model_p = [[list(range(st.lengths[b])) for _ in range(H_kv)] for b in range(B)]
    model_s = [[[0.0] * st.lengths[b] for _ in range(H_kv)] for b in range(B)]
    outs = serve(st, cache, scores, pos, next_pos, budget, gen(21), steps, T)
    assert cache.status() == 0
    freq = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    nxt = list(st.lengths)
    for q, qr, k, v, out, lse, p, take in outs:
        n = take.tolist()
        rk = oracle.rope(f64(k), p.cpu().numpy(), freq, np.arange(D // 2) % 2, "halves")
        rk = f64(torch.from_numpy(rk).to(DT["bf16"]))
        for b in range(B):
            for h in range(H_kv):
                mk, mv = np.array(model_k[b][h] + list(rk[b, :, h])), np.array(model_v[b][h] + list(f64(v)[b, :, h]))
                L0 = len(model_k[b][h])
                for t in range(T):
                    for x in range(h * 2, h * 2 + 2):
                        s = st.scale * (mk[:L0 + t + 1] @ f64(qr)[b, t, x])
                        e = np.exp(s - s.max())
                        w = e / e.sum()
                        got = f64(out)[b, t, x]
                        # a rotated key's element may round the other way where the oracle's lies next to a border:
                        # rare, at most 2^-7 of one product of the exponent (|q k| scale <= 4 * 4 / 8), so 2^-6 of a
                        # weight for one such element, beside the weights' and the result's own half steps
                        tol = (2.0 ** -6 + 3 * 2.0 ** -8) * (w @ np.abs(mv[:L0 + t + 1]))
                        assert (np.abs(got - w @ mv[:L0 + t + 1]) <= tol).all()
                        if t < n[b]:
                            model_s[b][h] += [0.0] * (L0 + t + 1 - len(model_s[b][h]))
                            for j in range(L0 + t + 1):
                                model_s[b][h][j] += w[j]
                model_k[b][h] += list(rk[b, :n[b], h])
                model_v[b][h] += list(f64(v)[b, :n[b], h])
                model_p[b][h] += list(p.cpu().numpy()[0, b, :n[b]])
                model_s[b][h] = model_s[b][h][:L0 + n[b]]
            nxt[b] += n[b]
            for h in range(H_kv):
                src = oracle.evict_sources(model_s[b][h], model_p[b][h], len(model_k[b][h]), budget, 2, T, nxt[b])
                model_k[b][h] = [model_k[b][h][i] for i in src]
                model_v[b][h] = [model_v[b][h][i] for i in src]
                model_p[b][h] = [model_p[b][h][i] for i in src]
                model_s[b][h] = [model_s[b][h][i] for i in src]
    assert cache.length.tolist() == [budget, budget] and next_pos.tolist() == nxt
    for b in range(B):
        for h in range(H_kv):
            assert pos[b, h, :budget].tolist() == model_p[b][h]
            assert np.allclose(scores[b, h, :budget].cpu().numpy(), model_s[b][h], rtol=1e-3, atol=1e-4)


def test_a_captured_step_replays_on_another_stream():
    """append, attend, weigh and evict captured once and replayed with new inputs
    on another stream, next to an eager cache on a third: the same bits as eager."""
    def make():
        st = Setup([300, 180], 4, 8, 2, 64, 32, seed=30, spare=16)
        st.k.nan_to_num_(), st.v.nan_to_num_()
        cache = st.cache()
        return st, cache, torch.zeros(2, 2, cache.capacity, device="cuda"), \
            torch.arange(cache.capacity, device="cuda", dtype=torch.int32).expand(2, 2, -1).contiguous(), \
            torch.tensor([400, 400], dtype=torch.int32, device="cuda")

    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    axis = torch.zeros(32, dtype=torch.int32, device="cuda")
    p = torch.arange(8, device="cuda", dtype=torch.int32).view(1, 2, 4)
    def step(st, cache, scores, pos, nxt, io):
        qr = cache.append(io["k"], io["v"], q=io["q"], rope=(p, freq, axis, "interleaved"))
        out, lse = cache.attend(qr)
        cache.weigh(qr, lse, scores)
        cache.length += 4
        cache.evict(scores, pos, nxt, 150, sinks=1, recent=1)
        return out, lse

    def inputs(seed):
        g = gen(seed)
        return {n: normal(g, (2, 4, h, 64), "bf16") for n, h in (("q", 8), ("k", 2), ("v", 2))}

    a, b = make(), make()
    io = inputs(0)
    warm = make()
    step(*warm, io)  # everything the capture needs is there (the workspace's size among it)
    torch.cuda.synchronize()
    a[1].reserve(150)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*a, io)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for seed in (1, 2, 3):
        fresh = inputs(seed)
        for n in io:
            io[n].copy_(fresh[n])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        with torch.cuda.stream(other):
            want = step(*b, fresh)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for x, y in zip(a[2:4], b[2:4]):
            assert torch.equal(x, y)
        assert torch.equal(a[0].k, b[0].k) and torch.equal(a[0].v, b[0].v)
        assert a[1].length.tolist() == b[1].length.tolist() == [150, 150]
    assert a[1].status() == 0 and b[1].status() == 0


def test_caches_may_share_a_workspace():
    st = Setup([300, 40], 2, 4, 2, 64, 16, seed=70)
    ws = bsa.CacheWorkspace("cuda:0")
    a, b = (bsa.PagedCache(st.k, st.v, st.table, st.length, workspace=ws) for _ in range(2))
    want = st.cache().attend(st.q, st.tree)
    for c in (a, b, a):
        got = c.attend(st.q, st.tree)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    st.table[0, 0] = -1
    b.attend(st.q, st.tree)
    assert a.status(clear=True) == 11 and b.status() == 0
    with pytest.raises(ValueError):
        bsa.PagedCache(st.k, st.v, st.table, st.length, workspace=bsa.CacheWorkspace("cpu"))
    torch.cuda.synchronize()
    before = ws.nbytes
    with pytest.raises(RuntimeError):  # a capture must not hold the memory of later eager calls
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.zeros(1, device="cuda")
            ws.grow(2 * before)
    assert ws.nbytes == before
    ws.grow(2 * before)
    got = a.attend(st.q, st.tree)
    assert b.status(clear=True) == 11 and got[0].shape == st.q.shape


def test_a_captured_graph_keeps_its_workspace_when_the_cache_takes_a_larger_one():
    st = Setup([300, 40], 2, 4, 2, 64, 16, seed=71)
    cache = st.cache()
    want = cache.attend(st.q, st.tree)
    torch.cuda.synchronize()
    graph, at, nbytes = torch.cuda.CUDAGraph(), cache.workspace.ptr, cache.workspace.nbytes
    with torch.cuda.graph(graph):
        got = cache.attend(st.q, st.tree)
    cache.workspace.grow(nbytes + 1)
    assert cache.workspace.ptr != at
    # whatever is allocated now is not the graph's
    others = [torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() + nbytes <= at or at + nbytes <= x.data_ptr() for x in others)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all((x == 7).all() for x in others)
    # and its errors are seen
    st.table[0, 0] = -1
    graph.replay()
    assert cache.status(clear=True) == 11 and cache.status() == 0


def test_an_eviction_takes_no_more_workspace_than_it_needs():
    """A capacity of 2^20 slots a head: one slot's lists fit any workspace, half of them do not."""
    k = torch.zeros(4, 64, 8, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 1 << 14, dtype=torch.int32, device="cuda")
    table[:, 1], table[:, 2] = 1, 2
    cache = bsa.PagedCache(k, k.clone(), table, torch.tensor([129, 100], dtype=torch.int32, device="cuda"))
    score, pos = torch.rand(2, 8, 1 << 20, device="cuda"), torch.zeros(2, 8, 1 << 20, dtype=torch.int32, device="cuda")
    nxt = torch.full((2,), 5, dtype=torch.int32, device="cuda")
    before = cache.workspace.nbytes
    for budget in ((1 << 20) - 1, 1 << 20, (1 << 31) - 1, 128):
        cache.evict(score, pos, nxt, budget)
        assert cache.workspace.nbytes == before
    assert cache.length.tolist() == [128, 100]
    cache.evict(score, pos, nxt, 1 << 19)
    assert cache.workspace.nbytes >= 4 * 4 * 16 << 19 and cache.status() == 0 and cache.length.tolist() == [128, 100]


def test_a_workspace_outlives_its_cache_on_another_stream():
    st = Setup([3000, 4000], 4, 8, 2, 128, 128, seed=72)
    want = st.cache().attend(st.q, st.tree)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        cache = st.cache()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                got = cache.attend(st.q, st.tree)
        n = cache.workspace.nbytes
        del cache
        scribble = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # on the stream the workspace came from
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (scribble == 255).all()


def test_a_cache_holds_the_tensors_it_was_made_with():
    st = Setup([20, 30], 3, 4, 2, 64, 16, seed=73)
    cache = st.cache()
    at = cache.length.data_ptr()
    cache.length += 1
    assert cache.length.data_ptr() == at and cache.length.tolist() == [21, 31]
    for name in ("k", "v", "page_table", "length"):
        with pytest.raises(ValueError):
            setattr(cache, name, getattr(cache, name) + 1)


def test_refusals():
    st = Setup([20, 30], 3, 4, 2, 64, 16, seed=40)
    cache = st.cache()
    q, k = st.q, st.q[:, :, :2].contiguous()
    sc = torch.zeros(2, 2, cache.capacity, device="cuda")
    ps = torch.zeros(2, 2, cache.capacity, dtype=torch.int32, device="cuda")
    lse = torch.zeros(2, 4, 3, device="cuda")
    np_ = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: cache.attend(q[:1]), lambda: cache.attend(q.half()), lambda: cache.attend(q[..., :32]),
                 lambda: cache.attend(q.cpu()), lambda: cache.attend(q, tree=torch.zeros(2, 3, device="cuda")),
                 lambda: cache.attend(q, tree=torch.zeros(2, 4, dtype=torch.int64, device="cuda")),
                 lambda: cache.attend(q, n_new=torch.zeros(2, device="cuda")), lambda: cache.attend(q, lse=lse[:, :2]),
                 lambda: cache.attend(q, out=q[:, :2]), lambda: cache.weigh(q, lse.double(), sc),
                 lambda: cache.weigh(q, lse, sc[:, :1]), lambda: cache.weigh(q, lse, sc, out=sc.double()),
                 lambda: cache.append(q, q), lambda: cache.append(k, k[:, :2]), lambda: cache.append(k, k, q=q[:, :2]),
                 lambda: cache.evict(sc, ps.float(), np_, 4), lambda: cache.evict(sc, ps, np_.long(), 4),
                 lambda: cache.evict(sc[..., :4], ps, np_, 4),
                 lambda: bsa.PagedCache(st.k.float(), st.v.float(), st.table, st.length),
                 lambda: bsa.PagedCache(st.k, st.v[1:], st.table, st.length),
                 lambda: bsa.PagedCache(st.k, st.v, st.table.long(), st.length),
                 lambda: bsa.PagedCache(st.k, st.v, st.table, st.length[:1]),
                 lambda: bsa.PagedCache(st.k, st.v, st.table.cpu(), st.length)):
        with pytest.raises(ValueError):
            call()
    for call, code in ((lambda: cache.evict(sc, ps, np_, 0), 1), (lambda: cache.evict(sc, ps, np_, 4, sinks=-1), 1),
                       (lambda: cache.attend(torch.zeros(2, 65, 4, 64, dtype=torch.bfloat16, device="cuda")), 1),
                       (lambda: cache.attend(torch.zeros(2, 1, 3, 64, dtype=torch.bfloat16, device="cuda")), 1),
                       (lambda: cache.attend(torch.zeros(2, 1, 258, 64, dtype=torch.bfloat16, device="cuda")), 2),
                       (lambda: bsa.PagedCache(st.k[:, :9], st.v[:, :9], st.table, st.length), 2),
                       (lambda: bsa.PagedCache(st.k[..., :32], st.v[..., :32], st.table, st.length), 2)):
        with pytest.raises(bsa.BsaError) as e:
            call()
        assert e.value.code == code


def test_outputs_that_overlap_inputs_are_refused():
    st = Setup([20, 30], 3, 4, 2, 64, 16, seed=42)
    cache = st.cache()
    lse = cache.attend(st.q, st.tree)[1]
    wide = torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = 2 * 2 * cache.capacity
    buf, ibuf = torch.zeros(n + 8, device="cuda"), torch.zeros(n + 8, dtype=torch.int32, device="cuda")
    shape = (2, 2, cache.capacity)
    sc, sc2, ps, ps2 = buf[:n].view(shape), buf[8:].view(shape), ibuf[:n].view(shape), ibuf[8:].view(shape)
    both = torch.zeros(3, dtype=torch.int32, device="cuda")
    nxt = torch.zeros(2, dtype=torch.int32, device="cuda")
    kv = st.q[:, :, :2].contiguous()
    for call in (lambda: cache.attend(st.q, out=st.q), lambda: cache.attend(st.q, out=st.q.view(st.q.shape)),
                 lambda: cache.attend(wide[:, :3], out=wide[:, 1:]), lambda: cache.weigh(st.q, lse, sc, out=sc2),
                 lambda: cache.evict(sc, ps, nxt, 4, scores_out=sc2), lambda: cache.evict(sc, ps, nxt, 4, pos_out=ps2),
                 lambda: cache.evict(sc, ps, nxt, 4, length_out=nxt), lambda: cache.evict(sc, ps, both[:2], 4, length_out=both[1:]),
                 lambda: cache.append(kv, kv.clone(), q=kv.clone(), q_out=kv),
                 lambda: cache.append(kv.clone(), kv, q=kv.clone(), q_out=kv),
                 lambda: cache.evict(sc, ps, nxt, 1 << 32), lambda: cache.evict(sc, ps, nxt, 4, sinks=1 << 32),
                 lambda: cache.evict(sc, ps, nxt, 4, recent=(1 << 32) + 1), lambda: cache.reserve(1 << 32)):
        with pytest.raises(ValueError):
            call()
    # in place by another view of the same memory is in place
    before = cache.length.clone()
    cache.evict(sc, ps, nxt, 4, scores_out=sc.view(shape), pos_out=ps.view(shape), length_out=cache.length.view(2))
    assert before.tolist() == [20, 30] and cache.length.tolist() == [4, 4] and cache.status() == 0


def test_empty_calls_do_nothing():
    st = Setup([20, 30], 0, 4, 2, 64, 16, seed=41)
    cache = st.cache()
    n = bsa.launch_count()
    out, lse = cache.attend(st.q)
    assert out.shape == (2, 0, 4, 64) and lse.shape == (2, 4, 0)
    cache.weigh(st.q, lse, torch.zeros(2, 2, cache.capacity, device="cuda"))
    cache.append(st.q[:, :, :2], st.q[:, :, :2])
    none = bsa.PagedCache(st.k, st.v, st.table[:0], st.length[:0])
    none.attend(st.q[:0])
    none.evict(torch.zeros(0, 2, cache.capacity, device="cuda"), torch.zeros(0, 2, cache.capacity, dtype=torch.int32, device="cuda"),
               st.length[:0], 4)
    assert bsa.launch_count() == n
