"""The paged cache where the range of a type, the length of a cache or the way the
work is cut makes the difference, against the fp64 oracle."""

import math
import os
import re

import numpy as np
import pytest
import torch

import block_sparse_attention_map_b200 as bsa
from oracle import serving as oracle
from tests.serving_common import DT, HALF_STEP, Setup, attend_tolerance, exponent_tolerance, f64, gen, normal

pytestmark = pytest.mark.gpu


def words(st):
    return oracle.words_or_chain(None if st.tree is None else st.tree.tolist(), st.B, st.T)


# ------------------------------------------------------------------ fp16's range

@pytest.mark.parametrize("keys,T,H,D", [(60, 1, 1, 64), (500, 3, 8, 128), (3000, 2, 4, 64), (1500, 40, 4, 128)])
@pytest.mark.parametrize("gap", [17.5, 18.5, 20.0])
def test_fp16_keeps_what_lies_far_below_the_heaviest_key(keys, T, H, D, gap):
    """One heavy key of no value in 64, the others' weights e^-gap (2^-25 .. 2^-29) of
    its and their values near the type's largest: all of O comes from them."""
    st = Setup([keys], T, H, 1, D, 64, "fp16", seed=keys, tree=None)
    st.k.zero_()
    st.q.zero_()
    st.q[..., 0] = math.sqrt(D)  # the score is the key's first element
    st.k[..., 0] = torch.rand(st.k.shape[:3], generator=st.g, device="cuda") * 0.5
    st.v[:] = 40000 + 20000 * torch.rand(st.v.shape, generator=st.g, device="cuda")
    st.k[:, 0, :, 0], st.v[:, 0] = gap, 0.0
    out, lse = st.cache().attend(st.q, scale=1 / math.sqrt(D))
    st.scale = 1 / math.sqrt(D)
    O, L, mass = oracle.attend(f64(st.q), st.seqs(), st.seqs(st.v), st.lengths, st.new, words(st), st.scale)
    assert O.min() > 0.004
    # a weight is stored as 2^7 or more times its share of the heaviest, in fp16, so off by 2^-25 / 2^7 where that is below
    # the type's normal range; 64 of them a heavy key (128 where the last page has just begun), of values up to 60000.
    # Beside it: the weights' and the result's half steps, and the fp32 exponents and sums (all as in attend_tolerance)
    u = HALF_STEP["fp16"]
    e = exponent_tolerance(f64(st.q), st.seqs(), st.scale)
    tol = 128 * 2.0 ** -32 * 60000 + u * O + 1.02 * u * (mass + O) + (2.0 ** -17 + 2 * e) * mass
    err = np.abs(f64(out) - O)
    assert (err <= tol).all(), (float(err.max()), float(O.min()), float(tol.min()))
    assert (np.abs(f64(lse) - L) <= e + 1e-6).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("keys", [200, 2000])
def test_scores_so_large_that_their_products_lose_powers_of_two(dtype, keys):
    """|s| up to 2^25: a product's rounding alone moves an exponent by more than 1,
    and a weight above its type's range would be infinite.  Every row whose first
    score leads by more than the fp32 products' error takes that key's value."""
    st = Setup([keys, 90], 3, 8, 2, 64, 32, dtype, seed=keys)
    st.k *= 1000
    st.q *= 1000
    out, lse = st.cache().attend(st.q, st.tree, scale=1.0)
    checked = 0
    for b in range(2):
        k, v, q = st.seqs()[b], st.seqs(st.v)[b], f64(st.q)[b]
        for t in range(3):
            seen = [j < st.lengths[b] or (words(st)[b][t] >> (j - st.lengths[b])) & 1 == 1 for j in range(len(k))]
            for h in range(8):
                s = np.where(seen, k[:, h // 4] @ q[t, h], -np.inf)
                first, second = np.argsort(s)[::-1][:2]
                if s[first] - s[second] <= 2 * 64 * 2.0 ** -23 * np.abs(k[:, h // 4] * q[t, h]).sum(1).max() + 64:
                    continue
                checked += 1
                want = v[first, h // 4]
                assert (np.abs(f64(out)[b, t, h] - want) <= HALF_STEP[dtype] * np.abs(want)).all()
                assert abs(f64(lse)[b, h, t] - s[first]) <= 2.0 ** -16 * abs(s[first])
    assert checked > 40


# ------------------------------------------------------------------ the serving step that README shows

def readme_step():
    """The block of README that makes a PagedCache."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    return next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "PagedCache" in b)


def test_the_readme_step_of_drafted_trees():
    """Three steps as README has them, on drafted trees whose accepted branch is not
    their first tokens, against an fp64 model of each head's keys: what is weighed are
    the accepted rows, over the keys that their softmax went over."""
    step = compile(readme_step(), "README.md", "exec")
    B, H, H_kv, D, page, T = 2, 4, 2, 64, 64, 7
    st = Setup([4093, 300], T, H, H_kv, D, page, "bf16", seed=80, spare=16)
    parents = torch.tensor([[-1, 0, 0, 2, 2, 4, 1], [-1, -1, 1, 2, 0, 3, 4]])
    paths, counts = [[0, 2, 4, 5], [1, 2, 3, 5]], [[4, 2], [3, 4], [4, 1]]
    depth = torch.tensor([[0, 1, 1, 2, 2, 3, 2], [0, 0, 1, 2, 1, 3, 2]], dtype=torch.int32, device="cuda")
    cap = st.table.shape[1] * page
    inv_freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    ns = dict(bsa=bsa, torch=torch, k_pages=st.k, v_pages=st.v, page_table=st.table, length=st.length,
              inv_freq=inv_freq, axis=torch.zeros(D // 2, dtype=torch.int32, device="cuda"), parents=parents.cuda(),
              path=torch.tensor(paths, device="cuda"), scores=torch.rand(B, H_kv, cap, generator=st.g, device="cuda"),
              key_pos=torch.arange(cap, device="cuda", dtype=torch.int32).expand(B, H_kv, -1).contiguous(),
              next_pos=st.length.clone())
    for b in range(B):
        ns["scores"][b, :, st.lengths[b]:] = 0
    seq = [[x[:n] for x, n in zip(st.seqs(w), st.lengths)] for w in (st.k, st.v)]
    keys, values = ([[list(seq[i][b][:, h]) for h in range(H_kv)] for b in range(B)] for i in range(2))
    score = [[list(f64(ns["scores"])[b, h, :st.lengths[b]]) for h in range(H_kv)] for b in range(B)]
    place = [[list(range(st.lengths[b])) for _ in range(H_kv)] for b in range(B)]
    tree = oracle.words_or_chain(bsa.tree_words(parents).tolist(), B, T)
    evicted = 0
    for count in counts:
        q, k, v = (normal(st.g, (B, T, n, D), "bf16") for n in (H, H_kv, H_kv))
        ns.update(q_new=q, k_new=k, v_new=v, pos=(ns["next_pos"][:, None] + depth)[None].contiguous(),
                  accepted=torch.tensor(count, dtype=torch.int32, device="cuda"))
        rq, rk = (f64(x) for x in bsa.rope(q, k, ns["pos"], inv_freq, ns["axis"], "halves"))
        at, before = ns["pos"][0].tolist(), ns["next_pos"].tolist()
        exec(step, ns)
        cache = ns["cache"]
        assert cache.status() == 0
        for b in range(B):
            n, L = count[b], len(keys[b][0])
            path = paths[b][:n]
            for h in range(H_kv):
                mk, mv = np.array(keys[b][h] + list(rk[b, :, h])), np.array(values[b][h] + list(f64(v)[b, :, h]))
                weight = np.zeros(L + T)
                for t in range(T):
                    seen = np.array([j < L or (tree[b][t] >> (j - L)) & 1 == 1 for j in range(L + T)])
                    for x in (2 * h, 2 * h + 1):
                        s = np.where(seen, st.scale * (mk @ rq[b, t, x]), -np.inf)
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        O, mass = w @ mv, w @ np.abs(mv)
                        err = np.abs(f64(ns["o"])[b, t, x] - O)
                        e = exponent_tolerance(rq[b, t, x], [mk], st.scale)
                        assert (err <= attend_tolerance(O, mass, L + T, 5.0, "bf16") + 2 * e * mass).all()
                        if t in path:
                            weight += w
                # the accepted rows see the cache and one another's tokens: all of their weight lands on kept tokens
                assert np.isclose(weight[:L].sum() + weight[[L + t for t in path]].sum(), 2 * n)
                keys[b][h] += [rk[b, t, h] for t in path]
                values[b][h] += [f64(v)[b, t, h] for t in path]
                place[b][h] += [at[b][t] for t in path]
                score[b][h] = [a + w for a, w in zip(score[b][h] + [0.0] * n, list(weight[:L]) + [weight[L + t] for t in path])]
                src = oracle.evict_sources(score[b][h], place[b][h], len(keys[b][h]), 4096, 4, 256, before[b] + n)
                evicted += len(keys[b][h]) - len(src)
                for m in (keys, values, place, score):
                    m[b][h] = [m[b][h][i] for i in src]
        assert ns["length"].tolist() == [len(keys[b][0]) for b in range(B)]
        assert ns["next_pos"].tolist() == [a + n for a, n in zip(before, count)]
        for b in range(B):
            s = np.arange(len(keys[b][0]))
            rows = st.table_np[b][s // page], s % page
            for h in range(H_kv):
                assert ns["key_pos"][b, h, :len(s)].tolist() == place[b][h]
                assert np.array_equal(f64(st.k)[rows][:, h], np.array(keys[b][h]))
                assert np.array_equal(f64(st.v)[rows][:, h], np.array(values[b][h]))
                # each weight off by the factor exp(+-(its exponent's and the lse's error)), fp32 sums of them and the score
                assert np.allclose(f64(ns["scores"])[b, h, :len(s)], score[b][h], rtol=2.0 ** -18, atol=2.0 ** -18)
    assert evicted == 2 * (4093 + 11 - 4096)


# ------------------------------------------------------------------ rows cut into the runs of several CTAs

CUT = [  # lengths, T, H_kv, G, dtype: the new tokens lie in two tiles, with a run or more a tile, or several items a run
    ([128 * 9 - 3, 641], 5, 2, 4, "bf16"),
    ([128 * 9 - 3, 638], 40, 2, 4, "bf16"),       # 128 + 32 rows
    ([128 * 9 - 30, 128 * 6 - 1], 64, 2, 4, "fp16"),  # 128 + 128 rows
    ([128 * 7 - 2 - 5 * i for i in range(16)], 6, 8, 2, "fp16"),
    ([128 * 7 - 1 - 40 * i for i in range(8)], 33, 4, 8, "bf16"),  # 128 + 128 + 8 rows, two groups of rows
]


@pytest.mark.parametrize("lengths,T,H_kv,G,dtype", CUT)
def test_what_a_row_does_not_see_never_reaches_it_in_cut_runs(lengths, T, H_kv, G, dtype):
    """NaN, infinities and the type's lowest value in the key and value of one drafted
    token of every sequence: the rows that do not see it give the bits they give
    without it; to the others the infinities and NaN of the value come through."""
    B, page = len(lengths), 32
    st = Setup(lengths, T, H_kv * G, H_kv, 128, page, dtype, seed=90 + T)
    assert st.table.shape[1] * page > 512
    ref_out, ref_lse = st.cache().attend(st.q, st.tree)
    assert ref_out.isfinite().all()
    sees = torch.stack([(st.tree >> j) & 1 for j in range(T)], -1).bool()  # [B, T, j]
    for j in sorted({0, 2, T // 2, T - 1}):
        at = torch.tensor([st.lengths[b] + j for b in range(B)], device="cuda")
        rows = st.table.long()[torch.arange(B, device="cuda"), at // page], at % page
        hit = sees[..., j]
        for bad in (math.nan, math.inf, -math.inf):
            k, v = st.k.clone(), st.v.clone()
            x = v[rows]
            x[..., ::3], x[..., 1::3] = bad, torch.finfo(DT[dtype]).min
            v[rows] = x
            x = k[rows]
            x[..., 5] = bad
            k[rows] = x
            for keys in (k, st.k):
                out, lse = bsa.PagedCache(keys, v, st.table, st.length).attend(st.q, st.tree)
                assert torch.equal(out[~hit], ref_out[~hit])
                assert torch.equal(lse.transpose(1, 2)[~hit], ref_lse.transpose(1, 2)[~hit])
            got = out[hit][..., ::3]
            assert torch.isnan(got).all() if math.isnan(bad) else (got == bad).all()
            assert torch.equal(lse, ref_lse) and torch.equal(out[hit][..., 2::3], ref_out[hit][..., 2::3])


@pytest.mark.parametrize("T,H,n_new", [(4, 4, [4, 3, 2, 4]), (40, 8, [40, 40, 2, 39])])
def test_rows_of_no_key_beside_a_long_sequence(T, H, n_new):
    st = Setup([0, 1500, 0, 3000], T, H, 2, 64, 16, seed=92 + T, n_new=n_new, tree=None)
    w = torch.full((4, T), -1, dtype=torch.int64, device="cuda")  # every bit: more than there are
    w[:, 1::3] = 0                                                # sees no new token
    st.tree = w
    cache = st.cache()
    out, lse = cache.attend(st.q, w, st.n_new)
    O, L, mass = oracle.attend(f64(st.q), st.seqs(), st.seqs(st.v), st.lengths, st.new, words(st), st.scale)
    assert (np.abs(f64(out) - O) <= attend_tolerance(O, mass, 3040, 6.0, "bf16")).all()
    assert np.array_equal(np.isneginf(f64(lse)), np.isneginf(L)) and np.isneginf(L[0, :, 1]).all()
    assert (out[0, 1::3] == 0).all() and (out[2, 2:] == 0).all()
    scores = torch.zeros(4, 2, cache.capacity, device="cuda")
    cache.weigh(st.q, lse, scores, w, st.n_new)
    assert cache.status() == 0
    total = scores.sum((1, 2)).cpu().numpy()
    assert np.allclose(total, np.isfinite(L).sum((1, 2)), rtol=1e-4)


@pytest.mark.parametrize("T,H", [(2, 4), (40, 8)])
def test_bad_lengths_and_pages_of_long_caches_are_reported_and_read_as_zeros(T, H):
    st = Setup([1000, 700, 900], T, H, 2, 64, 16, seed=95)
    cap = st.table.shape[1] * 16
    cache = st.cache()
    ref, _ = cache.attend(st.q, st.tree)
    for bad in (-3, st.k.shape[0], 2 ** 31 - 1):
        st.table[1, 1], st.table[1, 40] = bad, bad
        out, lse = cache.attend(st.q, st.tree)
        scores = torch.zeros(3, 2, cap, device="cuda")
        cache.weigh(st.q, lse, scores, st.tree)
        assert cache.status(clear=True) == 11
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
        k, v = st.k.clone(), st.v.clone()
        for p in (1, 40):
            st.table[1, p] = int(st.table_np[1][p])
            k[st.table[1, p].long()], v[st.table[1, p].long()] = 0, 0
        zeros = bsa.PagedCache(k, v, st.table, st.length)
        want, wlse = zeros.attend(st.q, st.tree)
        wscores = torch.zeros_like(scores)
        zeros.weigh(st.q, wlse, wscores, st.tree)
        assert torch.equal(out, want) and torch.equal(lse, wlse) and torch.equal(scores, wscores) and zeros.status() == 0
    # lengths out of range: the bits of the clamped ones (another cut of the rows than with the first length)
    n_new = torch.full((3,), T, dtype=torch.int32, device="cuda")
    for bad, good, n in ((-5, 0, T), (cap + 9, cap, 0), (2 ** 31 - 1, cap, 0), (-(2 ** 31), 0, T)):
        st.length[2] = bad
        out, lse = cache.attend(st.q, st.tree)
        assert cache.status(clear=True) == 11
        st.length[2], n_new[2] = good, n
        if n:  # what the clamped sequence then reads as its new tokens
            st.k.nan_to_num_(), st.v.nan_to_num_()
        want, wlse = cache.attend(st.q, st.tree, n_new)
        assert torch.equal(out, want) and torch.equal(lse, wlse) and cache.status() == 0
        assert n > 0 or ((out[2] == 0).all() and torch.isneginf(lse[2]).all())


# ------------------------------------------------------------------ evictions whose outputs are apart

@pytest.mark.parametrize("keys,H_kv,budget", [
    (3000, 3, 2990), (3000, 2, 1000), (12000, 2, 6000), (30000, 2, 17001), (30000, 3, 29900), (50000, 5, 20000),
    (50000, 3, 49990), (50000, 1, 49900), (90000, 3, 300), (150000, 1, 70000), (400000, 5, 1000), (900000, 1, 400000)])
def test_evict_out_of_place_of_every_size(keys, H_kv, budget):
    """Each way the selection is laid out with outputs of their own (all, or one alone
    and the others in place), a sequence to cut beside one within the budget: the
    outputs of the call in place, their slots past the length and the inputs as they were."""
    g = gen(keys + budget)
    page, B = 64, 2
    per = -(-keys // page)
    k0 = torch.randn(B * per, page, H_kv, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    v0 = torch.randn(B * per, page, H_kv, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).int()
    n0 = torch.tensor([keys - 7, budget - budget // 3], dtype=torch.int32, device="cuda")
    cap = per * page
    s0 = (torch.randn(B, H_kv, cap, generator=g, device="cuda") * 50).round()  # many equal ones
    p0 = torch.stack([torch.randperm(cap, generator=g, device="cuda") for _ in range(B * H_kv)]).int().view(B, H_kv, -1).contiguous()
    nxt = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    slot = torch.arange(cap, device="cuda")

    def call(outputs):
        k, v, n, s, p = k0.clone(), v0.clone(), n0.clone(), s0.clone(), p0.clone()
        so, po, no = torch.full_like(s, 5.0), torch.full_like(p, 9), torch.full_like(n, 77)
        kw = {name: x for name, x in (("scores_out", so), ("pos_out", po), ("length_out", no)) if name in outputs}
        cache = bsa.PagedCache(k, v, table, n)
        got = cache.evict(s, p, nxt, budget, sinks=5, recent=budget // 3, **kw)
        assert cache.status() == 0
        for name, x, x0 in (("scores_out", s, s0), ("pos_out", p, p0), ("length_out", n, n0)):
            assert name not in outputs or torch.equal(x, x0)
        return k, v, got

    k, v, (s, p, n) = call(())
    assert n.tolist() == [budget, int(n0[1])]
    # (the call in place is held to a stable sort elsewhere; here that it moved what it had to)
    order = torch.sort(torch.where((p0[0] < 5) | (p0[0] >= cap - budget // 3), math.inf, s0[0])[:, :keys - 7], dim=-1,
                       descending=True, stable=True).indices[:, :budget]
    for h in range(H_kv):
        assert torch.equal(p[0, h, :budget].sort().values, p0[0, h, order[h]].sort().values)
    for outputs in (("scores_out", "pos_out", "length_out"), ("scores_out",), ("pos_out",), ("length_out",)):
        k1, v1, (s1, p1, n1) = call(outputs)
        assert torch.equal(k1, k) and torch.equal(v1, v) and torch.equal(n1, n)
        for b in range(B):
            m = int(n0[b])
            for name, x, y, mark in (("scores_out", s1, s, 5.0), ("pos_out", p1, p, 9)):
                assert torch.equal(x[b, :, :m], y[b, :, :m])
                assert (x[b, :, m:] == mark).all() if name in outputs else torch.equal(x[b, :, m:], y[b, :, m:])


# ------------------------------------------------------------------ a prompt

@pytest.mark.parametrize("layout,dtype,D,page,T", [
    ("halves", "bf16", 128, 64, 1500), ("interleaved", "fp16", 64, 16, 777), ("halves", "fp16", 64, 128, 2100), ("interleaved", "bf16", 128, 8, 65)])
def test_append_of_a_rotated_prompt(layout, dtype, D, page, T):
    """Prompts of many tokens behind caches of any length, rotated by positions of three
    axes on their way: the rows that rope gives, v as it is, nothing else written."""
    lengths, new = [0, 130, 5, 64], [T, T - 60, 0, 1]
    st = Setup(lengths, T, 4, 2, D, page, dtype, seed=T, n_new=new, tree=None)
    k, v = normal(st.g, (4, T, 2, D), dtype), normal(st.g, (4, T, 2, D), dtype)
    inv_freq = 10000.0 ** (-torch.arange(D // 2 - 8, dtype=torch.float64, device="cuda") / (D // 2))
    axis = (torch.arange(D // 2 - 8, device="cuda") % 3).to(torch.int32)
    pos = torch.randint(0, 90000, (3, 4, T), generator=st.g, device="cuda").to(torch.int32)
    want_k, want_v = st.k.clone(), st.v.clone()
    rq, rk = bsa.rope(st.q, k, pos, inv_freq, axis, layout)
    for b in range(4):
        s = np.arange(lengths[b], lengths[b] + new[b])
        at = torch.from_numpy(st.table_np[b][s // page].astype(np.int64)).cuda(), torch.from_numpy(s % page).cuda()
        want_k[at], want_v[at] = rk[b, :new[b]], v[b, :new[b]]
    cache = st.cache()
    q = cache.append(k, v, q=st.q, rope=(pos, inv_freq, axis, layout), n_new=st.n_new)
    assert cache.status() == 0 and torch.equal(q, rq) and st.length.tolist() == lengths
    assert torch.equal(st.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(st.v.view(torch.int16), want_v.view(torch.int16))
    # and rope itself, on a token of each sequence, against the oracle
    t = T // 2
    args = pos[:, :, t:t + 1].cpu().numpy(), inv_freq.cpu().numpy(), axis.cpu().numpy(), layout
    for x, y in ((st.q, q), (k, rk)):
        ref = oracle.rope(f64(x[:, t:t + 1]), *args)
        m = np.abs(f64(x[:, t:t + 1])).max(-1, keepdims=True) * 2
        assert (np.abs(f64(y[:, t:t + 1]) - ref) <= HALF_STEP[dtype] * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -21 * m + 2.0 ** -25).all()
