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
