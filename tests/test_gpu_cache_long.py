"""The paged cache where the range of a type, the length of a cache or the way the
work is cut makes the difference, against the fp64 oracle."""

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
