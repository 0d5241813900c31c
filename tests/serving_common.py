"""Inputs and oracle views shared by the tests of the rotary positions and of
the paged cache."""

import math

import numpy as np
import torch

import block_sparse_attention_map_b200 as bsa

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # torch.finfo(t).eps / 2


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


class Setup:
    """A cache with B sequences of the given lengths, their pages anywhere, the
    unused slots NaN, and T new tokens already in it."""

    def __init__(self, lengths, T, H, H_kv, D, page, dtype="bf16", seed=0, n_new=None, extra_pages=1, tree="random",
                 spare=0):
        g = self.g = gen(seed)
        rng = np.random.default_rng(seed)
        B = len(lengths)
        self.B, self.T, self.H, self.H_kv, self.D, self.page, self.dtype = B, T, H, H_kv, D, page, dtype
        self.lengths = list(lengths)
        self.new = [T] * B if n_new is None else list(n_new)
        per = max(1, -(-(max(lengths) + T + spare) // page))
        n_pages = B * per + extra_pages
        self.table_np = rng.permutation(n_pages)[:B * per].reshape(B, per).astype(np.int32)
        self.k = torch.full((n_pages, page, H_kv, D), math.nan, dtype=DT[dtype], device="cuda")
        self.v = torch.full_like(self.k, math.nan)
        for b in range(B):
            n = self.lengths[b] + self.new[b]
            if n:
                s = torch.arange(n, device="cuda")
                at = torch.from_numpy(self.table_np[b].astype(np.int64)).cuda()[s // page]
                self.k[at, s % page] = normal(g, (n, H_kv, D), dtype)
                self.v[at, s % page] = normal(g, (n, H_kv, D), dtype)
        self.table = torch.from_numpy(self.table_np).cuda()
        self.length = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.n_new = None if n_new is None else torch.tensor(self.new, dtype=torch.int32, device="cuda")
        self.q = normal(g, (B, T, H, D), dtype)
        self.tree = None
        if tree == "random" and T:
            parents = torch.tensor([[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)]).view(B, T)
            self.tree = bsa.tree_words(parents).cuda()
        self.scale = 1.0 / math.sqrt(D)

    def cache(self):
        return bsa.PagedCache(self.k, self.v, self.table, self.length)

    def seqs(self, which=None):
        """Each sequence's rows in slot order, fp64 [slots, H_kv, D]."""
        x = f64(self.k if which is None else which)
        out = []
        for b in range(self.B):
            n = self.lengths[b] + self.new[b]
            s = np.arange(n)
            out.append(x[self.table_np[b][s // self.page], s % self.page])
        return out


def attend_tolerance(O, mass, n_keys, vmax, dtype):
    """O = sum p v / sum p with p rounded to the tensors' type (relative half step
    u, numerator and denominator with the same rounded p) and the result rounded:
    u |O| for the result, u (mass + |O|) for the weights, fp16 weights below its
    subnormal step another n 2^-25 vmax, and 2^-17 mass for the fp32 exponents and
    sums (|s| 2^-23 with |s| <= 40, and n 2^-24)."""
    u = HALF_STEP[dtype]
    tol = u * np.abs(O) + 1.02 * u * (mass + np.abs(O)) + 2.0 ** -17 * mass + 1e-7
    return tol + (n_keys * 2.0 ** -25 * vmax if dtype == "fp16" else 0.0)


def exponent_tolerance(q, seq_k, scale, lse_max=20.0):
    """Absolute error of scale q.k in fp32: D rounded (or truncated) additions of
    exact products, D 2^-23 scale sum|q k| <= D 2^-23 scale |q||k|, and the last
    roundings of the exponent, 4 2^-24 of |s| + |lse|."""
    D = q.shape[-1]
    qn = np.sqrt((q ** 2).sum(-1)).max(initial=0.0)
    kn = max((np.sqrt((np.nan_to_num(k) ** 2).sum(-1)).max(initial=0.0) for k in seq_k), default=0.0)
    return D * 2.0 ** -23 * scale * qn * kn + 2.0 ** -22 * (scale * qn * kn + lse_max)
