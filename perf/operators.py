"""Cases, inputs and plain forms of the rotary, paged-cache attention and cache-eviction operators.

``run`` computes an operator in elementary torch operations (fp32, rounded once
at the end) or, where ``own`` is set, through the package's entry points."""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # the positions of the 81-frame 720p video shape (21 x 45 x 80 latent tokens), q and k, training forward
        dict(name="rope_video", op="rope", B=1, S=75600, H=40, H_kv=40, D=128, axes=3, pairs=64, layout="interleaved",
             inverse=False, dtype="bf16"),
        # the gradient of the positions of the grouped-query training shape, half-split pairs
        dict(name="rope_gqa_bwd", op="rope", B=1, S=8192, H=16, H_kv=4, D=128, axes=3, pairs=64, layout="halves",
             inverse=True, dtype="bf16"),
        # a few images (height, width), an odd token count, three quarters of a small head rotated
        dict(name="rope_image_fp16", op="rope", B=3, S=1021, H=6, H_kv=6, D=64, axes=2, pairs=24, layout="halves",
             inverse=False, dtype="fp16"),
        # drafted tokens of a serving batch: rotate q, rotate k into the cache, v into the cache
        dict(name="append_draft", op="append", B=16, T=8, H=16, H_kv=4, D=128, page=64, keys=8192, axes=3, pairs=64,
             layout="halves", dtype="bf16"),
        # a short tree on a short cache: the latency of one call
        dict(name="tree_tiny_fp16", op="attend", B=1, T=7, H=2, H_kv=2, D=64, page=16, keys=250, dtype="fp16"),
        # plain decoding, one token a sequence
        dict(name="tree_one_token", op="attend", B=8, T=1, H=16, H_kv=4, D=128, page=64, keys=8192, dtype="bf16"),
        # drafted trees over long ragged caches
        dict(name="tree_draft_long", op="attend", B=16, T=32, H=16, H_kv=4, D=128, page=128, keys=33002, dtype="bf16"),
        # the widest tree, a group of five heads, the video's tokens as the cache
        dict(name="tree_wide", op="attend", B=2, T=64, H=40, H_kv=8, D=128, page=256, keys=75600, dtype="bf16"),
        # accumulating the weights of one decoded token
        dict(name="weigh_one_token", op="weigh", B=8, T=1, H=16, H_kv=4, D=128, page=64, keys=8192, dtype="bf16"),
        # accumulating the weights of drafted trees over long caches
        dict(name="weigh_draft_long", op="weigh", B=4, T=16, H=40, H_kv=8, D=128, page=128, keys=75600, dtype="bf16"),
        # a decoding step at the budget: one key leaves each head
        dict(name="evict_step", op="evict", B=16, H_kv=4, D=128, page=64, keys=4097, budget=4096, sinks=4, recent=256,
             dtype="bf16"),
        # a long prompt's cache cut to half
        dict(name="evict_half", op="evict", B=2, H_kv=8, D=128, page=128, keys=65536, budget=32768, sinks=4, recent=1024,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "weigh", "evict"])
    D = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    layout = rng.choice(["interleaved", "halves"])
    axes = rng.choice([1, 2, 3])
    pairs = rng.choice([D // 2, D // 2, D // 4, D // 2 - 8])
    if op == "rope":
        B = rng.choice([1, 1, 2, 3])
        H = H_kv * G
        S = _log(rng, 1, min(75600, int(3.5e8 / (B * H * D))))
        return dict(op=op, B=B, S=S, H=H, H_kv=H_kv, D=D, axes=axes, pairs=pairs, layout=layout,
                    inverse=rng.random() < 0.5, dtype=dtype)
    B = _log(rng, 1, 48)
    T = rng.choice([1, 1, _log(rng, 2, 64)])
    # at most the largest listed calls' cache, and their products
    most = min(int(2.5e8 / (B * H_kv * D)), int(2.5e8 / (B * H_kv * G * T)), 80000)
    keys = _log(rng, 1, max(2, most))
    if op == "append":
        return dict(op=op, B=B, T=T, H=H_kv * G, H_kv=H_kv, D=D, page=page, keys=min(keys, 8192), axes=axes, pairs=pairs,
                    layout=layout, dtype=dtype)
    if op in ("attend", "weigh"):
        return dict(op=op, B=B, T=T, H=H_kv * G, H_kv=H_kv, D=D, page=page, keys=keys, dtype=dtype)
    keys = max(keys, 16)
    budget = keys - 1 if rng.random() < 0.4 else max(8, int(keys * rng.uniform(0.1, 0.95)))
    return dict(op=op, B=B, H_kv=H_kv, D=D, page=page, keys=keys, budget=budget, sinks=min(4, budget // 4),
                recent=budget // rng.choice([2, 4, 16]), dtype=dtype)


# ----------------------------------------------------------------- the inputs

def _lengths(case):
    """Ragged lengths from the longest down to about half of it (in some order of the seed's)."""
    B, n = case["B"], case["keys"]
    return [max(1, n - (n // 2) * i // B) for i in range(B)]


def _news(case):
    """How many of a sequence's T rows are real: all, or a few fewer."""
    T = case.get("T", 0)
    return [max(1, T - (T // 4) * (i % 3) // 2) for i in range(case["B"])]


def _tables(case, gen):
    """Frequencies theta^(-2k/d) of each pair, pairs dealt to the axes in sections, and the axis of each pair."""
    n, axes = case["pairs"], case["axes"]
    share = [n // axes + (1 if a < n % axes else 0) for a in range(axes)]
    freq, axis = [], []
    for a, m in enumerate(share):
        freq += [10000.0 ** (-2.0 * k / (2 * m)) for k in range(m)]
        axis += [a] * m
    return (torch.tensor(freq, dtype=torch.float64, device=DEV), torch.tensor(axis, dtype=torch.int32, device=DEV))


def _grid_positions(B, S, axes, gen):
    """Positions of a token grid (time slowest), each sequence from a start of its own."""
    w = 80 if axes == 3 else max(1, math.isqrt(S))
    h = 45
    s = torch.arange(S, device=DEV)
    rows = {1: [s], 2: [s // w, s % w], 3: [s // (w * h), (s // w) % h, s % w]}[axes]
    start = torch.randint(0, 1000, (axes, B, 1), generator=gen, device=DEV)
    return (torch.stack(rows)[:, None, :] + start).to(torch.int32).contiguous()


def _trees(B, T, gen):
    """Each token's ancestors and itself as bits: a random tree, most tokens hanging deep."""
    r = torch.rand(B, T, generator=gen, device=DEV)
    idx = torch.arange(T, device=DEV)
    parent = torch.where(r < 0.6, idx[None] - 1, (r * (idx[None] + 1)).long() - 1)
    words = torch.zeros(B, T, dtype=torch.int64, device=DEV)
    for t in range(T):
        par = parent[:, t]
        up = torch.where(par >= 0, words.gather(1, par.clamp(min=0)[:, None])[:, 0], torch.zeros_like(par))
        words[:, t] = up | torch.tensor(1 << t if t < 63 else -(1 << 63), dtype=torch.int64, device=DEV)
    return words


def _scores_lse(st):
    """The LSE of every row over the keys it sees (an input of the weighing), sequence by sequence."""
    out = []
    for b in range(st["q"].shape[0]):
        sub = {k: (v[b:b + 1] if k in ("q", "table", "length", "tree", "new") else v) for k, v in st.items()}
        s, seen = _masked_scores(sub)
        out.append(torch.logsumexp(torch.where(seen, s, -math.inf), -1))
    lse = torch.cat(out)
    B, T, H, _ = st["q"].shape
    return lse.view(B, -1, T, H // lse.shape[1]).permute(0, 1, 3, 2).reshape(B, H, T).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dt if math.prod(shape) > 1 << 26 else None).to(dt)

    st = {"case": dict(case)}
    B, D = case["B"], case["D"]
    if case["op"] == "rope":
        S = case["S"]
        st.update(q=normal(B, S, case["H"], D), k=normal(B, S, case["H_kv"], D))
        st["freq"], st["axis"] = _tables(case, gen)
        st["pos"] = _grid_positions(B, S, case["axes"], gen)
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        return st

    # a paged cache whose sequences' pages lie anywhere, with room for the new tokens
    page, H_kv, T = case["page"], case["H_kv"], case.get("T", 0)
    per = -(-(case["keys"] + T) // page)
    n_pages = B * per + 1
    st["kc"], st["vc"] = normal(n_pages, page, H_kv, D), normal(n_pages, page, H_kv, D)
    st["table"] = torch.randperm(n_pages, generator=gen, device=DEV)[:B * per].view(B, per).to(torch.int32)
    order = torch.randperm(B, generator=gen, device=DEV)
    st["length"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)[order].contiguous()
    if case["op"] == "evict":
        cap, n = per * page, st["length"][:, None, None]
        # weights as they gather: a few heavy keys, a long light tail, and equal ones
        s = torch.randn(B, H_kv, cap, generator=gen, device=DEV).mul(2).exp()
        s = torch.where(s < 0.05, torch.zeros_like(s), s)
        slot = torch.arange(cap, device=DEV, dtype=torch.int32)
        there = slot < n
        st["scores"] = torch.where(there, s, 0.0)
        # the head and the tail of a sequence in any slot, as earlier evictions leave them
        head = torch.arange(H_kv, device=DEV, dtype=torch.int32)[:, None]
        mixed = (slot * torch.where(n % 7 == 0, 1, 7) + head) % n
        st["pos"] = torch.where(there, mixed, -1).to(torch.int32).contiguous()
        st["next_pos"] = st["length"].clone()
        st["scores_out"], st["pos_out"] = torch.zeros_like(st["scores"]), torch.full_like(st["pos"], -1)
        st["length_out"] = torch.zeros_like(st["length"])
        return st

    st["new"] = torch.tensor(_news(case), dtype=torch.int32, device=DEV)[order].contiguous()
    st["q"] = normal(B, T, case["H"], D)
    if case["op"] == "append":
        st["k"], st["v"] = normal(B, T, H_kv, D), normal(B, T, H_kv, D)
        st["freq"], st["axis"] = _tables(case, gen)
        start = st["length"][None, :, None] + torch.arange(T, device=DEV)
        st["pos"] = (start * torch.arange(1, case["axes"] + 1, device=DEV)[:, None, None]).to(torch.int32).contiguous()
        st["q_out"] = torch.empty_like(st["q"])
        return st
    st["tree"] = _trees(B, T, gen)
    if case["op"] == "weigh":
        st["lse"] = _scores_lse(st)
        st["scores"] = torch.rand(B, H_kv, per * page, generator=gen, device=DEV) * 0.01
        st["scores_out"] = st["scores"].clone()
    else:
        st["out"] = torch.empty_like(st["q"])
        st["lse_out"] = torch.empty(B, case["H"], T, dtype=torch.float32, device=DEV)
    return st


# ----------------------------------------------------------------- the plain forms

def _rotate(x, pos, freq, axis, layout, inverse):
    """x [B, S, H, D] turned pair by pair by the angle pos[axis[p]] * freq[p] (the other elements as they are)."""
    n = freq.numel()
    angle = pos.to(torch.float64)[axis.long()].permute(1, 2, 0) * freq
    c = torch.cos(angle).float()[:, :, None, :]
    s = torch.sin(angle).float()[:, :, None, :]
    s = -s if inverse else s
    y = x.float()
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if layout == "interleaved" else (y[..., :n], y[..., n:2 * n])
    u, w = a * c - b * s, a * s + b * c
    turned = torch.stack((u, w), -1).flatten(-2) if layout == "interleaved" else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., 2 * n:]), -1).to(x.dtype)


def _gathered(cache, table):
    """The cache's pages of each sequence in order, fp32 [B, H_kv, capacity, D]."""
    x = cache[table.long()]
    return x.flatten(1, 2).permute(0, 2, 1, 3).float()


def _masked_scores(st):
    """Scaled products [B, H_kv, T * G, capacity] of every row with every slot, and which of them count."""
    q, kc = st["q"], st["kc"]
    B, T, H, D = q.shape
    H_kv = kc.shape[2]
    G = H // H_kv
    k = _gathered(kc, st["table"])
    rows = q.float().view(B, T, H_kv, G, D).permute(0, 2, 1, 3, 4).reshape(B, H_kv, T * G, D)
    s = torch.matmul(rows, k.transpose(-1, -2)) / math.sqrt(D)
    slot = torch.arange(k.shape[2], device=q.device)
    n, new = st["length"].long()[:, None, None], st["new"].long()[:, None, None]
    ahead = slot - n
    bit = (st["tree"][:, :, None] >> ahead.clamp(0, 63)) & 1
    seen = (ahead < 0) | ((ahead < new) & (ahead < 64) & (bit == 1))
    seen = seen & (torch.arange(T, device=q.device)[None, :, None] < new)
    return s, seen[:, None].expand(B, H_kv, T, -1).repeat_interleave(G, 2)


def _by_head(x, T):
    """[B, H_kv, T * G, ...] -> [B, T, H, ...]."""
    B, H_kv, R = x.shape[:3]
    x = x.view(B, H_kv, T, R // T, *x.shape[3:])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(st):
    T = st["q"].shape[1]
    s, seen = _masked_scores(st)
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, _gathered(st["vc"], st["table"]))
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return _by_head(o, T).to(st["q"].dtype), _by_head(lse[..., 0], T).transpose(1, 2).contiguous()


def _plain_weigh(st):
    B, T, H, _ = st["q"].shape
    H_kv = st["kc"].shape[2]
    s, seen = _masked_scores(st)
    lse = st["lse"].view(B, H_kv, H // H_kv, T).transpose(2, 3).reshape(B, H_kv, -1, 1)
    return st["scores"] + torch.where(seen, torch.exp(s - lse), 0.0).sum(2)


def _plain_evict(st):
    case = st["case"]
    scores, pos, n = st["scores"], st["pos"], st["length"].long()[:, None, None]
    budget = case["budget"]
    slot = torch.arange(scores.shape[2], device=scores.device)
    there, over = (slot < n).expand_as(scores), n > budget
    first = (pos < case["sinks"]) | (pos >= st["next_pos"][:, None, None] - case["recent"])
    rank = torch.where(there, torch.where(first, math.inf, scores), -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.zeros_like(scores, dtype=torch.bool).scatter(-1, best, True) & there
    hole, mover = (over & (slot < budget) & ~keep).nonzero(), (over & (slot >= budget) & keep).nonzero()
    page = case["page"]
    (b, h, to), fr = hole.unbind(1), mover[:, 2]
    to_at, from_at = st["table"][b, to // page].long(), st["table"][b, fr // page].long()
    st["kc"][to_at, to % page, h] = st["kc"][from_at, fr % page, h]
    st["vc"][to_at, to % page, h] = st["vc"][from_at, fr % page, h]
    stays = there & ((slot < budget) | ~over)
    new_scores, new_pos = torch.where(stays, scores, 0.0), torch.where(stays, pos, -1)
    new_scores[b, h, to], new_pos[b, h, to] = scores[b, h, fr], pos[b, h, fr]
    return st["kc"], st["vc"], new_scores, new_pos, torch.clamp(st["length"], max=budget)


def _plain_append(st):
    case = st["case"]
    T, page = case["T"], case["page"]
    turn = (st["pos"], st["freq"], st["axis"], case["layout"], False)
    t = torch.arange(T, device=st["k"].device)
    b, t = (t[None] < st["new"][:, None]).nonzero().unbind(1)
    slot = st["length"].long()[b] + t
    at = st["table"][b, slot // page].long()
    st["kc"][at, slot % page] = _rotate(st["k"], *turn)[b, t]
    st["vc"][at, slot % page] = st["v"][b, t]
    return _rotate(st["q"], *turn), st["kc"], st["vc"]


def _plain_rope(st):
    case = st["case"]
    turn = (st["pos"], st["freq"], st["axis"], case["layout"], case["inverse"])
    return _rotate(st["q"], *turn), _rotate(st["k"], *turn)


def _own_run(st):
    import block_sparse_attention_map_b200 as bsa

    case = st["case"]
    if case["op"] == "rope":
        call = bsa.rope_bwd if case["inverse"] else bsa.rope
        return call(st["q"], st["k"], st["pos"], st["freq"], st["axis"], layout=case["layout"], q_out=st["q_out"],
                    k_out=st["k_out"])
    cache = st.get("cache")
    if cache is None:  # the handle a serving program keeps for the life of its cache
        cache = st["cache"] = bsa.PagedCache(st["kc"], st["vc"], st["table"], st["length"])
    if case["op"] == "append":
        q = cache.append(st["k"], st["v"], q=st["q"], rope=(st["pos"], st["freq"], st["axis"], case["layout"]),
                         n_new=st["new"], q_out=st["q_out"])
        return q, st["kc"], st["vc"]
    if case["op"] == "attend":
        return cache.attend(st["q"], tree=st["tree"], n_new=st["new"], out=st["out"], lse=st["lse_out"])
    if case["op"] == "weigh":
        return cache.weigh(st["q"], st["lse"], st["scores"], tree=st["tree"], n_new=st["new"], out=st["scores_out"])
    scores, pos, length = cache.evict(st["scores"], st["pos"], st["next_pos"], case["budget"], sinks=case["sinks"],
                                      recent=case["recent"], scores_out=st["scores_out"], pos_out=st["pos_out"],
                                      length_out=st["length_out"])
    return st["kc"], st["vc"], scores, pos, length


def run(state):
    if own:
        return _own_run(state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, D, op = case["B"], case["D"], case["op"]
    if op == "rope":
        n = B * case["S"] * (case["H"] + case["H_kv"])
        return {"bytes": 4 * n * D + 4 * case["axes"] * B * case["S"], "flops": 6 * n * case["pairs"]}
    H_kv = case["H_kv"]
    lengths = _lengths(case)
    if op == "evict":
        # which rows move goes by the scores: with the heaviest keys anywhere, the same share of the kept rows as
        # of all rows lies behind the budget
        moved = sum(min(case["budget"], n - case["budget"]) * case["budget"] / n for n in lengths if n > case["budget"])
        return {"bytes": H_kv * (8 * sum(lengths) + 8 * sum(min(n, case["budget"]) for n in lengths) + 8 * D * moved),
                "flops": 0}
    T, H, new = case["T"], case["H"], _news(case)
    if op == "append":
        return {"bytes": 4 * B * T * H * D + 8 * sum(new) * H_kv * D + 4 * case["axes"] * B * T,
                "flops": 6 * case["pairs"] * (B * T * H + sum(new) * H_kv)}
    keys = sum(n + m for n, m in zip(lengths, new))
    pairs = sum((n + m) * m for n, m in zip(lengths, new)) * H
    if op == "weigh":
        return {"bytes": 2 * keys * H_kv * D + 8 * keys * H_kv + 2 * sum(new) * H * D, "flops": 2 * pairs * D}
    return {"bytes": 4 * keys * H_kv * D + 4 * B * T * H * D + 4 * B * T * H, "flops": 4 * pairs * D}


# ----------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](case, st)


def _exact_turn(x, st, layout, back):
    """Pairs as complex numbers times exp(i angle)."""
    n = st["freq"].numel()
    out = x.double()
    first = torch.arange(n, device=x.device) * (2 if layout == "interleaved" else 1)
    second = first + (1 if layout == "interleaved" else n)
    for a in range(st["pos"].shape[0]):
        mine = (st["axis"] == a).nonzero()[:, 0]
        angle = st["pos"][a].double()[:, :, None] * st["freq"][mine]
        z = torch.polar(torch.ones_like(angle), -angle if back else angle)[:, :, None]
        z = torch.complex(out[..., first[mine]], out[..., second[mine]]) * z
        out[..., first[mine]], out[..., second[mine]] = z.real, z.imag
    return out


def _exact_rope(case, st):
    return tuple(_exact_turn(st[x], st, case["layout"], case["inverse"]) for x in ("q", "k"))


def _exact_append(case, st):
    kc, vc = st["kc"].double(), st["vc"].double()
    k = _exact_turn(st["k"], st, case["layout"], False)
    table, length, new = (st[x].tolist() for x in ("table", "length", "new"))
    for b in range(case["B"]):
        for t in range(new[b]):
            p, r = divmod(length[b] + t, case["page"])
            kc[table[b][p], r], vc[table[b][p], r] = k[b, t], st["v"][b, t].double()
    return _exact_turn(st["q"], st, case["layout"], False), kc, vc


def _exact_sequences(case, st):
    """Sequence by sequence and kv head by kv head: rows [T', G, D], keys and values [n, D] in 64 bits, and what is seen [T', n]."""
    H_kv = case["H_kv"]
    G = case["H"] // H_kv
    for b, (n, m) in enumerate(zip(st["length"].tolist(), st["new"].tolist())):
        slot = torch.arange(n + m, device=DEV)
        at = (st["table"][b].long()[slot // case["page"]], slot % case["page"])
        words = [w & ((1 << 64) - 1) for w in st["tree"][b].tolist()]
        seen = torch.tensor([[(words[t] >> j) & 1 for j in range(m)] for t in range(m)], dtype=torch.bool, device=DEV)
        seen = torch.cat((torch.ones(m, n, dtype=torch.bool, device=DEV), seen), 1)
        for h in range(H_kv):
            yield (b, m, h, slice(h * G, h * G + G), st["q"][b, :m, h * G:h * G + G].double(),
                   st["kc"][at[0], at[1], h].double(), st["vc"][at[0], at[1], h].double(), seen)


def _exact_attend(case, st):
    B, T, H, D = st["q"].shape
    o = torch.zeros(B, T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=DEV)
    for b, m, h, hs, q, k, v, seen in _exact_sequences(case, st):
        s = torch.einsum("tgd,nd->tgn", q, k) / math.sqrt(D)
        s = s.masked_fill(~seen[:, None], -math.inf)
        z = torch.logsumexp(s, -1)
        o[b, :m, hs] = torch.einsum("tgn,nd->tgd", torch.exp(s - z[..., None]), v)
        lse[b, hs, :m] = z.T
    return o, lse


def _exact_weigh(case, st):
    out = st["scores"].double()
    for b, m, h, hs, q, k, v, seen in _exact_sequences(case, st):
        s = torch.einsum("tgd,nd->tgn", q, k) / math.sqrt(case["D"])
        w = torch.exp(s - st["lse"][b, hs, :m].T.double()[..., None]) * seen[:, None]
        out[b, h, :k.shape[0]] += w.sum((0, 1))
    return out


def _exact_evict(case, st):
    budget, page = case["budget"], case["page"]
    scores, pos = st["scores"].double().cpu().numpy(), st["pos"].cpu().numpy()
    lengths, table = st["length"].cpu().numpy(), st["table"].cpu().numpy()
    nexts = st["next_pos"].cpu().numpy()
    kc, vc = st["kc"].double(), st["vc"].double()
    new_s, new_p = np.zeros_like(scores), np.full_like(pos, -1)
    for b, n in enumerate(lengths):
        for h in range(case["H_kv"]):
            s, p = scores[b, h, :n], pos[b, h, :n]
            src = np.arange(min(n, budget))
            if n > budget:
                must = (p < case["sinks"]) | (p >= nexts[b] - case["recent"])
                kept = np.lexsort((np.arange(n), -s, ~must))[:budget]
                gone = np.setdiff1d(np.arange(budget), kept)
                late = np.sort(kept[kept >= budget])
                src[gone] = late
                to, fr = torch.from_numpy(gone).to(DEV), torch.from_numpy(late).to(DEV)
                pages = torch.from_numpy(table[b].astype(np.int64)).to(DEV)
                kc[pages[to // page], to % page, h] = kc[pages[fr // page], fr % page, h]
                vc[pages[to // page], to % page, h] = vc[pages[fr // page], fr % page, h]
            new_s[b, h, :len(src)], new_p[b, h, :len(src)] = s[src], p[src]
    return (kc, vc, torch.from_numpy(new_s), torch.from_numpy(new_p),
            torch.from_numpy(np.minimum(lengths, budget).astype(np.int32)))
