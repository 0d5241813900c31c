"""The C ABI of the positions and the paged cache without a GPU: struct layouts,
workspace sizes, and every argument error before anything touches CUDA; and the
oracle's own pins."""

import ctypes
import math
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

from block_sparse_attention_map_b200 import _binding as bd
from block_sparse_attention_map_b200 import _serving as sv
from oracle import serving as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(bd.LIB_PATH):
        from block_sparse_attention_map_b200 import build
        build.build()
    return bd.lib()


STRUCTS = {"bsa_rope_spec": sv.RopeSpec, "bsa_tokens": sv.Tokens, "bsa_cache": sv.Cache, "bsa_evict_spec": sv.EvictSpec}


def test_ctypes_structs_match_c_layout():
    lines = []
    for c, py in STRUCTS.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"bsa.h\"\nint main(void) {" + "\n".join(lines) + "return 0; }"
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "l.c"), "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), os.path.join(d, "l.c"), "-o", os.path.join(d, "l")], check=True)
        out = subprocess.run([os.path.join(d, "l")], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.splitlines())
    for c, py in STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c}.{f}"]) == getattr(py, f).offset, (c, f)


def cache(**kw):
    c = sv.Cache(100, 16, 2, 64, 0, 3, 20)
    c.k, c.v, c.page_table, c.length = 4096, 8192, 256, 512
    for n, x in kw.items():
        if isinstance(x, tuple):
            getattr(c, n)[:] = x
        else:
            setattr(c, n, x)
    return c


def tokens(**kw):
    t = sv.Tokens(3, 4, 8, 2, 64, 0)
    for n, x in kw.items():
        if isinstance(x, tuple):
            getattr(t, n)[:] = x
        else:
            setattr(t, n, x)
    return t


def rope_spec(**kw):
    r = sv.RopeSpec(2, 32, 0, 0)
    r.inv_freq, r.axis, r.pos = 64, 128, 256
    for n, x in kw.items():
        if isinstance(x, tuple):
            getattr(r, n)[:] = x
        else:
            setattr(r, n, x)
    return r


WS = (4096, 1 << 30)
NODEV = 9


def size(c, budget=0):
    n = ctypes.c_size_t(0)
    return sv._fn("bsa_cache_workspace_size")(c, budget, ctypes.byref(n)), n.value


def test_workspace_sizes():
    rc, base = size(cache())
    assert rc == 0 and base >= 256 and base % 256 == 0
    rc, n = size(cache(), 100)
    assert rc == 0 and n >= base and n >= 256 + 6 * 100 * 16
    assert size(cache(), 1 << 30)[0] == 0
    assert size(cache(), -1)[0] == 1
    assert size(cache(max_pages=1 << 26))[0] == 0 and size(cache(max_pages=(1 << 26) + 1))[0] == 2


def test_a_workspace_of_one_budget_holds_every_smaller_one():
    # capacity 32768 * 16: more slots can move at budget 2^18 than at any other
    c, e = cache(max_pages=32768, B=16), sv.EvictSpec(10, 2, 3)
    e.next_pos = e.score_in = e.pos_in = e.score_out = e.pos_out = e.length_out = 64
    budgets = (1, 1000, 1 << 17, 1 << 18, 3 << 17, (1 << 19) - 1, 1 << 19, 1 << 20)
    sizes = [size(c, n)[1] for n in budgets]
    assert sizes == sorted(sizes)
    for i, n in enumerate(sizes):
        for small in budgets[:i + 1]:
            e.budget = small
            assert sv._fn("bsa_cache_evict")(c, e, 4096, n, None) == NODEV, (budgets[i], small)


@pytest.mark.parametrize("kw,code", [
    (dict(n_pages=0), 1), (dict(page_size=0), 1), (dict(max_pages=0), 1), (dict(H_kv=0), 1), (dict(B=-1), 1),
    (dict(D=96), 2), (dict(dtype=2), 2), (dict(page_size=12), 2), (dict(page_size=4), 2), (dict(page_size=1 << 17), 2),
    (dict(n_pages=(1 << 30) + 1), 2), (dict(k_stride=(2048, 128, 60)), 2), (dict(v_stride=(2048, 0, 64)), 1),
    (dict(k_stride=(1 << 40, 128, 64)), 2), (dict(table_stride=19), 1), (dict(table_stride=-1), 1), (dict(H_kv=1 << 24), 2)])
def test_cache_checks(kw, code):
    assert size(cache(**kw))[0] == code
    assert sv._fn("bsa_cache_attend")(cache(**kw), tokens(), 16, 32, 64, *WS, None) == code


def test_calls_reject_bad_arguments_before_cuda(L):
    before = L.bsa_launch_count()
    rope, append = sv._fn("bsa_rope"), sv._fn("bsa_cache_append")
    attend, weigh, evict = sv._fn("bsa_cache_attend"), sv._fn("bsa_cache_weigh"), sv._fn("bsa_cache_evict")
    t, r, c = tokens(), rope_spec(), cache()
    # valid calls get as far as the device
    assert rope(t, r, 16, 32, 48, 64, None) == NODEV
    assert rope(t, r, None, None, 48, 64, None) == NODEV
    assert append(c, t, r, 16, 32, 48, 64, *WS, None) == NODEV
    assert append(c, t, None, None, None, 48, 64, *WS, None) == NODEV
    assert attend(c, t, 16, 32, 64, *WS, None) == NODEV
    assert weigh(c, t, 16, 32, 64, 64, *WS, None) == NODEV
    e = sv.EvictSpec(10, 2, 3)
    e.next_pos = e.score_in = e.pos_in = e.score_out = e.pos_out = e.length_out = 64
    assert evict(c, e, *WS, None) == NODEV
    # tokens
    for kw, code in ((dict(B=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(H_kv=3), 1), (dict(dtype=5), 2), (dict(D=24), 2),
                     (dict(D=272), 2), (dict(q_stride=(2048, 512, 4)), 2), (dict(ko_stride=(-8, 128, 64)), 1),
                     (dict(T=1 << 28), 2)):
        assert rope(tokens(**kw), r, 16, 32, 48, 64, None) == code, kw
    assert rope(None, r, 16, 32, 48, 64, None) == 1 and rope(t, None, 16, 32, 48, 64, None) == 1
    for kw in (dict(H_kv=4), dict(D=128), dict(dtype=1), dict(B=2), dict(T=65)):
        assert attend(c, tokens(**kw), 16, 32, 64, *WS, None) == 1, kw
        assert weigh(c, tokens(**kw), 16, 32, 64, 64, *WS, None) == 1, kw
        assert append(c, tokens(**kw), None, None, None, 48, 64, *WS, None) == (NODEV if kw == dict(T=65) else 1)
    assert attend(c, tokens(H=2 * 129), 16, 32, 64, *WS, None) == 2
    # the rotation
    for kw, code in ((dict(n_axes=0), 1), (dict(n_axes=9), 1), (dict(n_pairs=0), 1), (dict(n_pairs=33), 1), (dict(layout=2), 1),
                     (dict(inverse=2), 1), (dict(layout=1, n_pairs=12), 2), (dict(inv_freq=None), 1), (dict(axis=None), 1),
                     (dict(pos=None), 1), (dict(inv_freq=68), 2), (dict(axis=130), 2), (dict(pos_stride=(-1, 4)), 1)):
        assert rope(t, rope_spec(**kw), 16, 32, 48, 64, None) == code, kw
        assert append(c, t, rope_spec(**kw), 16, 32, 48, 64, *WS, None) == code, kw
    # pointers: null, one of a pair, misaligned
    for q in ((None, None, None, None), (16, None, 48, 64), (None, 16, 48, 64), (16, 32, 48, None)):
        assert rope(t, r, *q, None) == 1
    for q in ((8, 32, 48, 64), (16, 40, 48, 64), (16, 32, 52, 64), (16, 32, 48, 66)):
        assert rope(t, r, *q, None) == 2
    for q in ((16, None, 48, 64), (None, None, None, 64), (None, None, 48, None)):
        assert append(c, t, None, *q, *WS, None) == 1
    assert append(c, t, None, None, None, 48, 72, *WS, None) == 2
    assert attend(c, t, None, 32, 64, *WS, None) == 1 and attend(c, t, 16, 32, None, *WS, None) == 1
    assert attend(c, t, 16, 36, 64, *WS, None) == 2 and attend(c, t, 16, 32, 66, *WS, None) == 2
    assert attend(c, tokens(tree=68), 16, 32, 64, *WS, None) == 2 and attend(c, tokens(n_new=66), 16, 32, 64, *WS, None) == 2
    assert weigh(c, t, 16, None, 64, 64, *WS, None) == 1 and weigh(c, t, 16, 32, 64, 65, *WS, None) == 2
    for name in ("k", "v", "page_table", "length"):
        assert attend(cache(**{name: None}), t, 16, 32, 64, *WS, None) == 1
        assert attend(cache(**{name: 4098}), t, 16, 32, 64, *WS, None) == 2
    # workspace
    assert attend(c, t, 16, 32, 64, None, 1 << 30, None) == 1
    assert attend(c, t, 16, 32, 64, 4096 + 16, 1 << 30, None) == 1
    assert attend(c, t, 16, 32, 64, 4096, 255, None) == 3
    assert evict(c, e, 4096, size(c, 10)[1] - 1, None) == 3
    # eviction
    for kw in (dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(next_pos=None), dict(score_in=None), dict(pos_in=None),
               dict(score_out=None), dict(pos_out=None), dict(length_out=None)):
        x = sv.EvictSpec.from_buffer_copy(e)
        for n, v in kw.items():
            setattr(x, n, v)
        assert evict(c, x, *WS, None) == 1, kw
    assert evict(c, None, *WS, None) == 1
    # empty: checked, then nothing
    for kw in (dict(T=0), dict(B=0)):
        cc = cache(B=kw.get("B", 3), k=None, v=None, page_table=None, length=None)
        assert attend(cc, tokens(**kw), None, None, None, None, 0, None) == 0
        assert weigh(cc, tokens(**kw), None, None, None, None, None, 0, None) == 0
        assert append(cc, tokens(**kw), None, None, None, None, None, None, 0, None) == 0
        assert rope(tokens(**kw), rope_spec(inv_freq=None, axis=None, pos=None), None, None, None, None, None) == 0
        assert attend(cc, tokens(D=128, **kw), None, None, None, None, 0, None) == 1
    assert evict(cache(B=0, k=None), sv.EvictSpec(1), None, 0, None) == 0
    assert L.bsa_launch_count() == before
    assert "cache" in L.bsa_status_string(11).decode()


def test_limits_that_keep_the_kernels_counters_in_range():
    # rows of a rotation: a block's step past the last one is added in 31 bits
    rope, r = sv._fn("bsa_rope"), rope_spec()
    for T, code in (((1 << 31) - (1 << 20), 2), ((1 << 31) - 1, 2), ((1 << 31) - (1 << 20) - 1, NODEV)):
        assert rope(tokens(B=1, H=1, H_kv=1, T=T), r, 16, 32, 48, 64, None) == code
    # sequences of the attention: its CTAs, and each joined row, read every length
    for B, code in (((1 << 16) + 1, 2), (1 << 16, NODEV)):
        assert sv._fn("bsa_cache_attend")(cache(B=B), tokens(B=B), 16, 32, 64, *WS, None) == code
        assert sv._fn("bsa_cache_weigh")(cache(B=B), tokens(B=B), 16, 32, 64, 64, *WS, None) == code


def test_tree_words():
    p = torch.tensor([[-1, 0, 0, 2, -1], [-1, -1, 1, 2, 3]])
    assert sv.tree_words(p).tolist() == [[1, 3, 5, 13, 16], [1, 2, 6, 14, 30]]
    chain = torch.arange(-1, 63)[None]
    w = sv.tree_words(chain)[0].tolist()
    assert w[63] == -1 and w[62] == (1 << 63) - 1
    for bad in ([[0]], [[-2]], [[-1, 1]]):
        with pytest.raises(ValueError):
            sv.tree_words(torch.tensor(bad))
    with pytest.raises(ValueError):
        sv.tree_words(torch.zeros(1, 65, dtype=torch.int64))


def test_oracle_pins():
    """A quarter turn, a dense softmax over a chain, weights that add to one per row, and a worked eviction."""
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 1, 8)
    y = oracle.rope(x, np.array([[[1]]]), np.array([math.pi / 2] * 2), np.array([0, 0]), "interleaved")
    assert np.allclose(y[0, 0, 0], [-1, 0, -3, 2, 4, 5, 6, 7])
    y = oracle.rope(x, np.array([[[1]]]), np.array([math.pi / 2] * 2), np.array([0, 0]), "halves")
    assert np.allclose(y[0, 0, 0], [-2, -3, 0, 1, 4, 5, 6, 7])
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((1, 3, 2, 4)), rng.standard_normal((8, 1, 4)), rng.standard_normal((8, 1, 4))
    w = oracle.words_or_chain(None, 1, 3)
    O, lse, _ = oracle.attend(q, [k], [v], [5], [3], w, 0.5)
    s = torch.from_numpy(np.einsum("thd,jd->htj", q[0], k[:, 0])) * 0.5
    s = s.masked_fill(torch.arange(8)[None] > 5 + torch.arange(3)[:, None], -math.inf)
    assert np.allclose(O[0], np.einsum("htj,jd->thd", torch.softmax(s, -1).numpy(), v[:, 0]))
    assert np.allclose(lse[0], torch.logsumexp(s, -1).numpy())
    sc = oracle.weigh(np.zeros((1, 1, 10)), q, [k], lse, [5], [3], w, 0.5)
    assert np.isclose(sc.sum(), 6) and (sc[0, 0, 8:] == 0).all()
    # five keys, keep three: position 0 is a sink, 9 is recent, then the higher score of the rest
    assert oracle.evict_sources([0.1, 5, 2, 0.2, 9], [3, 0, 4, 9, 5], 5, 3, 1, 1, 10) == [3, 1, 4]
