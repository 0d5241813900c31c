"""What the binding of the positions and the paged cache checks before it calls
the library, without a GPU: CPU tensors stand in for CUDA ones, and the call
itself is recorded instead of made."""

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
