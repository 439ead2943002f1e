"""Checks of the Python binding's arguments, on a machine without a GPU."""

import types

import pytest
import torch

from test_abi_host import FAKE, hq  # noqa: F401  (hq: the fixture)
from test_packed_host import rows, span, write


def paged(hq, **kw):
    return hq.PagedHeadQCache(2, 4, 128, 16, 128, 9, 3, device="cpu", **kw)


@pytest.mark.parametrize("table", [
    torch.zeros(2, 3, dtype=torch.int64),                       # read as pairs of words
    torch.zeros(2, 2, dtype=torch.int32),                       # too short for max_pages
    torch.zeros(1, 3, dtype=torch.int32),                       # a sequence is missing
    torch.zeros(6, dtype=torch.int32),
    torch.zeros(2, 6, dtype=torch.int32)[:, ::2],               # strided
    torch.zeros(2, 3, dtype=torch.int32, device="meta"),        # on another device than the planes
    [[0, 1, 2], [3, 4, 5]],
], ids=["int64", "pages", "sequences", "flat", "strided", "device", "list"])
def test_an_assigned_block_table_is_checked(hq, table):
    c = paged(hq)
    c.struct()
    c.block_table = table
    with pytest.raises(ValueError, match="block_table"):
        c.struct()


def test_from_planes_checks_the_table(hq, monkeypatch):
    """As for every other plane: the table lies on the planes' device."""
    monkeypatch.setattr(hq, "_cuda", lambda t, name: t)
    p = dict(k_codes=torch.zeros(9, 4, 128, 32, dtype=torch.uint8), k_scale=torch.zeros(9, 4, 128, 4),
             k_min=torch.zeros(9, 4, 128, 4), v=torch.zeros(9, 4, 128, 128))
    ok = torch.zeros(2, 3, dtype=torch.int32)
    assert hq.HeadQCache.from_planes(block_table=ok, **p).max_pages == 3
    with pytest.raises(ValueError, match="block_table"):
        hq.HeadQCache.from_planes(block_table=ok.to("meta"), **p)


@pytest.mark.parametrize("kw", [dict(n=2 ** 32 + 1), dict(n=2 ** 31), dict(n=-2 ** 31 - 1), dict(T=2 ** 32 + 5),
                                dict(rows=2 ** 32 + 2)])
def test_sizes_past_32_bits_are_refused(hq, kw):
    """They would wrap to other sizes in the C structures."""
    c = types.SimpleNamespace(B=2, T_cap=64)
    args = dict(seq_lens=None, cu=None, n=1, T=None, rows=2)
    hq._span(c, **args)
    with pytest.raises(ValueError, match="32 bits"):
        hq._span(c, **{**args, **kw})
    kw.pop("rows", None)
    if kw:
        with pytest.raises(ValueError, match="32 bits"):
            hq.tree_workspace(paged(hq), 4, kw.get("n", 1), kw.get("T"))


def test_the_status_of_a_workspace_is_read_on_its_own_device(hq, monkeypatch):
    """Whatever device is current: the stream waited for is the workspace's device's."""
    seen = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(("enter", self.device))

        def __exit__(self, *a):
            seen.append(("exit", self.device))

    def status(ws, stream):
        seen.append(("status", ws.value, stream.value))
        return 0

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream={None: 5}.get(d, 9)))
    monkeypatch.setattr(hq, "lib", lambda: types.SimpleNamespace(headq_workspace_status=status))
    ws = torch.zeros(256, dtype=torch.uint8)
    hq.headq_workspace_status(ws)
    assert seen == [("enter", ws.device), ("status", ws.data_ptr(), 9), ("exit", ws.device)]
    del seen[:]
    hq.headq_workspace_status(ws, stream=types.SimpleNamespace(cuda_stream=7))
    assert seen[1] == ("status", ws.data_ptr(), 7)


def test_a_gathered_write_of_nothing(hq):
    """No packed rows (an empty src has no address), or nothing to take them from."""
    assert write(hq, sp=span(hq, n=4, rows=0, cu=FAKE), src=None, src_rows=7) == 0
    assert write(hq, k=rows(hq, ptr=None), v=rows(hq, ptr=None), src=FAKE, src_rows=0) == 0
    assert write(hq, src=None, src_rows=7) == 1
    assert write(hq, src=FAKE + 4, sp=span(hq, n=4, rows=0, cu=FAKE)) == 1
