"""GPU tests of the cache page operators where calls meet: host threads, a pool that runs out, other owners of pages."""

import threading

import pytest
import torch

from tests._pages_model import Pool
from tests.test_gpu_pages import _dev, _same, _state, _ws

pytestmark = pytest.mark.gpu


def test_threads_with_tables_of_different_sizes(cuda_lib):
    """Calls of two host threads at once, each with its own state, stream and workspace, one with far more rows: the
    shared memory that one asks for does not depend on what the other does in between."""
    dash = cuda_lib
    lib, failed = dash.load(), {}

    def run(rows):
        table = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
        seqlens, refs = torch.zeros(rows, dtype=torch.int32, device="cuda"), _dev([0] * 4)
        ws = torch.empty(dash.pages_workspace_size(rows, 1, 4), dtype=torch.uint8, device="cuda")
        slots, none, src, dst = (torch.arange(rows, dtype=torch.int32, device="cuda") for _ in range(4))
        none.zero_()
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        state = (table.data_ptr(), rows, 1, seqlens.data_ptr(), refs.data_ptr(), 4)
        tail = (ws.data_ptr(), ws.numel(), stream.cuda_stream)
        free = (*state, slots.data_ptr(), rows, 64, *tail)
        grow = (*state, none.data_ptr(), 64, src.data_ptr(), dst.data_ptr(), *tail)
        failed[rows] = 0
        for _ in range(10000):
            failed[rows] += lib.dash_attn_pages_free(*free) != 0
            failed[rows] += lib.dash_attn_pages_grow(*grow) != 0
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(rows,)) for rows in (8192, 5300)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == {8192: 0, 5300: 0}


def test_a_pool_that_runs_out_is_seen(cuda_lib):
    """Growing without a workspace of one's own: the result says whether the sequences grew."""
    dash = cuda_lib
    m = Pool(3, 4, 4, 64)
    m.grow([100, 64, 0])
    table, seqlens, refs = _state(m)
    grown = dash.pages_grow(table, seqlens, refs, _dev([0, 0, 65]), 64)
    assert dash.device_status(grown.workspace) == 6
    _same(m, table, seqlens, refs)
    src, dst = grown
    assert (src == -1).all() and (dst == -1).all()
    want = m.grow([0, 0, 64])
    grown = dash.pages_grow(table, seqlens, refs, _dev([0, 0, 64]), 64)
    assert dash.device_status(grown.workspace) == 0
    assert [t.tolist() for t in grown] == list(want)
    _same(m, table, seqlens, refs)
    ws = _ws(dash, m)
    assert dash.pages_grow(table, seqlens, refs, _dev([0, 0, 0]), 64, workspace=ws).workspace is ws


def test_compaction_beside_another_owner(cuda_lib):
    """Pages that a second table holds move too; its entries follow by the list of moves."""
    dash, block = cuda_lib, 64
    gen = torch.Generator().manual_seed(3)
    ids = torch.randperm(40, generator=gen)
    mine, other = torch.full((2, 5), -1, dtype=torch.int32), torch.full((3, 4), -1, dtype=torch.int32)
    mine[0, :4], mine[1, :5] = ids[:4], ids[4:9]
    other[0, :3], other[1, :2] = ids[9:12], ids[12:14]
    other[2, :2] = mine[0, :2]  # a prefix that both hold
    refs = torch.zeros(40, dtype=torch.int32)
    for t in (mine, other):
        refs += torch.bincount(t[t >= 0].long(), minlength=40).to(torch.int32)
    pool = torch.randn(40, block, 1, 64, device="cuda")
    mine, other, refs, seqlens = mine.cuda(), other.cuda(), refs.cuda(), _dev([4 * block, 5 * block])

    def contents(table):
        return pool[table[table >= 0].long()]

    before = contents(mine), contents(other)
    moved = dash.pages_compact(mine, seqlens, refs, block, inplace=True)
    dash.pages_copy([pool], moved["src"], moved["dst"])
    src, dst = (moved[n][:int(moved["info"][0])].long() for n in ("src", "dst"))
    to = torch.arange(40, device="cuda", dtype=torch.int32)
    to[src] = dst.to(torch.int32)
    other = torch.where(other >= 0, to[other.clamp(min=0).long()], other)
    assert int(mine.max()) < 14 and int(other.max()) < 14 and int(moved["info"][1]) == 14
    assert torch.equal(contents(mine), before[0]) and torch.equal(contents(other), before[1])
    assert int(refs[:14].min()) == 1 and int(refs[14:].max()) == 0 and torch.equal(other[2, :2], mine[0, :2])
