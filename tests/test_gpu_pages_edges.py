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
