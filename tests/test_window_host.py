"""Host-side checks of the dense / sliding-window attention and cache page entry points, and their model (no GPU)."""

import ctypes
import random

import pytest

import sparse_hierarchical_attention_mean_b200 as dash
from tests._pages_model import Pool
from tests.test_abi import FAKE, tensor

BIG = 1 << 40


def _error():
    return dash.load().dash_attn_last_error().decode()


def _ref(*tensors):
    return [ctypes.byref(t) for t in tensors]


def _fwd(q, k, v, o, window=64, sinks=4, ws=FAKE, ws_bytes=BIG, rest=None):
    return dash.load().dash_attn_window_fwd(*_ref(q, k, v), None, window, sinks, ctypes.byref(o),
                                            rest and ctypes.byref(rest), None, ws, ws_bytes, None)


def _bwd(q, k, v, o, do, dq, dk, dv, window=64, sinks=4, lse=FAKE, ws=FAKE, ws_bytes=BIG, rest=None):
    return dash.load().dash_attn_window_bwd(*_ref(q, k, v, o), rest and ctypes.byref(rest), lse, ctypes.byref(do), None,
                                            window, sinks, *_ref(dq, dk, dv), ws, ws_bytes, None)


def _good():
    return [tensor(1, 256, 8, 128), tensor(1, 256, 2, 128), tensor(1, 256, 2, 128), tensor(1, 256, 8, 128)]


def _good_bwd():
    return _good() + [tensor(1, 256, 8, 128), tensor(1, 256, 8, 128), tensor(1, 256, 2, 128), tensor(1, 256, 2, 128)]


@pytest.mark.parametrize("change, status, text", [
    (lambda a: setattr(a[0], "d", 96), 2, "head dim"),
    (lambda a: setattr(a[1], "dtype", 1), 1, "dtype"),
    (lambda a: setattr(a[2], "dtype", 1), 1, "dtype"),
    (lambda a: setattr(a[3], "dtype", 0), 1, "dtype"),
    (lambda a: setattr(a[1], "h", 3), 1, "multiple"),
    (lambda a: setattr(a[0], "data", FAKE + 2), 1, "aligned"),
    (lambda a: setattr(a[0], "data", 0), 1, "null"),
    (lambda a: setattr(a[1], "stride_s", 260), 1, "16 bytes"),
    (lambda a: setattr(a[1], "stride_s", 0), 2, "stride of 0"),
    (lambda a: setattr(a[3], "stride_h", 0), 2, "stride of 0"),
    (lambda a: setattr(a[2], "stride_h", -128), 1, "negative"),
    (lambda a: setattr(a[1], "s", 255), 1, "shapes differ"),
    (lambda a: setattr(a[2], "s", 255), 1, "shape mismatch"),
    (lambda a: setattr(a[3], "h", 2), 1, "shape mismatch"),
    (lambda a: setattr(a[0], "s", 0), 1, "positive"),
])
def test_window_fwd_and_bwd_refuse(change, status, text):
    args = _good()
    change(args)
    assert _fwd(*args) == status and text in _error()
    args = _good_bwd()
    change(args)
    assert _bwd(*args) == status and text in _error()


def test_window_range_and_workspace():
    lib = dash.load()
    for window, sinks, status, text in ((-1, 0, 1, "window"), (5, -1, 1, "sinks"), (5, 129, 2, "sinks")):
        assert _fwd(*_good(), window, sinks) == status and text in _error()
        assert _bwd(*_good_bwd(), window, sinks) == status and text in _error()
        q, k = _good()[:2]
        assert lib.dash_attn_window_bwd_workspace_size(*_ref(q, k), window, sinks) == 0
    q, k = _good()[:2]
    need = lib.dash_attn_window_fwd_workspace_size(*_ref(q, k))
    assert need > 0 and need % 256 == 0
    assert _fwd(*_good(), ws_bytes=need - 1) == 3
    assert _fwd(*_good(), ws=FAKE + 128) == 1 and "256-byte" in _error()
    assert _fwd(*_good(), ws=None) == 1
    need = lib.dash_attn_window_bwd_workspace_size(*_ref(q, k), 64, 4)
    assert need >= 8 * 256 * 4
    assert _bwd(*_good_bwd(), ws_bytes=need - 1) == 3
    assert _bwd(*_good_bwd(), lse=None) == 1 and "lse" in _error()
    for rest in (tensor(1, 256, 8, 128, dtype=1), tensor(1, 255, 8, 128), tensor(1, 256, 8, 128, data=FAKE + 4)):
        assert _fwd(*_good(), rest=rest) == 1 and "rest" in _error()
        assert _bwd(*_good_bwd(), rest=rest) == 1 and "rest" in _error()
    fp32 = [tensor(1, 256, h, 128, dtype=0) for h in (8, 2, 2, 8, 8, 8, 2, 2)]
    assert _fwd(*fp32[:4], rest=fp32[3]) == 2 and "rest" in _error()
    assert _bwd(*fp32, rest=fp32[3]) == 2 and "rest" in _error()
    for i in (4, 5, 6, 7):
        args = _good_bwd()
        args[i].dtype = 0
        assert _bwd(*args) == 1 and "dtype" in _error()
        args = _good_bwd()
        args[i].s = 200
        assert _bwd(*args) == 1 and "shape" in _error()


def _decode(q, k, v, o, table="dense", window=0, sinks=0, seqlens=FAKE, most=16, ws_bytes=BIG):
    lib = dash.load()
    tail = (seqlens, window, sinks, ctypes.byref(o), None, FAKE, ws_bytes, None)
    if table == "dense":
        return lib.dash_attn_window_decode(*_ref(q, k, v), *tail)
    return lib.dash_attn_window_decode_paged(*_ref(q, k, v), table, most, *tail)


@pytest.mark.parametrize("table", ["dense", FAKE])
def test_window_decode_refuses(table):
    lib = dash.load()

    def good():
        k = (4, 1024, 2, 128) if table == "dense" else (90, 64, 2, 128)
        return [tensor(4, 1, 8, 128), tensor(*k), tensor(*k), tensor(4, 1, 8, 128)]

    for change, status, text in (
        (lambda a: setattr(a[0], "s", 2), 1, ""),
        (lambda a: [setattr(t, "dtype", 0) for t in a], 2, "f16 and bf16"),
        (lambda a: setattr(a[2], "dtype", 1), 1, "dtype"),
        (lambda a: [setattr(t, "dtype", 1) for t in a[1:3]], 1, "dtype"),
        (lambda a: [setattr(t, "h", 3) for t in a[1:3]], 1, "multiple"),
        (lambda a: setattr(a[1], "stride_s", 0), 2, "stride of 0"),
        (lambda a: setattr(a[3], "b", 3), 1, "shape"),
    ):
        args = good()
        change(args)
        assert _decode(*args, table) == status and text in _error()
    assert _decode(*good(), table, window=-1) == 1
    assert _decode(*good(), table, sinks=129) == 2
    assert _decode(*good(), table, seqlens=None) == 1 and "seqlens" in _error()
    need = lib.dash_attn_window_decode_workspace_size(8, 2, 128)
    assert _decode(*good(), table, ws_bytes=need - 1) == 3
    for bad in ((8, 3, 128), (8, 0, 128), (0, 2, 128), (8, 2, 96), (48, 3, 128)):
        assert lib.dash_attn_window_decode_workspace_size(*bad) == 0
    if table == "dense":
        args = good()
        args[1].b = args[2].b = 3
        assert _decode(*args) == 1 and "batch" in _error()
    else:
        args = good()
        args[1].s = args[2].s = 32
        assert _decode(*args, table) == 2 and "page size" in _error()
        assert _decode(*good(), None) == 1 and "block table" in _error()
        assert _decode(*good(), table, most=0) == 1
        assert _decode(*good(), table, most=1 << 28) == 2


def test_pages_refuse():
    lib = dash.load()
    assert lib.dash_attn_pages_workspace_size(4, 8, 100) % 256 == 0
    for bad in ((0, 8, 100), (4, 0, 100), (4, 8, 0), (8193, 8, 100), (4, 1 << 29, 100), (4, 8, (1 << 30) + 1)):
        assert lib.dash_attn_pages_workspace_size(*bad) == 0
    need = lib.dash_attn_pages_workspace_size(4, 8, 100)
    state = [FAKE, 4, 8, FAKE, FAKE, 100]

    def calls(state, block=64, ws=FAKE, room=need):
        tail = (ws, room, None)
        return (
            lambda: lib.dash_attn_pages_fork(*state, FAKE, FAKE, 2, block, *tail),
            lambda: lib.dash_attn_pages_free(*state, FAKE, 2, block, *tail),
            lambda: lib.dash_attn_pages_grow(*state, FAKE, block, FAKE, FAKE, *tail),
            lambda: lib.dash_attn_pages_compact(*state, block, FAKE, FAKE, FAKE, FAKE, FAKE, *tail),
        )

    for at, value, status in ((0, None, 1), (3, None, 1), (4, None, 1), (1, 0, 1), (1, 9000, 2), (2, 0, 1), (5, 0, 1)):
        broken = list(state)
        broken[at] = value
        for call in calls(broken):
            assert call() == status, (at, value)
    for kw, status in ((dict(block=32), 2), (dict(ws=None), 1), (dict(ws=FAKE + 8), 1), (dict(room=need - 1), 3)):
        for call in calls(state, **kw):
            assert call() == status, kw
    tail = (FAKE, need, None)
    assert lib.dash_attn_pages_fork(*state, None, FAKE, 2, 64, *tail) == 1
    assert lib.dash_attn_pages_fork(*state, FAKE, FAKE, 5, 64, *tail) == 1
    assert lib.dash_attn_pages_fork(*state, FAKE, FAKE, -1, 64, *tail) == 1
    assert lib.dash_attn_pages_free(*state, None, 2, 64, *tail) == 1
    assert lib.dash_attn_pages_grow(*state, None, 64, FAKE, FAKE, *tail) == 1
    assert lib.dash_attn_pages_compact(*state, 64, FAKE, FAKE, None, FAKE, FAKE, *tail) == 1


def test_pages_copy_refuses():
    lib = dash.load()

    def call(*pools, n=4, src=FAKE, dst=FAKE):
        return lib.dash_attn_pages_copy((dash.DashTensor * max(1, len(pools)))(*pools), len(pools), src, dst, n, None)

    good = tensor(90, 64, 2, 128)
    assert call() == 1
    assert call(*[good] * 65) == 1
    assert call(good, tensor(90, 64, 4, 128)) == 1 and "page shapes" in _error()
    assert call(good, tensor(90, 64, 2, 128, dtype=1)) == 1
    assert call(good, n=-1) == 1
    assert call(good, src=None) == 1
    bad = tensor(90, 64, 2, 128)
    bad.stride_b = 0
    assert call(bad) == 2
    assert call(tensor(90, 1 << 24, 2, 128)) == 2 and "1 GiB" in _error()
    assert call(good, n=1 << 40) == 2 and "too many" in _error()


def test_binding_refuses_host_tensors_and_wrong_arrays():
    import torch

    x = torch.zeros(1, 64, 1, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: dash.window_fwd(x, x, x), lambda: dash.window_attention(x, x, x),
                 lambda: dash.window_bwd(x, x, x, x, x, x), lambda: dash.window_decode(x, x, x, i[0]),
                 lambda: dash.pages_fork(i, i[0, :1], i[0], i[0], i[0], 64), lambda: dash.pages_copy([x], i[0], i[0]),
                 lambda: dash.pages_grow(i, i[0, :1], i[0], i[0, :1], 64), lambda: dash.pages_copy([], i[0], i[0]),
                 lambda: dash.pages_compact(i, i[0, :1], i[0], 64), lambda: dash.pages_free(i, i[0], i[0], i[0], 64)):
        with pytest.raises(ValueError):
            call()


def test_the_model_keeps_its_counts():
    """The Python model that the GPU tests compare with: pages are counted as the table holds them, and
    compaction leaves none in use at the pool's high end."""
    rng = random.Random(0)
    m = Pool(6, 5, 40, 64)
    for _ in range(400):
        kind = rng.randrange(4)
        if kind == 0:
            m.grow([min(rng.randrange(0, 90), 5 * 64 - s) for s in m.seqlens])
        elif kind == 1:
            n = rng.randrange(1, 6)
            m.fork([rng.randrange(6) for _ in range(n)], rng.sample(range(6), n))
        elif kind == 2:
            m.free(rng.sample(range(6), 2))
        else:
            src, dst, held = m.compact()
            assert len(src) == len(dst) and all(r == 0 for r in m.refs[held:])
        assert m.counted() == m.refs
