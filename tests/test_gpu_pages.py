"""GPU tests of the cache page operators (dash_attn_pages_*) against a model on Python lists, and of a run of them
together with the attention that reads the pages."""

import random

import pytest
import torch

from tests._pages_model import Pool
from tests.test_gpu_window import _check_decode, _check_forward, _inputs

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _ws(dash, m):
    return torch.full((dash.pages_workspace_size(m.batch, m.most, len(m.refs)),), 255, dtype=torch.uint8,
                      device="cuda")


def _state(m):
    return _dev(m.table), _dev(m.seqlens), _dev(m.refs)


def _same(m, table, seqlens, refs):
    assert seqlens.tolist() == m.seqlens and refs.tolist() == m.refs
    assert table.tolist() == m.table


@pytest.mark.parametrize("batch, most, n_pages, block, steps", [
    (1, 1, 1, 64, 12), (2, 3, 5, 128, 40), (7, 6, 40, 64, 120), (40, 9, 300, 64, 120), (130, 40, 2100, 128, 60),
    (3, 70, 20000, 64, 40), (1500, 33, 9000, 64, 12),
])
def test_random_runs(cuda_lib, batch, most, n_pages, block, steps):
    dash, rng = cuda_lib, random.Random(batch * 1000 + n_pages)
    m = Pool(batch, most, n_pages, block)
    table, seqlens, refs = _state(m)
    ws = _ws(dash, m)
    for step in range(steps):
        kind = rng.choice(["grow", "grow", "grow", "fork", "fork", "free", "compact"])
        if kind == "grow":
            n_new = [rng.choice([0, 0, 1, 2, block - 1, block, rng.randrange(0, 3 * block)]) for _ in range(batch)]
            n_new = [min(n, most * block - s) for n, s in zip(n_new, m.seqlens)]
            want = m.grow(n_new)
            src, dst = dash.pages_grow(table, seqlens, refs, _dev(n_new), block, workspace=ws)
            assert dash.device_status(ws) == (0 if want else 6)
            assert [src.tolist(), dst.tolist()] == (list(want) if want else [[-1] * batch] * 2)
        elif kind == "fork":
            n = rng.randrange(0, batch + 1)
            dst = rng.sample(range(batch), n)
            one = rng.randrange(batch)  # one parent, any parents, or a permutation of the rows
            src = [one] * n if step % 3 == 0 else rng.sample(dst, n) if step % 3 == 1 else \
                [rng.randrange(batch) for _ in range(n)]
            m.fork(src, dst)
            dash.pages_fork(table, seqlens, refs, _dev(src), _dev(dst), block, workspace=ws)
            assert dash.device_status(ws) == 0
        elif kind == "free":
            slots = rng.sample(range(batch), rng.randrange(0, max(2, batch // 3)))
            m.free(slots)
            dash.pages_free(table, seqlens, refs, _dev(slots), block, workspace=ws)
            assert dash.device_status(ws) == 0
        else:
            src, dst, held = m.compact()
            inplace = bool(step % 2)
            before = table.clone(), refs.clone()
            got = dash.pages_compact(table, seqlens, refs, block, inplace=inplace, workspace=ws)
            assert dash.device_status(ws) == 0
            assert got["info"].tolist() == [len(src), held]
            pad = [-1] * (n_pages // 2 - len(src))
            assert got["src"].tolist() == src + pad and got["dst"].tolist() == dst + pad
            if inplace:
                assert got["table"] is table and got["refs"] is refs
            else:
                assert torch.equal(before[0], table) and torch.equal(before[1], refs)
            table, refs = got["table"], got["refs"]
        _same(m, table, seqlens, refs)
        assert m.counted() == m.refs


def test_refusals_leave_the_state(cuda_lib):
    dash = cuda_lib
    m = Pool(4, 3, 6, 64)
    m.grow([100, 64, 0, 1])
    m.fork([0], [2])
    table, seqlens, refs = _state(m)
    ws = _ws(dash, m)

    def refused(code=1):
        assert dash.device_status(ws) == code
        _same(m, table, seqlens, refs)

    for src, dst in (([0], [4]), ([0], [-1]), ([4], [0]), ([-1], [0]), ([0, 1], [3, 3])):
        dash.pages_fork(table, seqlens, refs, _dev(src), _dev(dst), 64, workspace=ws)
        refused()
    for slots in ([4], [-1], [2, 2], [1 << 30]):
        dash.pages_free(table, seqlens, refs, _dev(slots), 64, workspace=ws)
        refused()
    for n_new in ([-1, 0, 0, 0], [0, 0, 0, 3 * 64], [0, 0, 0, (1 << 31) - 1]):
        src, dst = dash.pages_grow(table, seqlens, refs, _dev(n_new), 64, workspace=ws)
        refused()
        assert (src == -1).all() and (dst == -1).all()
    dash.pages_grow(table, seqlens, refs, _dev([92, 0, 0, 64]), 64, workspace=ws)  # a copy, a page and another
    refused(6)
    for bad in (-3, 3 * 64 + 1):
        lens = seqlens.clone()
        lens[1] = bad
        for call in (lambda: dash.pages_fork(table, lens, refs, _dev([1]), _dev([0]), 64, workspace=ws),
                     lambda: dash.pages_free(table, lens, refs, _dev([1]), 64, workspace=ws),
                     lambda: dash.pages_grow(table, lens, refs, _dev([0, 1, 0, 0]), 64, workspace=ws)):
            call()
            refused()
    # the call after a refused one is not affected
    want = m.grow([1, 0, 1, 0])
    src, dst = dash.pages_grow(table, seqlens, refs, _dev([1, 0, 1, 0]), 64, workspace=ws)
    assert [src.tolist(), dst.tolist()] == list(want)
    refused(0)


def test_bad_entries_are_reported_and_bounded(cuda_lib):
    """Entries outside the pool: skipped in the counts, moved as they are, and reported."""
    dash = cuda_lib
    for bad in (-1, 6, 1 << 30):
        table, seqlens, refs = _dev([[bad, 4], [-1, -1]]), _dev([100, 0]), _dev([0, 0, 0, 0, 1, 0])
        ws = torch.empty(dash.pages_workspace_size(2, 2, 6), dtype=torch.uint8, device="cuda")
        got = dash.pages_compact(table, seqlens, refs, 64, workspace=ws)
        assert dash.device_status(ws) == 1
        assert got["table"].tolist() == [[bad, 0], [-1, -1]] and got["refs"].tolist() == [1, 0, 0, 0, 0, 0]
        dash.pages_fork(table, seqlens, refs, _dev([0]), _dev([1]), 64, workspace=ws)
        assert dash.device_status(ws) == 1
        assert refs.tolist() == [0, 0, 0, 0, 2, 0]
        table[0, 1] = bad
        dash.pages_grow(table, seqlens, refs, _dev([1, 0]), 64, workspace=ws)
        assert dash.device_status(ws) == 1
        assert seqlens.tolist() == [100, 100]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["plain", "heads_first", "kv_in_one", "head_slice"])
def test_copy(cuda_lib, dtype, layout):
    dash = cuda_lib
    n, s, h, d = 23, 64, 3, 64
    pools = []
    for i in range(3):
        if layout == "plain":
            pools.append(torch.randn(n + i, s, h, d, device="cuda").to(dtype))
        elif layout == "heads_first":
            pools.append(torch.randn(n + i, h, s, d, device="cuda").to(dtype).transpose(1, 2))
        elif layout == "kv_in_one":
            pools.append(torch.randn(n + i, s, 2, h, d, device="cuda").to(dtype)[:, :, i % 2])
        else:
            pools.append(torch.randn(n + i, s, h + 2, d, device="cuda").to(dtype)[:, :, 1:h + 1])
    rng = torch.Generator().manual_seed(3)
    ids = torch.randperm(n, generator=rng)
    src, dst = ids[:9].to(torch.int32), ids[9:18].to(torch.int32)
    src[2], dst[5] = -1, -4  # skipped
    src[3], dst[7] = n + 2, 1 << 30  # outside every pool: skipped
    want = [p.clone() for p in pools]
    for a, b in zip(src.tolist(), dst.tolist()):
        if 0 <= a < n and 0 <= b < n:
            for w in want:
                w[b] = w[a]
    whole = [p._base.clone() if p._base is not None else None for p in pools]
    dash.pages_copy(pools, src.cuda(), dst.cuda())
    for p, w, base in zip(pools, want, whole):
        assert torch.equal(p, w)
        if base is not None and layout == "head_slice":
            assert torch.equal(p._base[:, :, 0], base[:, :, 0]) and torch.equal(p._base[:, :, -1], base[:, :, -1])
    dash.pages_copy(pools, src[:0].cuda(), dst[:0].cuda())


def test_copy_of_summaries(cuda_lib):
    """The summaries [B, Hkv, t_cap, d] of sparse layers: a pool whose pages are the sequences."""
    dash = cuda_lib
    summ = torch.randn(5, 2, 33, 64, device="cuda")
    want = summ.clone()
    want[4] = want[1]
    dash.pages_copy([summ.transpose(1, 2)], _dev([1]), _dev([4]))
    assert torch.equal(summ, want)


def test_captured(cuda_lib):
    """Fork, grow, copy and free captured into one graph, replayed on another state."""
    dash, block = cuda_lib, 64
    m = Pool(6, 4, 24, block)
    m.grow([100, 30, 0, 0, 0, 0])
    table, seqlens, refs = _state(m)
    pool = torch.randn(24, block, 2, 64, device="cuda")
    src, dst, n_new = _dev([0, 0, 1]), _dev([2, 3, 4]), _dev([0, 0, 1, 70, 3, 0])

    def run():
        dash.pages_fork(table, seqlens, refs, src, dst, block)
        pair = dash.pages_grow(table, seqlens, refs, n_new, block)
        dash.pages_copy([pool], *pair)
        return pair

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pair = run()
    for srcs, dsts in (([0, 0, 1], [2, 3, 4]), ([2, 1, 3], [1, 5, 0])):
        src.copy_(_dev(srcs))
        dst.copy_(_dev(dsts))
        m.fork(srcs, dsts)
        want, contents = m.grow(n_new.tolist()), pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        _same(m, table, seqlens, refs)
        assert [pair[0].tolist(), pair[1].tolist()] == list(want)
        for a, b in zip(*want):
            if a >= 0:
                contents[b] = contents[a]
        assert torch.equal(pool, contents)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_generation(cuda_lib, dtype):
    """A prompt, its cache in pages, branches of it that grow token by token and stay apart, some freed, the pool
    compacted: the attention of every step against the definition on each branch's own tokens."""
    dash, block, window, sinks = cuda_lib, 64, 100, 4
    h, hkv, d, n = 4, 2, 64, 150
    case = (1, n, h, hkv, d, dtype, window, sinks, None)
    q, k, v, _, _ = _inputs(case, 1)
    out, lse = dash.window_fwd(q, k, v, window, sinks, return_lse=True)
    _check_forward(case, q, k, v, out, lse)
    batch, most, n_pages = 5, 5, 17
    table, seqlens, refs = _dev([[-1] * most] * batch), _dev([0] * batch), _dev([0] * n_pages)
    pools = [torch.full((n_pages, block, hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]

    def write(b, at, kk, vv):  # what a model's cache write does
        page = table[b, at // block]
        pools[0][page, at % block], pools[1][page, at % block] = kk, vv

    src, dst = dash.pages_grow(table, seqlens, refs, _dev([0, n, 0, 0, 0]), block)
    dash.pages_copy(pools, src, dst)
    for i in range(n):
        write(1, i, k[0, i], v[0, i])
    text = {1: (k[0], v[0])}
    dash.pages_fork(table, seqlens, refs, _dev([1, 1, 1]), _dev([0, 3, 4]), block)
    text.update({b: text[1] for b in (0, 3, 4)})
    gen = torch.Generator(device="cuda").manual_seed(5)
    for step in range(60):
        if step == 20:  # one branch ends, another forks on
            dash.pages_free(table, seqlens, refs, _dev([1]), block)
            dash.pages_fork(table, seqlens, refs, _dev([3]), _dev([2]), block)
            text[2] = text[3]
            del text[1]
        if step == 40:
            moved = dash.pages_compact(table, seqlens, refs, block, inplace=True)
            dash.pages_copy(pools, moved["src"], moved["dst"])
            held = int(moved["info"][1])
            for p in pools:
                p[held:] = float("nan")
        n_new = _dev([1 if b in text else 0 for b in range(batch)])
        pair = dash.pages_grow(table, seqlens, refs, n_new, block)
        dash.pages_copy(pools, *pair)
        kn, vn = (torch.randn(batch, hkv, d, generator=gen, device="cuda").to(dtype) for _ in range(2))
        qn = torch.randn(batch, 1, h, d, generator=gen, device="cuda").to(dtype)
        for b in text:
            text[b] = tuple(torch.cat([t, x[b][None]]) for t, x in zip(text[b], (kn, vn)))
            write(b, len(text[b][0]) - 1, kn[b], vn[b])
        got, lse = dash.window_decode_paged(qn, *pools, table, seqlens, window, sinks, return_lse=True)
        if step % 7 == 0 or step in (20, 40, 59):
            assert seqlens.tolist() == [len(text[b][0]) if b in text else 0 for b in range(batch)]
            for b in range(batch):
                if b in text:
                    _check_decode((h, hkv, d, dtype, window, sinks, [len(text[b][0])]), qn[b:b + 1], text[b][0][None],
                                  text[b][1][None], got[b:b + 1], lse[b:b + 1])
                else:
                    assert (got[b] == 0).all()
    # the sparse layers read the same pages
    w_s = torch.eye(d, device="cuda")
    full = table.clamp(min=0)
    lens = seqlens.clamp(min=1)
    summ = dash.summarize_paged(pools[0], full, lens, w_s, block)
    sparse = dash.decode_paged(qn, *pools, full, lens, summ, 1.5, block)
    for b in text:
        one = len(text[b][0])
        kc, vc = (t[None].contiguous() for t in text[b])
        s1 = dash.summarize(kc, w_s, block, seqlens=_dev([one]))
        alone = dash.decode(qn[b:b + 1].contiguous(), kc, vc, _dev([one]), s1, 1.5, block)
        assert torch.equal(alone, sparse[b:b + 1])
