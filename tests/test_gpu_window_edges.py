"""GPU tests of dense / sliding-window attention at the edges between its work items, rows and number ranges (bounds of
tests/_window_ref.py where nothing else is said)."""

import math

import pytest
import torch

from tests import _window_ref as ref
from tests.test_gpu_window import BF16, F16, _check, _check_backward, _decode_inputs, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name, case", [
    ("one tile of rows", (48, 128, 8, 8, 64, F16, 0, 0, None)),
    ("one tile of rows, d 128", (40, 120, 8, 8, 128, BF16, 0, 0, None)),
    ("window inside a key tile", (1, 2100, 16, 2, 64, F16, 64, 0, None)),
    ("window inside a key tile, few keys", (4, 1024, 8, 1, 128, BF16, 8, 0, None)),
])
def test_items_of_one_step(cuda_lib, name, case):
    """Row tiles whose keys are one step, several of them per SM: each row's D for dk is corrected by its own sum of
    dS.  `out` is given with an error as large as itself, which that sum takes away again, so the sum of another row
    would show."""
    dash = cuda_lib
    b, s, h, hkv, d, dt, window, sinks, _ = case
    q, k, v, do, _ = _inputs(case, 21)
    out, lse = dash.window_fwd(q, k, v, window, sinks, return_lse=True)
    wrong = out + torch.randn(out.shape, generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(dt)
    grads = dash.window_bwd(q, k, v, wrong, lse, do, window, sinks)
    seen, refs = ref.visible(s, window, sinks, q.device), {}
    for i in range(b):
        for hh in range(h):
            g = hh // (h // hkv)
            refs[i, hh] = ref.forward(q[i, :, hh].double(), k[i, :, g].double(), v[i, :, g].double(), seen)
    _check_backward(case, q, k, v, do, wrong, refs, grads)
    for _ in range(10):
        again = dash.window_bwd(q, k, v, wrong, lse, do, window, sinks)
        assert all(torch.equal(grads[n], again[n]) for n in grads)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads, kv_heads, dim, window, sinks, lens", [
    (16, 2, 64, 0, 0, [1, 2, 3, 5, 17, 100]),
    (32, 8, 128, 0, 0, [2, 3, 70, 4000]),
    (16, 16, 64, 0, 0, [2, 9, 700, 3000]),
    (32, 4, 128, 200, 10, [150, 1000, 6000]),
])
def test_decode_is_rounded_once(cuda_lib, heads, kv_heads, dim, window, sinks, lens, dtype):
    """One token: the output's own rounding and the fp32 arithmetic are all of its error.  P goes into the product as
    two values of the cache's type, u^2 of each p apart (f16: multiples of 2^-24, so at most 2^-25)."""
    dash = cuda_lib
    q, k, v, seqlens = _decode_inputs((heads, kv_heads, dim, dtype, window, sinks, lens), 31)
    out = dash.window_decode(q, k, v, seqlens, window, sinks)
    u, group = ref.ROUNDOFF[dtype], heads // kv_heads
    for i, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        if window:
            j = j[(j >= n - window) | (j < sinks)]
        for g in range(kv_heads):
            hs = slice(g * group, (g + 1) * group)
            kk, vv = k[i, j, g].double(), v[i, j, g].double()
            f = ref.forward(q[i, 0, hs].double(), kk, vv, torch.ones(group, len(j), dtype=torch.bool, device="cuda"))
            bound = u * f["out"].abs() + (ref.moved(f, dim, dtype) + u * u)[:, None] * f["out_abs"]
            if dtype == F16:
                bound = bound + 2.0 ** -25 * (1 + len(j) * vv.abs().amax())
            _check(f"out {i} {g}", out[i, 0, hs], f["out"], bound)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads, kv_heads, dim", [(8, 1, 128), (4, 4, 64), (6, 3, 64)])
def test_decode_of_growing_logits(cuda_lib, heads, kv_heads, dim, dtype):
    """One token whose logits grow along the cache by hundreds, so that the reference moves again and again and takes
    both parts of the sum with it: the bound of one rounding."""
    dash = cuda_lib
    lens = [900, 333, 3000]
    q, k, v, seqlens = _decode_inputs((heads, kv_heads, dim, dtype, 0, 0, lens), 32)
    ramp = torch.linspace(0.1, 3.0, k.shape[1], device="cuda")[None, :, None, None]
    q, k = (q.float() * 6).to(dtype), (k.float() * ramp).to(dtype)
    out, lse = dash.window_decode(q, k, v, seqlens, return_lse=True)
    u, group = ref.ROUNDOFF[dtype], heads // kv_heads
    for i, n in enumerate(lens):
        for g in range(kv_heads):
            hs = slice(g * group, (g + 1) * group)
            kk, vv = k[i, :n, g].double(), v[i, :n, g].double()
            f = ref.forward(q[i, 0, hs].double(), kk, vv, torch.ones(group, n, dtype=torch.bool, device="cuda"))
            bound = u * f["out"].abs() + (ref.moved(f, dim, dtype) + u * u)[:, None] * f["out_abs"]
            if dtype == F16:
                bound = bound + 2.0 ** -25 * (1 + n * vv.abs().amax())
            _check(f"out {i} {g}", out[i, 0, hs], f["out"], bound)
            _check(f"lse {i} {g}", lse[i, hs], f["lse"], ref.lse_bound(f, dim, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads, kv_heads, dim", [(4, 1, 64), (8, 1, 128), (2, 2, 64)])
def test_what_stands_behind_the_end_moves_no_bit(cuda_lib, heads, kv_heads, dim, dtype):
    """Rows behind a sequence's end share warps with the last rows before it.  Logits that grow along the sequence make
    rows change their reference on the way, which must not depend on them."""
    dash = cuda_lib
    case = (3, 700, heads, kv_heads, dim, dtype, 500, 20, [699, 333, 401])
    q, k, v, do, seqlens = _inputs(case, 23)
    ramp = torch.linspace(0.2, 2.0, 700, device="cuda")[None, :, None, None]
    q, k = (q.float() * 2).to(dtype), (k.float() * ramp).to(dtype)
    runs = []
    for fill in (0.0, math.nan, 1e4, -math.inf):
        for t in (q, k, v, do):
            for i, n in enumerate(case[-1]):
                t[i, n:] = fill
        rest = torch.empty_like(q)
        out, lse = dash.window_fwd(q, k, v, 500, 20, seqlens, return_lse=True, rest=rest)
        runs.append([out, lse, rest, *dash.window_bwd(q, k, v, out, lse, do, 500, 20, seqlens, rest=rest).values()])
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(run, runs[0]))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_heads_move_no_bit_of_each_other(cuda_lib, dtype):
    """Heads of a group share tiles; one with far larger logits leaves the others' bits as they are."""
    dash = cuda_lib
    case = (1, 900, 4, 1, 64, dtype, 600, 9, None)
    q, k, v, _, _ = _inputs(case, 24)
    ramp = torch.linspace(0.2, 2.0, 900, device="cuda")[None, :, None, None]
    q, k = (q.float() * 2).to(dtype), (k.float() * ramp).to(dtype)
    want, lse = dash.window_fwd(q, k, v, 600, 9, return_lse=True)
    loud = q.clone()
    loud[:, :, 2] *= 16
    out, lse2 = dash.window_fwd(loud, k, v, 600, 9, return_lse=True)
    for h in (0, 1, 3):
        assert torch.equal(out[:, :, h], want[:, :, h]) and torch.equal(lse2[:, h], lse[:, h])


F16_RANGES = {
    # batch, seq, heads, kv_heads, dim, window, and the size of each sequence's incoming gradient
    "small": (1, 2048, 4, 2, 64, 0, [2.0 ** -10]),
    "large": (1, 600, 4, 1, 128, 4, [6200.0]),  # dS beyond 65504, the gradients below it
    "large, window": (1, 600, 2, 2, 64, 40, [2.0 ** 13]),
    "one small beside one large": (2, 700, 4, 2, 64, 0, [2.0 ** 8, 2.0 ** -8]),
    "zero beside ones": (2, 300, 2, 1, 64, 0, [0.0, 1.0]),
}


@pytest.mark.parametrize("name", list(F16_RANGES))
def test_gradients_over_the_range_of_f16(cuda_lib, name):
    """dS as an f16 operand neither overflows nor loses its low bits where the gradients themselves can be held.

    dS is scaled by a power of two c, 2^15 / (2 m) >= c > 2^13 / (2 m) with m the product of the largest norms of a
    row of dout and of v, and lies on multiples of 2^-24: half a step is 2^-25 / c < 2^-37 m.  P is scaled by 2^10."""
    dash = cuda_lib
    b, s, h, hkv, d, window, sizes = F16_RANGES[name]
    case = (b, s, h, hkv, d, F16, window, 0, None)
    q, k, v, do, _ = _inputs(case, 25)
    do = (do.float() * torch.tensor(sizes, device="cuda")[:, None, None, None]).half()
    rest = torch.empty_like(q)
    out, lse = dash.window_fwd(q, k, v, window, return_lse=True, rest=rest)
    grads = dash.window_bwd(q, k, v, out, lse, do, window, rest=rest)
    seen, group = ref.visible(s, window, 0, q.device), h // hkv
    for i in range(b):
        for g in range(hkv):
            kk, vv, tot, rel = k[i, :, g].double(), v[i, :, g].double(), {}, 0.0
            heads = range(g * group, (g + 1) * group)
            m = float(max(do[i, :, x].double().norm(dim=-1).max() for x in heads) * vv.norm(dim=-1).max())
            for hh in heads:
                f = ref.forward(q[i, :, hh].double(), kk, vv, seen)
                exact_out = out[i, :, hh].double() + rest[i, :, hh].double()
                one = ref.backward(q[i, :, hh].double(), kk, vv, exact_out, do[i, :, hh].double(), f)
                for x in ("dq_sub", "dk_sub"):
                    one[x] = one[x] * 2.0 ** -12 * m  # the reference's are those of half a step of 2^-25
                one["dv_sub"] = one["dv_sub"] * 2.0 ** -10
                r = float(ref.moved(f, d, F16).max()) * 2
                rel = max(rel, r)
                _check(f"dq {i} {hh}", grads["dq"][i, :, hh], one["dq"],
                       ref.grad_bound(one, "dq", r, F16, d, 0 < window <= 16))
                for key, x in one.items():
                    if key[:2] in ("dk", "dv"):
                        tot[key] = tot[key] + x if key in tot else x
            for n in ("dk", "dv"):
                _check(f"{n} {i} {g}", grads[n][i, :, g], tot[n], ref.grad_bound(tot, n, rel, F16, d))


def test_sequences_of_a_batch_stay_apart(cuda_lib):
    """A sequence's gradients are the same bits whatever the others of its batch hold."""
    dash = cuda_lib
    case = (3, 400, 4, 2, 64, F16, 100, 4, None)
    q, k, v, do, _ = _inputs(case, 26)
    out, lse = dash.window_fwd(q, k, v, 100, 4, return_lse=True)
    want = dash.window_bwd(q, k, v, out, lse, do, 100, 4)
    do[0] *= 2.0 ** 9
    do[2] = 0
    got = dash.window_bwd(q, k, v, out, lse, do, 100, 4)
    assert all(torch.equal(got[n][1], want[n][1]) for n in want)
    assert all((got[n][2] == 0).all() for n in got)


def test_f16_scales_follow_a_replay(cuda_lib):
    """The scale of dS belongs to the values that a captured backward meets when it is replayed, on whatever stream."""
    dash = cuda_lib
    case = (2, 500, 4, 2, 64, F16, 90, 4, [500, 123])
    q, k, v, do, seqlens = _inputs(case, 27)
    out, lse = dash.window_fwd(q, k, v, 90, 4, seqlens, return_lse=True)
    dash.window_bwd(q, k, v, out, lse, do, 90, 4, seqlens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = dash.window_bwd(q, k, v, out, lse, do, 90, 4, seqlens)
    first = do.clone()
    side = torch.cuda.Stream()
    for size in (2.0 ** -9, 2.0 ** 10, 1.0):
        do.copy_(first * size)
        want = dash.window_bwd(q, k, v, out, lse, do, 90, 4, seqlens)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        other = dash.window_bwd(q, k, v, out, lse, do, 90, 4, seqlens)  # beside the replay, in its own workspace
        torch.cuda.synchronize()
        assert all(torch.equal(grads[n], want[n]) and torch.equal(other[n], want[n]) for n in want)
