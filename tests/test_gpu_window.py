"""GPU parity of dense / sliding-window attention (dash_attn_window_*) against fp64 written from the definition.

The bounds are those of tests/_window_ref.py.  The backward is given the kernel's forward output, as a user gives it,
and the reference takes the same one.
"""

import math
import threading

import pytest
import torch

from tests import _window_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# batch, seq, heads, kv_heads, dim, dtype, window, sinks, lengths
CASES = {
    "one_token": (1, 1, 2, 1, 64, BF16, 0, 0, None),
    "two_tokens_window1": (1, 2, 8, 1, 128, F16, 1, 0, None),
    "window1_sink1": (1, 300, 4, 4, 64, F16, 1, 1, None),
    "dense_g1": (1, 513, 2, 2, 128, BF16, 0, 0, None),
    "dense_g8_f16": (1, 385, 8, 1, 64, F16, 0, 0, None),
    "window_of_seq": (1, 257, 4, 2, 128, F16, 257, 3, None),
    "window_seq_less_one": (1, 257, 4, 2, 128, F16, 256, 0, None),
    "window127": (1, 700, 4, 1, 128, BF16, 127, 0, None),
    "window128_sink128": (1, 1000, 8, 2, 128, F16, 128, 128, None),
    "window129_sink7": (2, 640, 2, 2, 64, F16, 129, 7, None),
    "sinks_above_seq": (1, 100, 2, 1, 64, BF16, 5, 128, None),
    "tile_edges": (1, 128, 4, 4, 128, F16, 64, 0, None),
    "tile_edge_plus": (1, 129, 1, 1, 128, F16, 64, 64, None),
    "longer": (1, 2500, 4, 2, 64, BF16, 300, 64, None),
    "longer_g8": (1, 1777, 8, 1, 128, F16, 515, 100, None),
    "padded": (4, 333, 4, 2, 64, F16, 100, 5, [0, 1, 333, 200]),
    "padded_dense": (3, 400, 8, 1, 128, BF16, 0, 0, [129, 400, 64]),
    "padded_g1": (3, 520, 2, 2, 128, F16, 60, 16, [300, 128, 513]),
    "f32": (2, 333, 4, 2, 64, F32, 100, 5, [333, 130]),
    "f32_dense": (1, 200, 8, 1, 128, F32, 0, 0, None),
    "f32_window1": (1, 70, 2, 2, 64, F32, 1, 0, None),
}


def _inputs(case, seed=0, scale=1.0):
    b, s, h, hkv, d, dt, window, sinks, lens = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, do = (torch.randn(b, s, h, d, generator=g, device="cuda", dtype=F32).mul(scale).to(dt) for _ in range(2))
    k, v = (torch.randn(b, s, hkv, d, generator=g, device="cuda", dtype=F32).mul(scale).to(dt) for _ in range(2))
    seqlens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    return q, k, v, do, seqlens


def _check(what, got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    excess = (got - want).abs() / bound
    assert excess.max() <= 1, f"{what}: {float(excess.max()):.3g} of its bound"


def _check_forward(case, q, k, v, out, lse):
    b, s, h, hkv, d, dt, window, sinks, lens = case
    refs = {}
    for i in range(b):
        n = s if lens is None else lens[i]
        assert (out[i, n:] == 0).all() and (lse[i, :, n:] == -math.inf).all()
        if n == 0:
            continue
        seen = ref.visible(n, window, sinks, q.device)
        for hh in range(h):
            g = hh // (h // hkv)
            f = ref.forward(q[i, :n, hh].double(), k[i, :n, g].double(), v[i, :n, g].double(), seen)
            _check(f"out {i} {hh}", out[i, :n, hh], f["out"], ref.out_bound(f, v[i, :n, g].double(), d, dt))
            _check(f"lse {i} {hh}", lse[i, hh, :n], f["lse"], ref.lse_bound(f, d, dt))
            refs[i, hh] = f
    return refs


def _check_backward(case, q, k, v, do, out, refs, grads):
    b, s, h, hkv, d, dt, window, sinks, lens = case
    for i in range(b):
        n = s if lens is None else lens[i]
        for name in ("dq", "dk", "dv"):
            assert (grads[name][i, n:] == 0).all(), name
        if n == 0:
            continue
        for g in range(hkv):
            tot, rel = {}, 0.0
            for hh in range(g * (h // hkv), (g + 1) * (h // hkv)):
                f = refs[i, hh]
                one = ref.backward(q[i, :n, hh].double(), k[i, :n, g].double(), v[i, :n, g].double(),
                                   out[i, :n, hh].double(), do[i, :n, hh].double(), f)
                r = float(ref.moved(f, d, dt).max()) * 2  # p comes from the logits and from the log-sum-exp
                rel = max(rel, r)
                few = (window or s) + sinks <= 16
                _check(f"dq {i} {hh}", grads["dq"][i, :n, hh], one["dq"], ref.grad_bound(one, "dq", r, dt, d, few))
                for key, x in one.items():
                    if key[:2] in ("dk", "dv"):
                        tot[key] = tot[key] + x if key in tot else x
            for name in ("dk", "dv"):
                _check(f"{name} {i} {g}", grads[name][i, :n, g], tot[name], ref.grad_bound(tot, name, rel, dt, d))


def _poison(case, *tensors):
    """NaN behind the sequences' ends."""
    if case[-1] is not None:
        for t in tensors:
            for i, n in enumerate(case[-1]):
                t[i, n:] = math.nan


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_backward(cuda_lib, name):
    dash, case = cuda_lib, CASES[name]
    window, sinks = case[6:8]
    q, k, v, do, seqlens = _inputs(case)
    _poison(case, q, k, v, do)
    ws = torch.empty(dash.window_fwd_workspace_size(q, k), dtype=torch.uint8, device="cuda")
    out, lse = dash.window_fwd(q, k, v, window, sinks, seqlens, return_lse=True, workspace=ws)
    assert dash.device_status(ws) == 0
    refs = _check_forward(case, q, k, v, out, lse)
    wsb = torch.empty(dash.window_bwd_workspace_size(q, k, window, sinks), dtype=torch.uint8, device="cuda")
    wsb.fill_(255)  # what an earlier use left there does not matter
    grads = dash.window_bwd(q, k, v, out, lse, do, window, sinks, seqlens, workspace=wsb)
    assert dash.device_status(wsb) == 0
    _check_backward(case, q, k, v, do, out, refs, grads)
    if q.dtype != F32:
        # with what rounding took from out
        rest = torch.full_like(out, math.nan)
        assert torch.equal(dash.window_fwd(q, k, v, window, sinks, seqlens, rest=rest), out)
        assert (rest.double().abs() <= ref.ROUNDOFF[q.dtype] * out.double().abs() + 2.0 ** -24).all()
        better = dash.window_bwd(q, k, v, out, lse, do, window, sinks, seqlens, rest=rest)
        _check_backward(case, q, k, v, do, out.double() + rest.double(), refs, better)
    # one writer per element: the same values again
    again = dash.window_bwd(q, k, v, out, lse, do, window, sinks, seqlens)
    assert all(torch.equal(grads[x], again[x]) for x in grads)
    assert torch.equal(dash.window_fwd(q, k, v, window, sinks, seqlens), out)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window", [2, 3, 8, 100])
def test_gradients_of_few_keys(cuda_lib, window, dtype):
    """Where few keys are visible, D's error matters most.  Three independent roundings (the output's, dS's or P's, and
    what P's left in D) of at most u / sqrt(3) of the gradient's norm each: u together."""
    dash = cuda_lib
    case = (1, 1000, 4, 2, 64, dtype, window, 0, None)
    q, k, v, do, _ = _inputs(case, 13)
    rest = torch.empty_like(q)
    out, lse = dash.window_fwd(q, k, v, window, return_lse=True, rest=rest)
    refs = _check_forward(case, q, k, v, out, lse)
    g = dash.window_bwd(q, k, v, out, lse, do, window, rest=rest)
    err, size = {"dq": 0.0, "dk": 0.0}, {"dq": 0.0, "dk": 0.0}
    for kv in range(2):
        dk = 0.0
        for h in (2 * kv, 2 * kv + 1):
            one = ref.backward(q[0, :, h].double(), k[0, :, kv].double(), v[0, :, kv].double(), refs[0, h]["out"],
                               do[0, :, h].double(), refs[0, h])
            err["dq"] += float((g["dq"][0, :, h].double() - one["dq"]).square().sum())
            size["dq"] += float(one["dq"].square().sum())
            dk = dk + one["dk"]
        err["dk"] += float((g["dk"][0, :, kv].double() - dk).square().sum())
        size["dk"] += float(dk.square().sum())
    for n in err:
        assert math.sqrt(err[n] / size[n]) <= ref.ROUNDOFF[dtype], n


@pytest.mark.parametrize("scale", [0.05, 8.0])
def test_flat_and_peaked_rows(cuda_lib, scale):
    """Nearly uniform rows, and rows whose running maximum keeps growing (logits of a few hundred)."""
    dash = cuda_lib
    case = (1, 700, 4, 2, 64, F16, 333, 9, None)
    q, k, v, do, _ = _inputs(case, 3)
    q, k = (q.float() * scale).half(), k
    ramp = torch.linspace(0.2, 1.5, 700, device="cuda")[None, :, None, None]
    k = (k.float() * ramp).half()
    out, lse = dash.window_fwd(q, k, v, 333, 9, return_lse=True)
    refs = _check_forward(case, q, k, v, out, lse)
    _check_backward(case, q, k, v, do, out, refs, dash.window_bwd(q, k, v, out, lse, do, 333, 9))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("layout", ["packed", "heads_first"])
def test_strides(cuda_lib, dtype, layout):
    dash = cuda_lib
    case = (2, 290, 4, 2, 64, dtype, 70, 6, None)
    q, k, v, do, _ = _inputs(case, 1)
    if layout == "packed":
        qkv = torch.cat([q, k, v], 2)
        q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
        out = torch.full((2, 290, 6, 64), 7.0, dtype=dtype, device="cuda")[:, :, 1:5]
    else:
        q, k, v, do = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, do))
        out = torch.empty(2, 4, 290, 64, dtype=dtype, device="cuda").transpose(1, 2)
    got, lse = dash.window_fwd(q, k, v, 70, 6, out=out, return_lse=True)
    assert got is out
    refs = _check_forward(case, q, k, v, out, lse)
    grads = {n: torch.empty_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    dash.window_bwd(q, k, v, out, lse, do, 70, 6, grads=grads)
    _check_backward(case, q, k, v, do, out, refs, grads)


@pytest.mark.parametrize("dtype", [F32, F16])
def test_autograd(cuda_lib, dtype):
    dash = cuda_lib
    case = (2, 150, 4, 1, 64, dtype, 40, 3, [150, 77])
    q, k, v, do, seqlens = _inputs(case, 2)
    leaves = [t.requires_grad_(True) for t in (q, k, v)]
    out = dash.window_attention(*leaves, window=40, sinks=3, seqlens=seqlens)
    (out.float() * do.float()).sum().backward()
    rest = None if dtype == F32 else torch.empty_like(do)
    plain, lse = dash.window_fwd(q.detach(), k.detach(), v.detach(), 40, 3, seqlens, return_lse=True, rest=rest)
    want = dash.window_bwd(q.detach(), k.detach(), v.detach(), plain, lse, do, 40, 3, seqlens, rest=rest)
    assert torch.equal(out.detach(), plain)
    for t, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(t.grad, want[n])
    # an incoming gradient that does not start at a 16-byte boundary
    odd = torch.cat([do.flatten()[:1], do.flatten()])[1:].view(do.shape)
    assert odd.data_ptr() % 16 != 0
    (gk,) = torch.autograd.grad(dash.window_attention(q, k, v, 40, 3, seqlens), k, odd)
    assert torch.equal(gk, want["dk"])
    # one in another order of dimensions, and one whose rows are 65 elements apart
    turned = do.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.nn.functional.pad(do, (0, 1))[..., :64]
    assert not turned.is_contiguous() and wide.stride(2) == 65
    for d in (turned, wide):
        got = torch.autograd.grad(dash.window_attention(q, k, v, 40, 3, seqlens), (q, k, v), d)
        assert all(torch.equal(a, want[n]) for a, n in zip(got, ("dq", "dk", "dv")))
    # one that is a broadcast view
    total = dash.window_attention(q, k, v, 40, 3, seqlens).sum()
    (gq,) = torch.autograd.grad(total, q)
    ones = dash.window_bwd(q.detach(), k.detach(), v.detach(), plain, lse, torch.ones_like(do), 40, 3, seqlens,
                           rest=rest)["dq"]
    assert torch.equal(gq, ones)


def test_gradients_against_differences(cuda_lib):
    """Central differences of the fp32 forward along random directions.

    The loss sums out times a fixed tensor.  Its differences carry the forward's rounding, about 2^-20 of the sum of
    magnitudes A of the loss over a step of 2 h, and a third-order term, about h^2 of the derivative's scale; with
    h = 2^-6 both stay below 2^-13 A."""
    dash = cuda_lib
    case = (1, 130, 2, 1, 64, F32, 37, 2, None)
    q, k, v, do, _ = _inputs(case, 4, scale=0.5)
    out, lse = dash.window_fwd(q, k, v, 37, 2, return_lse=True)
    grads = dash.window_bwd(q, k, v, out, lse, do, 37, 2)
    g = torch.Generator(device="cuda").manual_seed(9)
    h = 2.0 ** -6
    size = float((out.double().abs() * do.double().abs()).sum())
    for x, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        way = torch.randn(x.shape, generator=g, device="cuda")
        way = way / way.norm() * math.sqrt(130)
        ends = []
        for sign in (1, -1):
            args = {"dq": (q, k, v), "dk": (q, k, v), "dv": (q, k, v)}[name]
            args = tuple(t + sign * h * way if t is x else t for t in args)
            ends.append(float((dash.window_fwd(*args, 37, 2).double() * do.double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        want = float((grads[name].double() * way.double()).sum())
        assert abs(slope - want) <= 2.0 ** -13 * size, (name, slope, want, size)


def test_captured_and_replayed(cuda_lib):
    dash = cuda_lib
    case = (2, 260, 4, 2, 128, BF16, 90, 4, [260, 100])
    q, k, v, do, seqlens = _inputs(case, 5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # first calls outside the capture
        o, l = dash.window_fwd(q, k, v, 90, 4, seqlens, return_lse=True)
        dash.window_bwd(q, k, v, o, l, do, 90, 4, seqlens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = dash.window_fwd(q, k, v, 90, 4, seqlens, return_lse=True)
        grads = dash.window_bwd(q, k, v, out, lse, do, 90, 4, seqlens)
    q2, k2, v2, do2, _ = _inputs(case, 6)
    for a, b in ((q, q2), (k, k2), (v, v2), (do, do2)):
        a.copy_(b)
    seqlens.copy_(torch.tensor([3, 259], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    eager, lse2 = dash.window_fwd(q, k, v, 90, 4, seqlens, return_lse=True)
    assert torch.equal(out, eager) and torch.equal(lse, lse2)
    want = dash.window_bwd(q, k, v, eager, lse2, do, 90, 4, seqlens)
    assert all(torch.equal(grads[n], want[n]) for n in want)


def test_captured_training_step(cuda_lib):
    """Forward and gradients through autograd in one graph, of leaves that no eager graph holds."""
    dash = cuda_lib
    case = (1, 300, 4, 2, 64, F16, 60, 3, None)
    q, k, v, do, _ = _inputs(case, 5)
    leaves = [t.requires_grad_(True) for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(dash.window_attention(*leaves, window=60, sinks=3), leaves, do)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dash.window_attention(*leaves, window=60, sinks=3)
        grads = torch.autograd.grad(out, leaves, do)
    with torch.no_grad():
        for a, b in zip((q, k, v, do), _inputs(case, 6)):
            a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    leaves = [t.detach().requires_grad_(True) for t in leaves]
    eager = dash.window_attention(*leaves, window=60, sinks=3)
    want = torch.autograd.grad(eager, leaves, do)
    assert torch.equal(out, eager) and all(torch.equal(a, b) for a, b in zip(grads, want))


def test_without_gradients(cuda_lib):
    """The differentiable form under no_grad: the forward's bits, nothing kept; transposed inputs keep their layout."""
    dash = cuda_lib
    case = (2, 200, 4, 2, 64, F16, 60, 3, None)
    q, k, v, _, _ = _inputs(case, 9)
    want = dash.window_attention(q.requires_grad_(True), k, v, 60, 3)
    with torch.no_grad():
        out = dash.window_attention(q, k, v, 60, 3)
        t = dash.window_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, 60, 3)
    assert want.requires_grad and not out.requires_grad and torch.equal(out, want)
    assert torch.equal(t, want) and t.transpose(1, 2).is_contiguous()


def test_other_stream(cuda_lib):
    """Buffers that the call makes belong to the stream it runs on, also while another stream is current."""
    dash = cuda_lib
    case = (1, 400, 4, 2, 64, F16, 50, 4, None)
    q, k, v, do, _ = _inputs(case, 7)
    want, lse = dash.window_fwd(q, k, v, 50, 4, return_lse=True)
    wantg = dash.window_bwd(q, k, v, want, lse, do, 50, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [dash.window_fwd(q, k, v, 50, 4, return_lse=True, stream=side) for _ in range(5)]
    grads = dash.window_bwd(q, k, v, *outs[0], do, 50, 4, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(x, lse) for o, x in outs)
    assert all(torch.equal(grads[n], wantg[n]) for n in wantg)


def test_first_cuda_work_of_a_thread(cuda_lib):
    """Every call works in a thread that has done no CUDA work before (as autograd's threads)."""
    dash = cuda_lib
    case = (1, 200, 4, 2, 64, F16, 50, 4, None)
    q, k, v, do, _ = _inputs(case, 7)
    want, lse = dash.window_fwd(q, k, v, 50, 4, return_lse=True)
    wantg = dash.window_bwd(q, k, v, want, lse, do, 50, 4)
    seqlens = torch.tensor([200], dtype=torch.int32, device="cuda")
    q1 = q[:, -1:].contiguous()
    want1 = dash.window_decode(q1, k, v, seqlens, 50, 4)
    out, lse2, out1 = torch.empty_like(want), torch.empty_like(lse), torch.empty_like(want1)
    grads = {n: torch.empty_like(t) for n, t in wantg.items()}
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    calls = [lambda: dash.window_fwd(q, k, v, 50, 4, out=out, lse=lse2, workspace=ws),
             lambda: dash.window_bwd(q, k, v, out, lse2, do, 50, 4, grads=grads, workspace=ws),
             lambda: dash.window_decode(q1, k, v, seqlens, 50, 4, out=out1, workspace=ws)]
    failed = []

    def run(call):
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    for call in calls:
        t = threading.Thread(target=run, args=(call,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert torch.equal(out, want) and torch.equal(lse2, lse) and torch.equal(out1, want1)
    assert all(torch.equal(grads[n], wantg[n]) for n in wantg)


def test_length_out_of_range_is_reported(cuda_lib):
    dash = cuda_lib
    case = (2, 100, 2, 1, 64, F16, 0, 0, [100, 100])
    q, k, v, do, seqlens = _inputs(case)
    want, lse = dash.window_fwd(q, k, v, return_lse=True)
    seqlens.copy_(torch.tensor([-5, 101], dtype=torch.int32))
    ws = torch.empty(dash.window_fwd_workspace_size(q, k), dtype=torch.uint8, device="cuda")
    out = dash.window_fwd(q, k, v, seqlens=seqlens, workspace=ws)
    assert dash.device_status(ws) == 1
    assert (out[0] == 0).all() and torch.equal(out[1], want[1])
    seqlens.fill_(100)
    dash.window_fwd(q, k, v, seqlens=seqlens, workspace=ws)
    assert dash.device_status(ws) == 0


# ------------------------------------------------------------------ one token over a cache

# heads, kv_heads, dim, dtype, window, sinks, lengths
DECODE = {
    "short": (4, 4, 64, F16, 0, 0, [0, 1, 2, 63, 64, 65, 128, 129]),
    "one_long": (8, 1, 128, BF16, 0, 0, [20000]),
    "ragged": (8, 2, 128, F16, 0, 0, [1, 5000, 0, 777, 64, 12345, 0, 3]),
    "window": (16, 4, 64, BF16, 100, 4, [1, 99, 100, 101, 105, 163, 164, 165, 4000]),
    "window1": (4, 1, 128, F16, 1, 0, [1, 64, 65, 1000]),
    "window_sinks128": (8, 8, 128, F16, 64, 128, [64, 128, 191, 192, 193, 256, 3000]),
    "window_g1": (2, 2, 128, BF16, 300, 7, [5000, 301, 308, 10]),
    "sinks_in_band": (4, 2, 64, F16, 130, 100, [140, 230, 231, 300]),
    "pairs": (4, 4, 64, F16, 0, 0, [3000, 0, 1, 777, 64, 2999, 128, 500]),  # 64-wide KV heads two at a time
    "pairs_g8_window": (16, 2, 64, BF16, 500, 70, [(97 * i) % 1500 for i in range(40)]),
    "pairs_odd_heads": (6, 3, 64, F16, 0, 0, [2500, 100, 1900, 2000]),
    "many": (2, 1, 64, F16, 0, 0, [(37 * i) % 300 for i in range(200)]),
}


def _decode_inputs(case, seed=0):
    h, hkv, d, dt, window, sinks, lens = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    most = max(max(lens), 1) + 9
    q = torch.randn(len(lens), 1, h, d, generator=g, device="cuda").to(dt)
    k, v = (torch.randn(len(lens), most, hkv, d, generator=g, device="cuda").to(dt) for _ in range(2))
    for i, n in enumerate(lens):  # nothing that is not visible is used
        j = torch.arange(most, device="cuda")
        hidden = j >= n
        if window:
            hidden |= (j < n - window) & (j >= sinks)
        k[i, hidden] = math.nan
        v[i, hidden] = math.inf
    return q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda")


def _check_decode(case, q, k, v, out, lse):
    h, hkv, d, dt, window, sinks, lens = case
    for i, n in enumerate(lens):
        if n == 0:
            assert (out[i] == 0).all() and (lse[i] == -math.inf).all()
            continue
        j = torch.arange(n, device=q.device)
        if window:
            j = j[(j >= n - window) | (j < sinks)]
        for g in range(hkv):
            hs = slice(g * (h // hkv), (g + 1) * (h // hkv))
            kk, vv = k[i, j, g].double(), v[i, j, g].double()
            f = ref.forward(q[i, 0, hs].double(), kk, vv, torch.ones(h // hkv, len(j), dtype=torch.bool,
                                                                   device=q.device))
            _check(f"out {i} {g}", out[i, 0, hs], f["out"], ref.out_bound(f, vv, d, dt))
            _check(f"lse {i} {g}", lse[i, hs], f["lse"], ref.lse_bound(f, d, dt))


def _paged(k, v, lens, block, seed=0, spare=3):
    """The dense caches as pages in a shuffled pool; entries and pages that hold nothing are out of range / NaN."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-n // block) for n in lens]
    most = max(max(used), 1) + 2
    ids = torch.randperm(sum(used) + spare, generator=g).tolist()
    table = torch.full((len(lens), most), -7, dtype=torch.int32)
    pools = [torch.full((len(ids), block, *t.shape[2:]), math.nan, dtype=t.dtype, device=t.device) for t in (k, v)]
    at = 0
    for i, n in enumerate(used):
        for c in range(n):
            table[i, c] = ids[at]
            rows = min(block, k.shape[1] - c * block)
            for pool, t in zip(pools, (k, v)):
                pool[ids[at], :rows] = t[i, c * block:c * block + rows]
            at += 1
    return (*pools, table.cuda())


@pytest.mark.parametrize("name", list(DECODE))
def test_decode(cuda_lib, name):
    dash, case = cuda_lib, DECODE[name]
    window, sinks, lens = case[4:]
    q, k, v, seqlens = _decode_inputs(case)
    ws = torch.empty(dash.window_decode_workspace_size(case[0], case[1], case[2]), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    out, lse = dash.window_decode(q, k, v, seqlens, window, sinks, return_lse=True, workspace=ws)
    assert dash.device_status(ws) == 0
    _check_decode(case, q, k, v, out, lse)
    assert torch.equal(dash.window_decode(q, k, v, seqlens, window, sinks), out)
    for block in (64, 128):
        kp, vp, table = _paged(k, v, lens, block, block)
        got, lse2 = dash.window_decode_paged(q, kp, vp, table, seqlens, window, sinks, return_lse=True, workspace=ws)
        assert dash.device_status(ws) == 0
        assert torch.equal(got, out) and torch.equal(lse2, lse)  # the same steps in the same order


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_decode_is_the_last_row(cuda_lib, dtype):
    """The one-token form on a prompt's cache against the prompt's last row."""
    dash = cuda_lib
    case = (1, 900, 4, 2, 64, dtype, 333, 20, None)
    q, k, v, _, _ = _inputs(case, 8)
    out, lse = dash.window_fwd(q, k, v, 333, 20, return_lse=True)
    seqlens = torch.tensor([900], dtype=torch.int32, device="cuda")
    got, lse2 = dash.window_decode(q[:, -1:].contiguous(), k, v, seqlens, 333, 20, return_lse=True)
    # both are within their bounds of the same value
    f = [ref.forward(q[0, -1:, h].double(), k[0, :, h // 2].double(), v[0, :, h // 2].double(),
                     ref.visible(900, 333, 20, q.device)[-1:]) for h in range(4)]
    for h in range(4):
        bound = 2 * ref.out_bound(f[h], v[0, :, h // 2].double(), 64, dtype)
        assert ((got[0, 0, h].double() - out[0, -1, h].double()).abs() <= bound[0]).all()
        assert abs(float(lse2[0, h] - lse[0, h, -1])) <= 2 * float(ref.lse_bound(f[h], 64, dtype)[0])


def test_decode_offsets_past_32_bits(cuda_lib):
    """Pages whose elements lie past 2^31 in the pool, and a dense cache with such a stride."""
    dash = cuda_lib
    n_pages, hkv, d, block = 36000, 8, 128, 64  # 2.36e9 elements
    pool = torch.empty(n_pages, block, hkv, d, dtype=F16, device="cuda")
    ids = [35999, 0, 35000, 17]
    pool[ids] = torch.randn(4, block, hkv, d, device="cuda").half()
    q = torch.randn(1, 1, 8, d, device="cuda").half()
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    seqlens = torch.tensor([250], dtype=torch.int32, device="cuda")
    got, lse = dash.window_decode_paged(q, pool, pool, table, seqlens, return_lse=True)
    cache = pool[ids].reshape(1, 4 * block, hkv, d)
    _check_decode((8, 8, d, F16, 0, 0, [250]), q, cache, cache, got, lse)
    far = pool.view(2, n_pages // 2 * block, hkv, d)  # the second sequence starts past 2^30 elements
    far[1, :250] = cache[0, :250]
    far[0, :250] = cache[0, :250]
    lens = torch.tensor([250, 250], dtype=torch.int32, device="cuda")
    both = dash.window_decode(q.expand(2, 1, 8, d).contiguous(), far, far, lens)
    assert torch.equal(both[0], both[1]) and torch.equal(both[:1], got)


def test_more_pages_than_sequences_may_be(cuda_lib):
    """Pools of more than 65535 pages."""
    dash = cuda_lib
    n_pages = 70000
    pool = torch.zeros(n_pages, 64, 1, 64, dtype=F16, device="cuda")
    ids = [69999, 66000, 5]
    pool[ids] = torch.randn(3, 64, 1, 64, device="cuda").half()
    dash.pages_copy([pool], torch.tensor([69999, 5], dtype=torch.int32, device="cuda"),
                    torch.tensor([7, 69998], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[7], pool[69999]) and torch.equal(pool[69998], pool[5])
    q = torch.randn(1, 1, 2, 64, device="cuda").half()
    table = torch.tensor([[69999, 66000, 69998]], dtype=torch.int32, device="cuda")
    seqlens = torch.tensor([190], dtype=torch.int32, device="cuda")
    got, lse = dash.window_decode_paged(q, pool, pool, table, seqlens, return_lse=True)
    cache = pool[ids].reshape(1, 192, 1, 64)
    _check_decode((2, 1, 64, F16, 0, 0, [190]), q, cache, cache, got, lse)


def test_calls_on_two_streams_at_once(cuda_lib):
    """Calls that overlap, each with its own buffers, give what they give alone."""
    dash = cuda_lib
    case = (1, 3000, 8, 2, 128, BF16, 500, 20, None)
    one, two = _inputs(case, 11), _inputs(case, 12)
    dec = _decode_inputs(DECODE["pairs"], 5)

    def work(x, stream):
        q, k, v, do, _ = x
        out, lse = dash.window_fwd(q, k, v, 500, 20, return_lse=True, stream=stream)
        g = dash.window_bwd(q, k, v, out, lse, do, 500, 20, stream=stream)
        return [out, lse, g["dq"], g["dk"], g["dv"], dash.window_decode(*dec, stream=stream)]

    want = [work(x, None) for x in (one, two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[work(x, s) for x, s in zip((one, two), streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for round_ in got:
        for a, b in zip(round_, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_decode_captured_with_growing_lengths(cuda_lib):
    """One captured call serves every length: the work is split on the device.  Two graphs have their own scratch."""
    dash = cuda_lib
    case = (8, 2, 64, F16, 200, 8, [1200, 700, 3])
    q, k, v, seqlens = _decode_inputs((*case[:4], 0, 0, [1200] * 3), 4)
    dash.window_decode(q, k, v, seqlens, 200, 8)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for window in (200, 0):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(dash.window_decode(q, k, v, seqlens, window, 8, return_lse=True))
        graphs.append(graph)
    for lens in ([1200, 700, 3], [0, 64, 1199], [1, 0, 0], [0, 0, 0], [1200, 1200, 1200]):
        seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for window, (out, lse) in zip((200, 0), outs):
            _check_decode((*case[:4], window, 8, lens), q, k, v, out, lse)


def test_decode_strides_and_output_views(cuda_lib):
    dash = cuda_lib
    case = (4, 2, 128, BF16, 50, 4, [400, 90])
    q, k, v, seqlens = _decode_inputs(case, 2)
    want, lse = dash.window_decode(q, k, v, seqlens, 50, 4, return_lse=True)
    kv = torch.stack([k, v], 3)  # [B, S, Hkv, 2, d]
    heads_first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v)]
    wide = torch.full((2, 1, 9, 128), 3.0, dtype=BF16, device="cuda")
    for kk, vv in ((kv[:, :, :, 0], kv[:, :, :, 1]), heads_first):
        out = wide[:, :, 2:6]
        got = dash.window_decode(q, kk, vv, seqlens, 50, 4, out=out)
        assert torch.equal(got, want)
    assert (wide[:, :, :2] == 3).all() and (wide[:, :, 6:] == 3).all()


def test_decode_reports_bad_pages_and_lengths(cuda_lib):
    """A page outside the pool is read as zeros (never outside it) and reported; lengths are clamped and reported."""
    dash = cuda_lib
    case = (2, 1, 64, F16, 0, 0, [200, 60])
    q, k, v, seqlens = _decode_inputs(case, 3)
    kp, vp, table = _paged(k, v, case[-1], 64)
    ws = torch.empty(dash.window_decode_workspace_size(2, 1, 64), dtype=torch.uint8, device="cuda")
    want = dash.window_decode_paged(q, kp, vp, table, seqlens, workspace=ws)
    for bad in (-1, kp.shape[0], 1 << 30):
        broken = table.clone()
        broken[0, 1] = bad
        got = dash.window_decode_paged(q, kp, vp, broken, seqlens, workspace=ws)
        assert dash.device_status(ws) == 1
        assert torch.isfinite(got).all() and torch.equal(got[1], want[1])
    for bad in (-1, table.shape[1] * 64 + 1):
        dash.window_decode_paged(q, kp, vp, table, seqlens, workspace=ws)
        assert dash.device_status(ws) == 0
        lens = seqlens.clone()
        lens[0] = bad
        full = table.clone()
        full[full < 0] = 0
        got = dash.window_decode_paged(q, kp, vp, full, lens, workspace=ws)
        assert dash.device_status(ws) == 1
        assert torch.equal(got[1], want[1])
