"""GPU tests of dense / sliding-window attention at the edges between its work items, rows and number ranges (bounds of
tests/_window_ref.py where nothing else is said)."""

import pytest
import torch

from tests import _window_ref as ref
from tests.test_gpu_window import BF16, F16, _check_backward, _inputs

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
