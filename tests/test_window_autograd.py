"""The differentiable form of sliding-window attention around its kernels, which a stand-in replaces (no GPU)."""

import pytest
import torch
from torch.autograd import forward_ad

import sparse_hierarchical_attention_mean_b200 as dash


@pytest.fixture
def asked(monkeypatch):
    """What the forward kernel was asked for, call by call."""
    calls = []

    def window_fwd(q, k, v, window=0, sinks=0, seqlens=None, out=None, return_lse=False, lse=None, rest=None,
                   workspace=None, stream=None):
        calls.append(dict(lse=return_lse, rest=rest is not None))
        return (q.clone(), q.new_zeros(q.shape[:3])) if return_lse else q.clone()

    monkeypatch.setattr(dash, "window_fwd", window_fwd)
    return calls


def _qkv(dtype=torch.float16):
    return torch.randn(1, 8, 2, 64).to(dtype), torch.randn(1, 8, 1, 64).to(dtype), torch.randn(1, 8, 1, 64).to(dtype)


@pytest.mark.parametrize("grad_mode", [True, False])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_tangent_is_never_dropped(asked, grad_mode, which):
    """Forward-mode derivatives are not offered: a dual tensor is refused, with gradients on or off."""
    args = list(_qkv())
    with forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            dash.window_attention(*args, 4)


def test_nothing_is_kept_when_no_input_asks_for_a_gradient(asked):
    """The log-sum-exp and what rounding took are made for a backward only."""
    q, k, v = _qkv()
    out = dash.window_attention(q, k, v, 4)
    assert not out.requires_grad and asked[-1] == dict(lse=False, rest=False)
    with torch.no_grad():
        dash.window_attention(q.requires_grad_(True), k, v, 4)
    assert asked[-1] == dict(lse=False, rest=False)
    for i in range(3):
        args = list(_qkv())
        args[i].requires_grad_(True)
        assert dash.window_attention(*args, 4).requires_grad
        assert asked[-1] == dict(lse=True, rest=True)
    args = [t.requires_grad_(True) for t in _qkv(torch.float32)]
    dash.window_attention(*args, 4)
    assert asked[-1] == dict(lse=True, rest=False)
