"""fp64 sliding-window attention written from its definition, with the quantities its error bounds need.

Row i sees key j when j <= i and (window == 0 or j > i - window or j < sinks); rows and keys at or past a sequence's
length are not there.

Rounding model.  u is the unit roundoff of the inputs' type (half a step: bf16 2^-8, f16 2^-11, f32 2^-24).
  logits   fp32 sums of d products: |error| <= (d + 8) 2^-24 M, M = max_j sum_e |q_e k_je| / sqrt(d) (the 8 covers
           the scale and the subtraction of the reference); p and the row sum each move by that relative amount
  exp      2^-20 relative (the special-function unit's 2^x is within 2^-22)
  sums     n visible terms in fp32: n 2^-24 relative to the sum of magnitudes
  P        rounded to the inputs' type as an operand (not on the fp32 path): u relative
  out      rounded once: u |out|
f16 also rounds values below 2^-14 to multiples of 2^-24: half a step of that per value, 2^-25.
"""

import math

import torch

ROUNDOFF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def visible(n, window, sinks, device):
    i, j = torch.arange(n, device=device)[:, None], torch.arange(n, device=device)[None]
    seen = j <= i
    if window:
        seen = seen & ((j > i - window) | (j < sinks))
    return seen


def forward(q, k, v, seen):
    """One head: q [n, d], k, v [m, d] fp64, seen [n, m] -> dict of out, p, lse and the bounds of out and lse."""
    d = q.shape[-1]
    s = (q @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    mags = (q.abs() @ k.abs().T / math.sqrt(d)).masked_fill(~seen, 0)
    return dict(out=p @ v, p=p, lse=lse, out_abs=p @ v.abs(), mag=mags.amax(-1), count=seen.sum(-1).double())


def moved(f, d, dtype):
    """Relative amount by which the fp32 arithmetic may move each p of a row."""
    exp = 2.0 ** -20
    return (2 * (d + 8) * f["mag"] + 2 * f["count"]) * 2.0 ** -24 + exp


def out_bound(f, v, d, dtype):
    u = ROUNDOFF[dtype]
    rel = moved(f, d, dtype) + (0.0 if dtype == torch.float32 else u)
    bound = u * f["out"].abs() + rel[:, None] * f["out_abs"] + 1e-30
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25 * (1 + f["count"][:, None] * v.abs().amax())
    return bound


def lse_bound(f, d, dtype):
    return moved(f, d, dtype) + 2.0 ** -22 * f["lse"].abs()


def backward(q, k, v, out, dout, f):
    """One head: gradients, their magnitude sums and root sums of squares.  dq has D = dout . out from the given out
    (the forward's, with the rest of its rounding or without); for dk and dv D is that of the definition."""
    scale = 1 / math.sqrt(q.shape[-1])
    p = f["p"]
    dp = dout @ v.T
    ds_q = p * (dp - (dout * out).sum(-1, keepdim=True))
    ds = p * (dp - (dout * f["out"]).sum(-1, keepdim=True))
    ads, p2, ds2 = ds.abs(), p * p, ds * ds
    # fp32 sums behind dS: dp and D are sums of d products each
    slack = p * (dout.abs() @ v.abs().T + (dout * out).abs().sum(-1, keepdim=True))
    # f16 operands below 2^-14 lie on multiples of 2^-24: half a step each
    w = (p > 0).double() * 2.0 ** -25
    return dict(dq_sub=w @ k.abs() * scale, dk_sub=w.T @ q.abs() * scale, dv_sub=w.T @ dout.abs(),
                dq=ds_q @ k * scale, dq_abs=ds_q.abs() @ k.abs() * scale, dq_slack=slack @ k.abs() * scale,
                dq_sq=(ds_q * ds_q) @ (k * k) * scale ** 2,
                dk_d=(p * (p * dp.abs()).sum(-1, keepdim=True)).T @ q.abs() * scale,
                dk=ds.T @ q * scale, dk_abs=ads.T @ q.abs() * scale, dk_sq=(ds2.T @ (q * q)) * scale ** 2,
                dk_slack=slack.T @ q.abs() * scale,
                dv=p.T @ dout, dv_abs=p.T @ dout.abs(), dv_sq=p2.T @ (dout * dout), dv_slack=torch.zeros_like(v))


def grad_bound(g, name, rel, dtype, d, few=False):
    """P (for dv) and dS (for dq, dk) are rounded once as operands, unbiased and independent: a standard deviation of
    u / sqrt(3) times the root sum of squares of the terms; 3.5 u of it is six of those.  Where a row sees few keys
    (at most 16), dS for dq is two such values: u^2 of each term.  rel: how far the fp32 arithmetic may move each p (the largest over the rows); it moves the D of
    dk, a sum of p dp, too; dp and D carry (d + 8) 2^-24 of their magnitudes."""
    u = ROUNDOFF[dtype]
    bound = u * g[name].abs() + (rel + 2.0 ** -20) * g[name + "_abs"] + 2 * (d + 8) * 2.0 ** -24 * g[name + "_slack"]
    if name == "dk":
        bound = bound + rel * g["dk_d"]
    if dtype != torch.float32:
        bound = bound + (u * u * g["dq_abs"] if name == "dq" and few else 3.5 * u * g[name + "_sq"].sqrt())
    if dtype == torch.float16:
        bound = bound + g[name + "_sub"] + 2.0 ** -25
    return bound + 1e-7 * float(g[name + "_abs"].max().clamp(min=0)) + 1e-30
