"""The attention's backward pass in 64 bits, from its formula, with a bound on
how far the kernel's arithmetic may be from it, element by element.

The bound counts every rounding of the documented arithmetic at its worst:
  scores and dP      fp32 sums of D products: D 2^-23 sum |a b|
  P                  the exponent's own rounding and 7.5e-5 for the polynomial
  P, dS to bf16      2^-8 each, relative
  gradients          fp32 sums of n terms: n 2^-23 sum |terms|; bf16: 2^-8
`rms` is the same with the roundings of independent terms added as variances
(a rounding is uniform below half a step, so its deviation is the bound over
sqrt(3); no factor is taken off for that)."""
import math

import torch

U = 2.0 ** -23
BF = 2.0 ** -8


def visible(seg_q, seg_kv, S_q, S_kv, causal, device):
    """bool [B or 1, 1, S_q, S_kv]: which keys each query sees."""
    see = torch.ones((1, 1, S_q, S_kv), dtype=torch.bool, device=device)
    if seg_q is not None:
        see = (seg_q[:, :, None] == seg_kv[:, None, :])[:, None]
    if causal:
        i = torch.arange(S_q, device=device)[:, None]
        j = torch.arange(S_kv, device=device)[None]
        see = see & (j <= i + (S_kv - S_q))
    return see


def forward(q, k, v, see, scale):
    """out and lse in 64 bits; rows that see nothing: 0 and -inf."""
    s = (q.double() @ k.double().transpose(2, 3) * scale).masked_fill(~see, -math.inf)
    lse = s.logsumexp(-1)
    p = (s - lse.clamp_min(-1e300)[..., None]).exp()
    return p @ v.double(), lse


def backward(q, k, v, out, dout, lse, dlse, see, scale):
    """name -> (gradient, bound, rms bound) for dq, dk and dv, all fp64."""
    D, S_q, S_kv = q.shape[3], q.shape[2], k.shape[2]
    q, k, v, out, dout, lse = (t.double() for t in (q, k, v, out, dout, lse))
    T = lambda t: t.transpose(2, 3)
    s = q @ T(k)
    lse = lse.clamp_min(-1e300)[..., None]
    p = torch.where(see, (s * scale - lse).exp(), 0.0)
    dp = dout @ T(v)
    delta = (dout * out).sum(-1, keepdim=True)
    if dlse is not None:
        delta = delta - dlse.double()[..., None]
    ds = p * (dp - delta)
    g = dict(dq=scale * ds @ k, dk=scale * T(ds) @ q, dv=T(p) @ dout)

    lse_abs = torch.where(lse > -1e299, lse.abs(), 0.0)
    arg = torch.where(see, (s * scale).abs() + lse_abs, 0.0)
    e_p = abs(scale) * D * U * (q.abs() @ T(k.abs())) + 3 * U * arg + 7.5e-5 + 4 * U
    e_dp = D * U * (dout.abs() @ T(v.abs()))
    e_delta = D * U * (dout * out).abs().sum(-1, keepdim=True) + 3 * U * delta.abs()
    e_ds = p * (e_dp + e_delta) + ds.abs() * (e_p + 4 * U)
    dsa = ds.abs() + e_ds
    r_ds = BF * dsa                                   # rounding of dS to bf16
    r_p = BF * p * (1 + e_p)
    a = abs(scale)
    res = {}
    for name, acc, e, r, other, n, mul in (
            ("dq", dsa, e_ds, r_ds, k, S_kv, a), ("dk", T(dsa), T(e_ds), T(r_ds), q, S_q, a),
            ("dv", T(p), T(p * e_p), T(r_p), dout, S_q, 1.0)):
        x = other.abs()
        sysm = mul * (e @ x + n * U * (acc @ x))
        out_r = BF * g[name].abs()
        bound = sysm + mul * (r @ x) + out_r * 1.01 + 1e-30
        rms = sysm + mul * ((r * r) @ (x * x)).sqrt() + out_r + 1e-30
        res[name] = (g[name], bound, rms)
    return res


def check(got, ref, what=""):
    """got: name -> tensor; ref: backward()'s result."""
    for name, t in got.items():
        exact, bound, rms = ref[name]
        err = (t.double() - exact).abs()
        assert torch.isfinite(t).all(), f"{what} {name}: not finite"
        if err.numel() == 0:
            continue
        over = (err - bound).max().item()
        assert over <= 0, f"{what} {name}: {over:.3e} above its bound, max err {err.max():.3e}"
        # the deviations of all elements together: at most their rms bounds
        lhs, rhs = err.square().sum().sqrt().item(), rms.square().sum().sqrt().item()
        assert lhs <= rhs, f"{what} {name}: rms error {lhs:.3e} > {rhs:.3e}"
