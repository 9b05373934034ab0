"""The differentiable functions' handling of what autograd hands them: the
kernels' calls are replaced by their formulas behind the binding's own layout
checks, so this runs without a GPU."""
import pytest
import torch

from video_diffusion_transformer_non_b200 import autograd, binding

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def plain(monkeypatch):
    def layer_norm(x, weight=None, bias=None, eps=1e-6):
        binding._rows("x", x)
        m = x.float().mean(-1)
        r = ((x.float() - m[..., None]).square().mean(-1) + eps).rsqrt()
        y = (x.float() - m[..., None]) * r[..., None]
        if weight is not None:
            y = y * weight.float() + (0.0 if bias is None else bias.float())
        return y.to(x.dtype), m, r

    def layer_norm_bwd(dy, x, mean, rstd, weight=None, params=True):
        binding._rows("dy", dy, x.shape)
        xh, g = (x.float() - mean[..., None]) * rstd[..., None], dy.float()
        gw = g if weight is None else g * weight.float()
        dx = (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True)) * \
            rstd[..., None]
        axes = tuple(range(x.dim() - 1))
        if weight is None or not params:
            return dx.to(x.dtype), None, None
        return dx.to(x.dtype), (g * xh).sum(axes).to(weight.dtype), g.sum(axes).to(weight.dtype)

    monkeypatch.setattr(binding, "layer_norm", layer_norm)
    monkeypatch.setattr(binding, "layer_norm_bwd", layer_norm_bwd)


def losses(N):
    """Losses whose gradient reaches the norm with a last dim that is not contiguous."""
    gen = torch.Generator().manual_seed(3)
    a, c = torch.randn(5, generator=gen), torch.randn(4, N, 3, generator=gen)
    return dict(sum=lambda y: y.sum(),
                mean=lambda y: y.mean(),
                matmul=lambda y: (y.transpose(-1, -2) @ a.to(y).reshape(1, 5, 1)).square().sum(),
                conv1d=lambda y: torch.nn.functional.conv1d(y.transpose(-1, -2), c.to(y))
                .square().sum(),
                column=lambda y: y[..., 1].square().sum())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("loss", ["sum", "mean", "matmul", "conv1d", "column"])
def test_layer_norm_takes_any_gradient_layout(plain, loss, dtype):
    """The bits of the call with the same gradient, made contiguous."""
    N = 6
    gen = torch.Generator().manual_seed(1)
    x, w, b = (torch.randn(s, generator=gen).to(dtype).requires_grad_() for s in
               ((2, 5, N), (N,), (N,)))
    y = autograd.layer_norm(x, w, b)
    losses(N)[loss](y).backward()
    at = y.detach().requires_grad_()
    dy, = torch.autograd.grad(losses(N)[loss](at), at)
    _, mean, rstd = binding.layer_norm(x.detach(), w.detach(), b.detach())
    want = binding.layer_norm_bwd(dy.contiguous(), x.detach(), mean, rstd, w.detach())
    for t, g in zip((x, w, b), want):
        assert torch.equal(t.grad, g)


def test_rope_of_one_tensor(monkeypatch):
    """rope3d(q, None) has a gradient as binding.rope3d_scaled(q) has a value."""
    def turn(q, k=None, sign=1.0, **turn):
        return 2.0 * sign * q, None if k is None else 2.0 * sign * k

    monkeypatch.setattr(binding, "rope3d_scaled", turn)
    monkeypatch.setattr(binding, "rope3d_scaled_bwd",
                        lambda dq, dk=None, **kw: turn(dq, dk, -1.0, **kw))
    q = torch.ones(1, 2, 8, 64, requires_grad=True)
    for args in ((q, None), (q,)):
        q.grad = None
        got, none = autograd.rope3d(*args, grid=(1, 2, 4), bands=(8, 8, 8))
        assert none is None
        got.sum().backward()
        assert bool((q.grad == -2.0).all())


def test_rope_options_are_taken_at_the_call(monkeypatch):
    """What the caller changes in its lists between the forward and the backward
    pass does not reach the gradient."""
    seen = []

    def turn(q, k=None, out_q=None, out_k=None, **turn):
        seen.append({n: tuple(v) if n != "interleaved" else v for n, v in turn.items()})
        return 1.0 * q, None

    monkeypatch.setattr(binding, "rope3d_scaled", turn)
    monkeypatch.setattr(binding, "rope3d_scaled_bwd", turn)
    options = dict(grid=[1, 2, 4], bands=[8, 8, 8], freqs=[0.5] * 12, pos_scale=[1.0, 0.5, 1.0])
    q = torch.ones(1, 2, 8, 64, requires_grad=True)
    got, _ = autograd.rope3d(q, **options)
    for v in options.values():
        v[0] = 7
    got.sum().backward()
    assert seen[0] == seen[1] and seen[0]["freqs"] == (0.5,) * 12
    freqs = torch.full((12,), 0.25)
    got, _ = autograd.rope3d(q, grid=(1, 2, 4), bands=(8, 8, 8), freqs=freqs)
    freqs.zero_()
    got.sum().backward()
    assert seen[2] == seen[3] and seen[3]["freqs"] == (0.25,) * 12
