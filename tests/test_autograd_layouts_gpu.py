"""The differentiable functions under losses whose gradients arrive in layouts
other than the outputs': the bits of the binding's calls on contiguous ones."""
import pytest
import torch

from video_diffusion_transformer_non_b200 import autograd, binding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def randn(seed, *shape, dtype=BF):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


LOSSES = dict(sum=lambda y, a, c: y.sum(),
              matmul=lambda y, a, c: (y.transpose(-1, -2) @ a).square().sum(),
              conv1d=lambda y, a, c: torch.nn.functional.conv1d(y.transpose(-1, -2), c)
              .square().sum(),
              transposed=lambda y, a, c: y.transpose(-1, -2).contiguous().square().sum())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("loss", list(LOSSES))
def test_layer_norm_takes_any_gradient_layout(loss, dtype):
    N = 200
    f = LOSSES[loss]
    a, c = randn(1, 2, 33, 1, dtype=dtype), randn(2, 4, N, 3, dtype=dtype)
    x, w, b = (randn(3 + i, *s, dtype=dtype).requires_grad_()
               for i, s in enumerate(((2, 33, N), (N,), (N,))))
    y = autograd.layer_norm(x, w, b)
    at = y.detach().requires_grad_()
    dy, = torch.autograd.grad(f(at, a, c), at)
    y.backward(dy)   # the layout as it comes, the values of one evaluation
    _, mean, rstd = binding.layer_norm(x.detach(), w.detach(), b.detach())
    want = binding.layer_norm_bwd(dy.contiguous(), x.detach(), mean, rstd, w.detach())
    for t, g in zip((x, w, b), want):
        assert torch.equal(t.grad, g)
    x.grad = None
    f(autograd.layer_norm(x, w, b), a, c).backward()
    assert torch.isfinite(x.grad).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_of_one_tensor(interleaved):
    turn = dict(grid=(2, 4, 5), bands=(8, 16, 24), amplitude=1.1, interleaved=interleaved)
    q, dq = randn(1, 2, 3, 50, 64).requires_grad_(), randn(2, 2, 3, 50, 64)
    got, none = autograd.rope3d(q, None, **turn)
    assert none is None
    got.backward(dq)
    args = autograd.rope_arguments(turn)
    assert torch.equal(got, binding.rope3d_scaled(q.detach(), **args)[0])
    assert torch.equal(q.grad, binding.rope3d_scaled_bwd(dq, **args)[0])
    q.grad = None
    autograd.rope3d(q, **turn)[0].sum().backward()   # the gradient comes expanded
    assert torch.equal(q.grad, binding.rope3d_scaled_bwd(torch.ones_like(dq), **args)[0])
