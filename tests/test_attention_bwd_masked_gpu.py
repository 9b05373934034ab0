"""The attention's backward pass where queries see no key: the forward's lse is
-inf there, so the gradient that reaches it is often an infinity or a NaN (0
times -inf, a logaddexp of two such rows); it has no share in anything."""
import math

import pytest
import torch

from test_attention_bwd_gpu import make
from video_diffusion_transformer_non_b200 import autograd, binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S_q,S_kv,ids,causal,n_split", [
    (300, 100, None, True, 0), (450, 300, "any", False, 0), (450, 300, "any", True, 3)])
def test_lse_gradient_of_rows_that_see_nothing(bad, D, S_q, S_kv, ids, causal, n_split):
    """The bits of a call with zeros there."""
    x = make(2, 2, S_q, S_kv, D, 100 + S_q, ids, with_dlse=True)
    seg = x["seg_q"], x["seg_kv"]
    out, lse = binding.attention(x["q"], x["k"], x["v"], *seg, causal=causal)
    empty = lse == -math.inf
    assert bool(empty.any()) and not bool(empty.all())
    grads = []
    for value in (0.0, bad):
        dlse = x["dlse"].masked_fill(empty, value)
        grads.append(binding.attention_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, *seg,
                                           causal=causal, dlse=dlse, n_split=n_split))
    for a, b in zip(*grads):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_losses_of_lse():
    """A masked square of lse, and the merge of two partial results."""
    x = make(1, 2, 300, 100, 64, 7)
    leaves = [x[n].requires_grad_() for n in "qkv"]
    out, lse = autograd.attention(*leaves, causal=True)
    seen = (lse != -math.inf).float()
    torch.nan_to_num(lse.square() * seen, nan=0.0).sum().backward()
    assert all(torch.isfinite(t.grad).all() for t in leaves)
    want = [t.grad.clone() for t in leaves]
    for t in leaves:
        t.grad = None
    out, lse = autograd.attention(*leaves, causal=True)
    lse[seen.bool()].square().sum().backward()
    for t, w in zip(leaves, want):
        assert torch.equal(t.grad, w)
        t.grad = None
    _, a = autograd.attention(*leaves, causal=True)
    _, b = autograd.attention(*leaves, causal=True)
    torch.nan_to_num(torch.logaddexp(a, b), neginf=0.0, nan=0.0).sum().backward()
    assert all(torch.isfinite(t.grad).all() for t in leaves)
