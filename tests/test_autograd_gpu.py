"""The differentiable functions: each the same bits as the calls it is made of,
and the whole path (norm, rotary embedding, attention; forward and backward)
against torch's autograd over the plain formulas in 64 bits.

The path rounds to bf16 about ten times between its inputs and a gradient (norm,
rotation, P, out, dP's operands, dS, dq, rotation, norm, twice where products
meet), each by at most 2^-8 relative and none amplified beyond about 1 at these
scales (logits of deviation 1), so gradients lie within 10 x 2^-8 = 0.04 of the
exact ones in the Frobenius norm."""
import math

import pytest
import torch

import _bwd_ref as ref
from video_diffusion_transformer_non_b200 import autograd, binding
from video_diffusion_transformer_non_b200.ulysses import ulysses_attention

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TOL = 10 * 2.0 ** -8


def randn(seed, *shape, dtype=BF, scale=1.0, shift=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)


def leaf(t):
    return t.detach().requires_grad_()


def norm64(x, w, b, eps):
    m = x.mean(-1, keepdim=True)
    y = (x - m) / ((x - m).square().mean(-1, keepdim=True) + eps).sqrt()
    return y if w is None else y * w + (0.0 if b is None else b)


def rope64(x, turn):
    T, Hg, Wg = turn["grid"]
    off, amp = turn.get("token_offset", 0), turn.get("amplitude", 1.0)
    scale = turn.get("pos_scale", (1.0,) * 3)
    n = torch.arange(x.shape[2], device="cuda") - off
    video = (n >= 0) & (n < T * Hg * Wg)
    coords = [n // (Hg * Wg), (n // Wg) % Hg, n % Wg]
    y, start, at = x.clone(), 0, 0
    for a, d in enumerate(turn["bands"]):
        for c in range(d // 2):
            f = (start + 2 * c, start + 2 * c + 1) if turn.get("interleaved", True) \
                else (start + c, start + c + d // 2)
            ang = torch.where(video, coords[a].double() * scale[a] * turn["freqs"][at + c], 0.0)
            g = torch.where(video, amp, 1.0)
            u, v = x[..., f[0]], x[..., f[1]]
            y = y.index_copy(3, torch.tensor(f, device="cuda"), torch.stack(
                [g * (u * ang.cos() - v * ang.sin()), g * (u * ang.sin() + v * ang.cos())], -1))
        start, at = start + d, at + d // 2
    return y


def path64(q, k, v, params, eps, turn, see, scale):
    wq, bq, wk, bk = params
    qn, kn = norm64(q, wq, bq, eps), norm64(k, wk, bk, eps)
    if turn is not None:
        qn, kn = rope64(qn, turn), rope64(kn, turn)
    s = (qn @ kn.transpose(2, 3) * scale).masked_fill(~see, -math.inf)
    lse = s.logsumexp(-1)
    return (s - lse[..., None]).exp() @ v, lse


@pytest.mark.parametrize("D,interleaved,causal,with_ids", [
    (64, True, False, True), (128, False, True, False), (128, True, False, True)])
def test_path_against_64_bits(D, interleaved, causal, with_ids):
    B, H, S = 2, 3, 330
    turn = dict(grid=(4, 8, 9), bands=(8, 16, 20), token_offset=3, amplitude=1.1,
                freqs=binding.rope3d_frequencies((8, 16, 20), 200.0, (2, 4, 4), 2.0),
                pos_scale=(1.0, 0.5, 1.0), interleaved=interleaved)
    qkv = randn(1, B, S, 3, H, D, scale=1.5, shift=0.2)     # the projection's output
    p = [randn(2, D, dtype=torch.float32, scale=0.1, shift=1.0),
         randn(3, D, dtype=torch.float32, scale=0.1),
         randn(4, D, dtype=BF, scale=0.1, shift=1.0), randn(5, D, dtype=BF, scale=0.1)]
    seg = None
    if with_ids:
        seg = (torch.arange(S, device="cuda") // 110).int().expand(B, S).contiguous()
    see = ref.visible(seg, seg, S, S, causal, "cuda")
    dout, dlse = randn(6, B, H, S, D), randn(7, B, H, S, dtype=torch.float32)
    scale = D ** -0.5

    mine = leaf(qkv)
    params = [leaf(t) for t in p]
    q, k, v = (mine[:, :, i].transpose(1, 2) for i in range(3))
    out, lse = autograd.qkv_attention(
        q, k, v, dict(q=params[:2], k=params[2:], eps=1e-5), turn, seg, seg, causal=causal)
    torch.autograd.backward((out, lse), (dout, dlse))

    exact = leaf(qkv.double())
    eparams = [leaf(t.double()) for t in p]
    eo, el = path64(*(exact[:, :, i].transpose(1, 2) for i in range(3)), eparams, 1e-5, turn, see,
                    scale)
    torch.autograd.backward((eo, el), (dout.double(), dlse.double()))

    for name, a, b in [("out", out, eo), ("lse", lse, el), ("dqkv", mine.grad, exact.grad)] + \
            [(f"param {i}", s.grad, t.grad) for i, (s, t) in enumerate(zip(params, eparams))]:
        assert a.dtype == (torch.float32 if name == "lse" else a.dtype) and torch.isfinite(a).all()
        rel = ((a.double() - b).norm() / b.norm()).item()
        assert rel <= TOL, (name, rel)
    assert [t.grad.dtype for t in params] == [t.dtype for t in p]


def test_path_is_its_calls():
    """qkv_attention gives the bits of the separate differentiable functions,
    and of the binding's calls."""
    B, H, S, D = 1, 4, 200, 64
    turn = dict(grid=(4, 5, 9), bands=(16, 24, 24), freqs=binding.rope3d_frequencies((16, 24, 24)))
    x = [leaf(randn(i, B, S, H, D).transpose(1, 2)) for i in range(3)]
    w = [leaf(randn(10 + i, D, scale=0.1, shift=1.0 - i % 2)) for i in range(4)]
    dout = randn(20, B, H, S, D)
    out, _ = autograd.qkv_attention(*x, dict(q=w[:2], k=w[2:]), turn)
    out.backward(dout)
    got = [t.grad for t in x + w]
    for t in x + w:
        t.grad = None
    q, k = autograd.layer_norm(x[0], *w[:2]), autograd.layer_norm(x[1], *w[2:])
    q, k = autograd.rope3d(q, k, **turn)
    o2, _ = autograd.attention(q, k, x[2].contiguous())
    o2.backward(dout)
    assert torch.equal(out, o2)
    for a, t in zip(got, x + w):
        assert torch.equal(a, t.grad)

    with torch.no_grad():
        qn, mq, rq = binding.layer_norm(x[0], *w[:2])
        kn, mk, rk = binding.layer_norm(x[1], *w[2:])
        qr, kr = binding.rope3d_scaled(qn, kn, **turn)
        v = x[2].contiguous()
        o3, lse = binding.attention(qr, kr, v)
        assert torch.equal(out, o3)
        dq, dk, dv = binding.attention_bwd(dout, qr, kr, v, o3, lse)
        dq, dk = binding.rope3d_scaled_bwd(dq, dk, **turn)
        gq = binding.layer_norm_bwd(dq, x[0], mq, rq, w[0])
        gk = binding.layer_norm_bwd(dk, x[1], mk, rk, w[2])
        for a, b in zip(got, (gq[0], gk[0], dv, gq[1], gq[2], gk[1], gk[2])):
            assert torch.equal(a, b)


def test_parts_of_the_path():
    """Without a norm, without parameters, without a rope; gradients only where
    they are asked for; through lse alone."""
    B, H, S, D = 1, 2, 150, 64
    turn = dict(grid=(2, 8, 9), bands=(16, 24, 24), theta=500.0)
    q, k, v = (leaf(randn(i, B, H, S, D)) for i in range(3))
    out, lse = autograd.qkv_attention(q, k, v, rope=turn)
    lse.sum().backward()
    assert bool((v.grad == 0).all()) and bool((q.grad != 0).any())
    for t in (q, k, v):
        t.grad = None
    out, lse = autograd.qkv_attention(q, k, v, qk_norm={})
    out.float().sum().backward()
    qn, kn = binding.layer_norm(q)[0], binding.layer_norm(k)[0]
    assert torch.equal(out, binding.attention(qn, kn, v)[0])
    w = leaf(randn(9, D, shift=1.0))
    x = randn(10, 30, D)
    autograd.layer_norm(x, w).float().sum().backward()
    assert w.grad is not None and w.grad.dtype == BF
    x = leaf(x)
    autograd.layer_norm(x, w.detach()).float().sum().backward()
    assert x.grad.shape == x.shape
    with pytest.raises(ValueError):
        autograd.layer_norm(x, None, w)
    with pytest.raises(ValueError):
        autograd.qkv_attention(q, k, v, rope=dict(turn, freqs=[1.0] * 32))
    with pytest.raises(ValueError):
        autograd.qkv_attention(q, k, v, qk_norm=dict(weight=w))
    out, _ = autograd.attention(q, k, v)
    g, = torch.autograd.grad(out.float().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):   # first derivatives only
        torch.autograd.grad(g.float().sum(), q)


def test_rows_that_see_nothing():
    """Causal with more queries than keys: the first rows give 0 and pass on
    nothing."""
    q, k, v = leaf(randn(1, 1, 2, 300, 64)), leaf(randn(2, 1, 2, 100, 64)), leaf(randn(3, 1, 2, 100, 64))
    out, lse = autograd.attention(q, k, v, causal=True)
    assert bool((out[:, :, :200] == 0).all()) and bool((lse[:, :, :200] == -math.inf).all())
    out.backward(randn(4, 1, 2, 300, 64))
    assert bool((q.grad[:, :, :200] == 0).all())
    for t in (q, k, v):
        assert torch.isfinite(t.grad).all()


def test_shared_inputs():
    """One tensor as q, k and v; keys and values shared by all heads (expanded):
    the gradients of every use are summed."""
    B, H, S, D = 1, 4, 130, 64
    x = leaf(randn(1, B, H, S, D))
    dout = randn(2, B, H, S, D)
    out, lse = autograd.attention(x, x, x)
    out.backward(dout)
    dq, dk, dv = binding.attention_bwd(dout, x.detach(), x.detach(), x.detach(), out.detach(),
                                       lse.detach())
    exact = dq.double() + dk.double() + dv.double()
    bound = 2.0 ** -8 * 2 * (dq.double().abs() + dk.double().abs() + dv.double().abs())
    assert bool(((x.grad.double() - exact).abs() <= bound).all())
    k1 = leaf(randn(3, B, 1, S, D))
    q = randn(4, B, H, S, D)
    kk = k1.expand(B, H, S, D)
    out, lse = autograd.qkv_attention(q, kk, kk, qk_norm={})
    out.backward(dout)
    assert k1.grad.shape == k1.shape and torch.isfinite(k1.grad).all()


def test_training_step_in_a_graph():
    """Forward and backward of the path captured together, replayed on new data."""
    B, H, S, D = 1, 2, 260, 64
    turn = dict(grid=(5, 6, 8), bands=(16, 24, 24))
    data = [randn(i, B, S, 3, H, D) for i in range(3)]
    dout = randn(9, B, H, S, D)
    w = [randn(20 + i, D, scale=0.1, shift=1.0 - i % 2) for i in range(4)]

    def step(x):
        x = leaf(x)
        p = [leaf(t) for t in w]
        q, k, v = (x[:, :, i].transpose(1, 2) for i in range(3))
        out, _ = autograd.qkv_attention(q, k, v, dict(q=p[:2], k=p[2:]), turn, causal=True)
        return (out, *torch.autograd.grad(out, [x] + p, dout))

    buf = data[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step(buf)
    for x in data[1:]:
        buf.copy_(x)
        g.replay()
        want = step(x)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_ulysses_one_rank():
    """qk_norm and the scaled rotation through the sequence-parallel entry (one
    rank, no process group): the bits of the direct calls; inputs unchanged."""
    B, H, S, D = 2, 4, 190, 64
    turn = dict(grid=(4, 5, 9), bands=(8, 16, 16), freqs=binding.rope3d_frequencies((8, 16, 16)),
                amplitude=1.2, interleaved=False)
    q, k, v = (randn(i, B, H, S, D) for i in range(3))
    q0, k0 = q.clone(), k.clone()
    w = randn(5, D, shift=1.0)
    out, lse = ulysses_attention(q, k, v, n_chunks=2, qk_norm=dict(q=(w, None), eps=1e-5),
                                 rope=dict(turn, offset=4))
    qn, kn = binding.layer_norm(q, w, None, 1e-5)[0], binding.layer_norm(k, eps=1e-5)[0]
    qr, kr = binding.rope3d_scaled(qn, kn, token_offset=4, **turn)
    o, l = binding.attention(qr, kr, v)
    assert torch.equal(out, o) and torch.equal(lse, l)
    assert torch.equal(q, q0) and torch.equal(k, k0)
