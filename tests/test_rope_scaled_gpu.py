"""The scaled 3D rotary embedding and its gradient against the formula in 64
bits.  Bound: the angle rounds to fp32 within [-pi, pi] (pi 2^-24), sine and
cosine by 2 steps, amplitude, products and sum by 2^-24 each: below 1e-6 of
amplitude (|x| + |y|); the result to bf16 by 2^-8."""
import math

import pytest
import torch

from video_diffusion_transformer_non_b200 import binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def randn(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(BF)


def reference(x, grid, bands, freqs, pos_scale, amplitude, interleaved, offset, sign):
    """(y, |x| + |partner| of turned features and 0 of copied ones), fp64."""
    T, Hg, Wg = grid
    S = x.shape[2]
    n = torch.arange(S, device="cuda") - offset
    video = (n >= 0) & (n < T * Hg * Wg)
    coords = [n // (Hg * Wg), (n // Wg) % Hg, n % Wg]
    X = x.double()
    y, mag = X.clone(), torch.zeros_like(X)
    start = at = 0
    for a, d in enumerate(bands):
        for c in range(d // 2):
            f = (start + 2 * c, start + 2 * c + 1) if interleaved else (start + c, start + c + d // 2)
            ang = coords[a].double() * pos_scale[a] * freqs[at + c] * sign
            u, v = X[..., f[0]], X[..., f[1]]
            for i, r in ((0, u * ang.cos() - v * ang.sin()), (1, u * ang.sin() + v * ang.cos())):
                y[..., f[i]] = torch.where(video, amplitude * r, X[..., f[i]])
                mag[..., f[i]] = torch.where(video, abs(amplitude) * (u.abs() + v.abs()), 0.0)
        start, at = start + d, at + d // 2
    return y, mag


def check(got, x, turn, sign=1.0):
    ref, mag = reference(x, turn["grid"], turn["bands"], turn["freqs"],
                         turn.get("pos_scale", (1, 1, 1)), turn.get("amplitude", 1.0),
                         turn.get("interleaved", True), turn.get("token_offset", 0), sign)
    err = (got.double() - ref).abs()
    over = (err - 2.0 ** -8 * ref.abs() - 1e-6 * mag).max().item()
    assert over <= 0, f"{over:.3e} above its bound"
    same = mag == 0
    assert torch.equal(got[same].view(torch.int16), x[same].view(torch.int16)), "not copied"


TURNS = [
    # grid, bands, offset, S behind the video, D
    ((3, 4, 5), (44, 42, 42), 0, 0, 128),
    ((2, 6, 7), (16, 24, 24), 5, 30, 64),
    ((1, 1, 1), (2, 2, 2), 0, 0, 64),           # a single token, most of the head copied
    ((4, 3, 3), (0, 8, 0), 1, 1, 128),          # one band
    ((5, 1, 9), (10, 14, 22), 3, 4, 128),       # bands that end inside a 16-byte piece
    ((2, 2, 40), (0, 0, 0), 0, 3, 64),          # nothing to turn
    ((30, 1, 1), (64, 0, 0), 0, 0, 64),
]


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("grid,bands,offset,tail,D", TURNS)
def test_against_the_formula(grid, bands, offset, tail, D, interleaved):
    S = offset + math.prod(grid) + tail
    q, k = randn(1, 2, 3, S, D), randn(2, 2, 3, S, D)
    turn = dict(grid=grid, bands=bands, freqs=binding.rope3d_frequencies(bands, 100.0, grid, 1.5),
                pos_scale=(0.5, 1.0, 2.0 / 3), amplitude=1.25, interleaved=interleaved,
                token_offset=offset)
    a, b = binding.rope3d_scaled(q, k, **turn)
    check(a, q, turn)
    check(b, k, turn)
    a, b = binding.rope3d_scaled_bwd(q, k, **turn)
    check(a, q, turn, -1.0)
    check(b, k, turn, -1.0)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_equals_rope3d(interleaved, D):
    """Plain frequencies, no scales, whole bands: the bits of vidattn_rope3d."""
    grid, bands = (5, 8, 9), ((44, 42, 42) if D == 128 else (16, 24, 24))
    q, k = randn(1, 2, 5, 380, D), randn(2, 2, 5, 380, D)
    a = binding.rope3d(q, k, grid, bands, interleaved=interleaved, token_offset=7)
    b = binding.rope3d_scaled(q, k, grid, bands, binding.rope3d_frequencies(bands),
                              interleaved=interleaved, token_offset=7)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("interleaved", [True, False])
def test_strides_and_in_place(interleaved):
    """From a fused [B,S,3,H,D] projection into another one, and in place."""
    B, S, H, D = 2, 300, 3, 64
    turn = dict(grid=(5, 6, 9), bands=(12, 16, 16), freqs=binding.rope3d_frequencies((12, 16, 16)),
                amplitude=0.9, interleaved=interleaved)
    qkv = randn(1, B, S, 3, H, D)
    q, k = (qkv[:, :, i].transpose(1, 2) for i in (0, 1))
    a, b = binding.rope3d_scaled(q, k, **turn)
    assert a.is_contiguous()
    check(a, q, turn)
    out = torch.full_like(qkv, 3.0)
    o = [out[:, :, i].transpose(1, 2) for i in (0, 1)]
    binding.rope3d_scaled(q, k, out_q=o[0], out_k=o[1], **turn)
    assert torch.equal(o[0], a) and torch.equal(o[1], b)
    assert bool((out[:, :, 2] == 3.0).all()), "the values beside were written"
    v = qkv[:, :, 2].clone()
    binding.rope3d_scaled(q, k, out_q=q, out_k=k, **turn)
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, :, 2], v)
    only, none = binding.rope3d_scaled(q, **turn)
    assert none is None
    check(only, q, turn)


def test_gradient_is_the_transpose():
    """<R x, g> = <x, R^T g> up to the outputs' roundings."""
    turn = dict(grid=(3, 5, 7), bands=(20, 20, 24), freqs=binding.rope3d_frequencies((20, 20, 24)),
                pos_scale=(0.7, 0.7, 0.7), amplitude=1.3, interleaved=False)
    x, g = randn(1, 1, 4, 110, 64), randn(2, 1, 4, 110, 64)
    y = binding.rope3d_scaled(x, **turn)[0].double()
    d = binding.rope3d_scaled_bwd(g, **turn)[0].double()
    tol = 2.0 ** -8 * ((y * g).abs().sum() + (x * d).abs().sum()) + 1e-5 * x.numel()
    assert abs((y * g.double()).sum() - (x.double() * d).sum()) <= tol


def test_far_positions():
    """Angles of 10^5 and more keep their fraction (fp64)."""
    turn = dict(grid=(2000, 1, 3), bands=(32, 0, 32), freqs=[7.0 * 0.9 ** c for c in range(32)],
                pos_scale=(50.0, 1.0, 1.0))
    x = randn(1, 1, 1, 6000, 64)
    check(binding.rope3d_scaled(x, **turn)[0], x, turn)


@pytest.mark.parametrize("interleaved", [True, False])
def test_infinities_stay_where_they_are(interleaved):
    """Copied features and tokens keep their bits beside an infinity or a NaN."""
    turn = dict(grid=(2, 3, 4), bands=(8, 8, 12), freqs=binding.rope3d_frequencies((8, 8, 12)),
                interleaved=interleaved, token_offset=2)
    x = randn(1, 1, 2, 40, 64)
    x[:, :, 5, 29], x[:, :, 0, 3], x[:, :, 30, 10] = math.inf, math.nan, -math.inf
    y = binding.rope3d_scaled(x, **turn)[0]
    copied = torch.zeros(40, 64, dtype=torch.bool, device="cuda")
    copied[:, 28:] = True
    copied[:2], copied[26:] = True, True
    m = copied.expand(1, 2, 40, 64)
    assert torch.equal(y[m].view(torch.int16), x[m].view(torch.int16))
    assert torch.isfinite(y[~m]).all()


def test_many_heads_few_tokens_and_many_tokens():
    """Shared token tiles (few tokens, many heads) and a persistent walk."""
    bands = (16, 24, 24)
    for B, H, grid in ((2, 40, (1, 3, 5)), (1, 2, (21, 30, 52))):
        turn = dict(grid=grid, bands=bands, freqs=binding.rope3d_frequencies(bands))
        S = math.prod(grid) + 9
        q, k = randn(3, B, H, S, 64), randn(4, B, H, S, 64)
        a, b = binding.rope3d_scaled(q, k, **turn)
        check(a, q, turn)
        check(b, k, turn)


def test_stream_and_graph():
    bands = (16, 24, 24)
    turn = dict(grid=(4, 9, 9), bands=bands, freqs=binding.rope3d_frequencies(bands))
    q, k = randn(3, 1, 4, 330, 64), randn(4, 1, 4, 330, 64)
    ref = binding.rope3d_scaled(q, k, **turn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.rope3d_scaled(q, k, stream=side, **turn)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        rep = binding.rope3d_scaled(q, k, **turn)
    g.replay()
    torch.cuda.synchronize()
    for r, s, t in zip(ref, got, rep):
        assert torch.equal(r, s) and torch.equal(r, t)
