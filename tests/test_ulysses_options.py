"""The options of ulysses_attention's rotation and norm are those of the
differentiable functions: the same dict turns and normalises the same way, and
what one refuses the other does.  CPU tests look at the calls that are made, the
GPU test at their results."""
import pytest
import torch

from video_diffusion_transformer_non_b200 import autograd, binding
from video_diffusion_transformer_non_b200.ulysses import ulysses_attention

GRID, BANDS, PART = (2, 3, 4), (16, 24, 24), (8, 16, 16)
FREQS = [0.9 ** c for c in range(20)]

# options, and whether the scaled rotation is needed
ROPES = [
    (dict(grid=GRID, bands=BANDS), False),
    (dict(grid=GRID, bands=BANDS, theta=300.0, interleaved=False, offset=3), False),
    (dict(grid=GRID, bands=BANDS, theta=300.0, token_offset=3), False),
    (dict(grid=GRID, bands=BANDS, theta=None, freqs=None, amplitude=None, offset=None), False),
    (dict(grid=GRID, bands=BANDS, theta=300.0, pos_scale=(1.0, 0.5, 0.5)), True),
    (dict(grid=GRID, bands=BANDS, amplitude=1.25, token_offset=2), True),
    (dict(grid=GRID, bands=PART, theta=300.0), True),
    (dict(grid=GRID, bands=PART, freqs=FREQS, pos_scale=(0.5, 0.5, 1.0), amplitude=0.5,
          interleaved=False, offset=1), True),
]
WRONG = [dict(grid=GRID, bands=PART, freqs=FREQS, theta=300.0),
         dict(grid=GRID, bands=BANDS, scale=2.0),
         dict(grid=GRID, bands=BANDS, offset=1, token_offset=1),
         dict(bands=BANDS), dict(grid=GRID)]


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(binding, "rope3d_scaled",
                        lambda q, k=None, **kw: seen.append(("scaled", kw)) or (q, k))

    def rope3d(q, k, grid, bands, theta, interleaved, token_offset):
        seen.append(("plain", dict(grid=grid, bands=bands, theta=theta, interleaved=interleaved,
                                   token_offset=token_offset)))
        return q, k

    monkeypatch.setattr(binding, "rope3d", rope3d)
    return seen


def run(rope=None, **kw):
    x = torch.zeros(1, 2, 30, 64)
    return ulysses_attention(x, x, x, rope=rope,
                             attn_fn=lambda q, k, v, *a, **n: (v, v[..., 0]), **kw)


@pytest.mark.parametrize("rope,scaled", ROPES)
def test_rope_options_reach_the_rotation(calls, rope, scaled):
    run(rope)
    (kind, got), = calls
    assert kind == ("scaled" if scaled else "plain")
    want = autograd.rope_arguments(rope)
    if scaled:
        assert got == want
    else:
        assert got == dict(grid=GRID, bands=BANDS, theta=rope.get("theta") or 10000.0,
                           interleaved=want.get("interleaved", True),
                           token_offset=want.get("token_offset", 0))
    if rope.get("offset") or rope.get("token_offset"):
        assert got["token_offset"] == (rope.get("offset") or rope.get("token_offset"))


@pytest.mark.parametrize("rope", WRONG)
def test_wrong_rope_options_are_refused(calls, rope):
    with pytest.raises(ValueError):
        run(rope)
    assert not calls
    with pytest.raises(ValueError):
        autograd.rope_arguments(rope)


def test_a_rotation_of_the_callers_own_takes_any_options():
    seen = []
    run(dict(by=1), rope_fn=lambda q, k, rope: seen.append(rope) or (q, k))
    assert seen == [dict(by=1)]


def test_wrong_norm_options_are_refused(monkeypatch):
    monkeypatch.setattr(binding, "layer_norm", lambda x, w, b, eps: (x, eps, None))
    w = torch.ones(64)
    with pytest.raises(ValueError):
        run(qk_norm=dict(weight=w))
    with pytest.raises(ValueError):
        run(qk_norm=dict(q=(w, None), epsilon=1e-5), norm_fn=lambda x, w, b, eps: x)
    run(qk_norm=dict(q=(w, None), eps=1e-5))
    run(qk_norm=dict(eps=None))


@pytest.mark.gpu
@pytest.mark.parametrize("rope,scaled", ROPES)
def test_the_bits_of_the_training_path(rope, scaled):
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(2, 4, 30, 64, generator=gen, device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(64, generator=gen, device="cuda")
    norm = dict(q=(w, None), eps=1e-5)
    out, lse = ulysses_attention(q, k, v, n_chunks=2, rope=rope, qk_norm=norm)
    o, l = autograd.qkv_attention(q, k, v, norm, rope)
    assert torch.equal(out, o) and torch.equal(lse, l)
