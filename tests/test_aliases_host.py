"""Calls whose outputs lie over an input in another layout, or over the other
tensor: the kernels would read what they have written.  Refused at the C entry
points before anything is enqueued, and so in the binding; no GPU."""
import pytest

from test_norm_rope_host import A, codes, ln, ln_bwd, rope   # noqa: F401

X = (1920, 640, 64)          # [2,3,10,64] contiguous
T = (1920, 64, 192)          # a [2,10,3,64] projection's transpose
B = A + (1 << 16)            # memory of its own


@pytest.mark.parametrize("kw,name", [
    (dict(sx=X, sy=T), "BAD_SHAPE"), (dict(sx=T, sy=X), "BAD_SHAPE"),
    (dict(sx=(0, 640, 64), sy=X), "BAD_SHAPE")])
def test_norm_over_its_input_in_another_layout(codes, kw, name):
    assert ln(x=A, y=A, **kw) == codes[name]


@pytest.mark.parametrize("kw", [
    dict(x=A, dy=B, sx=X, sdy=X, sdx=T), dict(x=B, dy=A, sx=X, sdy=X, sdx=T),
    dict(x=B, dy=A, sx=T, sdy=T, sdx=X), dict(x=A, dy=A, sx=X, sdy=T, sdx=X)])
def test_norm_gradient_over_an_input_in_another_layout(codes, kw):
    assert ln_bwd(dx=A, **kw) == codes["BAD_SHAPE"]


R = (7680, 3840, 64)
RT = (7680, 64, 128)


@pytest.mark.parametrize("kw", [
    dict(q=A, qo=A, si=R, so=RT), dict(k=A, ko=A, q=B, qo=B + (1 << 16), si=RT, so=R),
    dict(q=A, k=B, qo=B, ko=B + (1 << 16)), dict(q=A, k=B, qo=B + (1 << 16), ko=A),
    dict(q=A, k=B, qo=B, ko=A),
    dict(q=A, k=B, qo=B + (1 << 16), ko=B + (1 << 16)),
    dict(q=A, k=A, qo=A, ko=B), dict(q=A, k=A, qo=A, ko=A)])
def test_rope_over_another_tensor(codes, kw):
    """q and k one tensor, rotated in place, among them."""
    assert rope(B=1, **kw) == codes["BAD_SHAPE"]
