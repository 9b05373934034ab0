"""The layer norm and its gradients against their formulas in 64 bits: per head
and per token, odd row lengths, strides, types, in place, rows of one value.

Bounds count fp32 arithmetic at its worst: a row's sums pass at most 64
additions in a row (16 in a thread, the lanes, the warps), so
  |d mean| <= 65 u mean|x|,  |d var| <= d mean^2 + 70 u var  (u = 2^-24)
and what follows from them through the formulas; outputs round by half a step
of their type.  Sums over rows pass at most rows + 64 additions."""
import pytest
import torch

from video_diffusion_transformer_non_b200 import binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half_step(t):
    return torch.finfo(t).eps / 2


def randn(seed, *shape, dtype=F32, scale=1.0, shift=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (err - bound).max().item() if err.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} above its bound (max err {err.max():.3e})"


def check_fwd(x, w, b, eps, y, mean, rstd):
    X = x.double()
    m = X.mean(-1, keepdim=True)
    d = X - m
    var = (d * d).mean(-1, keepdim=True)
    r = (var + eps).rsqrt()
    dm = 65 * U * X.abs().mean(-1, keepdim=True)
    # eps itself is rounded to fp32
    rel = 0.5 * (dm * dm + 70 * U * var + U * eps) / (var + eps) + 5 * U
    xh = d * r
    W = 1.0 if w is None else w.double()
    ref = xh * W + (0.0 if b is None else b.double())
    e = (r * dm * (1 + rel) + xh.abs() * (rel + 3 * U)) * (abs(W) if w is None else W.abs())
    e = e + 2 * U * ((xh * W).abs() + ref.abs())
    within(mean[..., None], m, dm, "mean")
    within(rstd[..., None], r, rel * r, "rstd")
    within(y, ref, e + half_step(x.dtype) * (ref.abs() + e), "y")


def check_bwd(dy, x, mean, rstd, w, dx, dw, db):
    G, X = dy.double(), x.double()
    m, r = mean.double()[..., None], rstd.double()[..., None]
    xh = (X - m) * r
    W = torch.ones((), dtype=torch.float64, device=x.device) if w is None else w.double()
    g = G * W
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    ref = r * (g - c1 - xh * c2)
    e1 = 66 * U * g.abs().mean(-1, keepdim=True)
    e2 = 70 * U * (g * xh).abs().mean(-1, keepdim=True)
    e = r * (e1 + xh.abs() * e2 + 8 * U * (g.abs() + c1.abs() + (xh * c2).abs()))
    within(dx, ref, e + half_step(x.dtype) * (ref.abs() + e), "dx")
    if dw is None:
        return
    axes = tuple(range(x.dim() - 1))
    n = x[..., 0].numel() + 64
    for name, got, terms in (("dweight", dw, G * xh), ("dbias", db, G)):
        ref = terms.sum(axes) if axes else terms
        mag = terms.abs().sum(axes) if axes else terms.abs()
        e = (n + 4) * U * mag
        within(got, ref, e + half_step(got.dtype) * (ref.abs() + e), name)


def both(x, w, b, eps=1e-6, dy=None, seed=7):
    y, mean, rstd = binding.layer_norm(x, w, b, eps)
    assert y.is_contiguous() and y.shape == x.shape and mean.shape == x.shape[:-1]
    dy = randn(seed, *x.shape, dtype=x.dtype) if dy is None else dy
    dx, dw, db = binding.layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    check_fwd(x, w, b, eps, y, mean, rstd)
    check_bwd(dy, x, mean, rstd, w, dx, dw, db)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("N", [1, 2, 7, 8, 63, 64, 65, 96, 128, 200, 256, 257, 504, 512, 1000, 1001,
                               1024, 1032, 2047, 3000, 4104, 5120, 5128, 8192, 8193, 12000, 16384])
@pytest.mark.parametrize("dtype,ptype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_row_lengths(N, dtype, ptype):
    rows = 37 if N > 1024 else 301
    x = randn(N, rows, N, dtype=dtype, scale=1.5, shift=0.3)
    both(x, randn(N + 1, N, dtype=ptype, scale=0.2, shift=1.0),
         randn(N + 2, N, dtype=ptype, scale=0.2))


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 31, 33, 5000])
@pytest.mark.parametrize("N", [64, 128, 1000, 1600])
def test_row_counts(rows, N):
    x = randn(rows, rows, N, dtype=BF)
    both(x, randn(3, N, dtype=BF), randn(4, N, dtype=BF))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1024, 5120, 5121, 6143, 6144, 8184])
def test_wide_rows_over_several_turns(N, dtype):
    """An odd number of rows, more than two turns of every CTA."""
    x = randn(N, 1501, N, dtype=dtype, scale=1.5, shift=0.3)
    both(x, randn(N + 1, N, scale=0.2, shift=1.0), randn(N + 2, N, scale=0.2))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,S,N", [(2, 5, 77, 128), (1, 3, 200, 64), (3, 2, 50, 100),
                                     (2, 2, 9, 2000), (1, 1, 6, 1536)])
def test_strided_rows(dtype, B, H, S, N):
    """x from a fused projection [B,S,3,H,N], dy from a [B,S,H,N] view, results
    into [B,S,H,N]: the same bits as on contiguous copies."""
    qkv = randn(1, B, S, 3, H, N, dtype=dtype)
    x = qkv[:, :, 1].transpose(1, 2)
    w, b = randn(2, N, scale=0.2, shift=1.0), randn(3, N)
    dy = randn(4, B, S, H, N, dtype=dtype).transpose(1, 2)
    y, mean, rstd, dx, dw, db = both(x, w, b, dy=dy)
    buf = torch.full((B, S, H, N + 8), 7.0, dtype=dtype, device="cuda")
    out = buf[..., :N].transpose(1, 2)
    got = binding.layer_norm(x, w, b, out=out)
    assert got[0] is out and torch.equal(out, y)
    grads = binding.layer_norm_bwd(dy, x, mean, rstd, w, out=out)
    assert grads[0] is out and torch.equal(out, dx)
    assert bool((buf[..., N:] == 7.0).all()), "written behind a row"
    plain = binding.layer_norm(x.contiguous(), w, b)
    assert torch.equal(plain[0], y) and torch.equal(plain[1], mean) and torch.equal(plain[2], rstd)
    plain = binding.layer_norm_bwd(dy.contiguous(), x.contiguous(), mean, rstd, w)
    for s, t in zip(plain, (dx, dw, db)):
        assert torch.equal(s, t)


def test_rows_off_16_bytes():
    """Rows on any element: the same values as on aligned rows."""
    wide = randn(1, 40, 137, dtype=BF)
    x = wide[:, 1:129]
    both(x, randn(2, 128), randn(3, 128))


def test_broadcast_input():
    x = randn(1, 1, 128, dtype=BF).expand(50, 128)
    y, mean, *_ = both(x, None, None)
    assert bool((y == y[0]).all()) and bool((mean == mean[0]).all())


@pytest.mark.parametrize("N", [64, 1000, 1600])
def test_in_place(N):
    x, w, b = randn(1, 4, 33, N, dtype=BF), randn(2, N), randn(3, N)
    dy = randn(4, 4, 33, N, dtype=BF)
    y, mean, rstd = binding.layer_norm(x, w, b)
    dx, dw, db = binding.layer_norm_bwd(dy, x, mean, rstd, w)
    dy2 = dy.clone()
    got = binding.layer_norm_bwd(dy2, x, mean, rstd, w, out=dy2)
    for s, t in zip(got, (dx, dw, db)):
        assert torch.equal(s, t)
    x2 = x.clone()
    binding.layer_norm(x2, w, b, out=x2)
    assert torch.equal(x2, y)


def test_without_parameters():
    x = randn(1, 2, 3, 50, 128, dtype=BF)
    *_, dw, db = both(x, None, None)
    assert dw is None and db is None
    y, mean, rstd = binding.layer_norm(x, randn(2, 128), None)
    check_fwd(x, randn(2, 128), None, 1e-6, y, mean, rstd)
    y, mean, rstd = binding.layer_norm(x, None, randn(3, 128))
    check_fwd(x, None, randn(3, 128), 1e-6, y, mean, rstd)
    w = randn(2, 128)
    dx, dw, db = binding.layer_norm_bwd(x, x, mean, rstd, w, params=False)
    assert dw is None and db is None
    check_bwd(x, x, mean, rstd, w, dx, None, None)


def test_far_from_zero_and_constant_rows():
    """Rows whose mean is 1000 times their spread; rows of one value (the
    variance is 0, eps alone is left)."""
    both(randn(1, 64, 512, scale=1.0, shift=1000.0), randn(2, 512), randn(3, 512), eps=1e-5)
    x = randn(4, 16, 1).expand(16, 640).contiguous()
    y, mean, rstd = binding.layer_norm(x, None, None, eps=1e-4)
    check_fwd(x, None, None, 1e-4, y, mean, rstd)


def test_a_bad_row_stays_alone():
    """An infinity or a NaN spoils its own row and the sums over rows only."""
    x = randn(1, 40, 128, dtype=BF)
    x[3, 5], x[17, 0] = float("inf"), float("nan")
    y, mean, rstd = binding.layer_norm(x, None, None)
    ok = torch.ones(40, dtype=torch.bool, device="cuda")
    ok[3] = ok[17] = False
    assert torch.isfinite(y[ok]).all() and not torch.isfinite(y[~ok]).any()
    dx, _, _ = binding.layer_norm_bwd(torch.ones_like(x), x, mean, rstd)
    assert torch.isfinite(dx[ok]).all()


def test_many_rows():
    """More rows than a launch holds at once, sums over 200 000 of them."""
    x = randn(1, 2, 8, 12500, 64, dtype=BF)
    a = both(x, randn(2, 64, dtype=BF), randn(3, 64, dtype=BF))
    b = both(x, randn(2, 64, dtype=BF), randn(3, 64, dtype=BF))
    for s, t in zip(a, b):
        assert torch.equal(s, t), "not the same bits"


def test_no_rows():
    x = torch.empty((0, 64), device="cuda")
    y, mean, rstd = binding.layer_norm(x, randn(1, 64), randn(2, 64))
    assert y.shape == x.shape and mean.shape == (0,)
    dx, dw, db = binding.layer_norm_bwd(x, x, mean, rstd, randn(1, 64))
    assert dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())


def test_stream_and_graph():
    x, w, b = randn(1, 900, 1280, dtype=BF), randn(2, 1280), randn(3, 1280)
    dy = randn(4, 900, 1280, dtype=BF)
    direct = (*binding.layer_norm(x, w, b),)
    direct += binding.layer_norm_bwd(dy, x, direct[1], direct[2], w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.layer_norm(x, w, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = (*binding.layer_norm(x, w, b),)
        got += binding.layer_norm_bwd(dy, x, got[1], got[2], w)
    for t in got:
        t.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    for s, t in zip(got, direct):
        assert torch.equal(s, t)


def test_differences():
    """Central differences of sum(y * dy) in 64 bits along random directions."""
    x, w, b = randn(1, 6, 96), randn(2, 96, shift=1.0), randn(3, 96)
    dy = randn(4, 6, 96)
    _, mean, rstd = binding.layer_norm(x, w, b, 1e-5)
    grads = binding.layer_norm_bwd(dy, x, mean, rstd, w)

    def loss(X, W, Bb):
        m = X.mean(-1, keepdim=True)
        var = ((X - m) ** 2).mean(-1, keepdim=True)
        return ((((X - m) / (var + 1e-5).sqrt()) * W + Bb) * dy.double()).sum()

    at = [t.double() for t in (x, w, b)]
    for i, grad in enumerate(grads):
        u = randn(9 + i, *at[i].shape).double()
        h = 1e-4
        f = [loss(*[t + s * h * u if j == i else t for j, t in enumerate(at)]) for s in (1, -1)]
        slope = ((f[0] - f[1]) / (2 * h)).item()
        # fp32 gradients: each element to about 1e-6 of the largest term
        tol = 1e-5 * (grad.double().abs() * u.abs()).sum().item() + 1e-5 * u.abs().sum().item()
        assert abs((grad.double() * u).sum().item() - slope) <= tol


@pytest.mark.parametrize("N", [1, 2, 3, 31, 63, 64, 127, 128, 255, 511, 513, 1023, 1024, 2047, 5119])
@pytest.mark.parametrize("off,pitch", [(0, 0), (1, 0), (1, 1), (3, 2), (2, 4)])
def test_bf16_rows_on_any_place(N, off, pitch):
    """Rows that start on any 2 bytes, the same or another in every row, of even
    and odd length, into rows of other places; nothing beside them is written."""
    rows = 70
    w, b = randn(2, N, scale=0.2, shift=1.0), randn(3, N, scale=0.2)

    def place(o, seed=None, fill=None):
        buf = randn(seed, rows * (N + pitch) + 16, dtype=BF) if seed else \
            torch.full((rows * (N + pitch) + 16,), fill, dtype=BF, device="cuda")
        return buf, buf[o:].as_strided((rows, N), (N + pitch, 1), buf.storage_offset() + o)

    x, dy = place(off, 1)[1], place(off + 1, 5)[1]
    buf, out = place(off + 2, fill=7.0)
    y, mean, rstd = binding.layer_norm(x, w, b, 1e-3, out=out)
    check_fwd(x, w, b, 1e-3, y, mean, rstd)
    dbuf, dout = place(off + 3, fill=7.0)
    dx, dw, db = binding.layer_norm_bwd(dy, x, mean, rstd, w, out=dout)
    check_bwd(dy, x, mean, rstd, w, dx, dw, db)
    for whole, o in ((buf, off + 2), (dbuf, off + 3)):
        inside = torch.zeros(whole.shape, dtype=torch.bool, device="cuda")
        inside.as_strided((rows, N), (N + pitch, 1), o).fill_(True)
        assert bool((whole[~inside] == 7.0).all()), "written beside a row"
    # in place, from the same places (the order of a row's sums goes by its place)
    whole, here = place(off, 1)
    y, mean, rstd = binding.layer_norm(here, w, b, 1e-3, out=here)
    check_fwd(x, w, b, 1e-3, y, mean, rstd)
