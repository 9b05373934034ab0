"""The layer norm with enough rows that every CTA of every form goes round its
ring of rows (at most 4 turns deep) at least six times: per-row results of all
turns and the sums over rows, against the formulas in 64 bits."""
import pytest
import torch

from test_layernorm_gpu import BF, F32, U, check_bwd, check_fwd, half_step, randn, within
from video_diffusion_transformer_non_b200 import binding

pytestmark = pytest.mark.gpu

TURNS = 6


def rows_for(N):
    """Six turns of as many CTAs as could ever be resident (2048 threads an SM),
    and some rows more; rows a CTA: 256 threads of 8, 16 or 32 lanes a row and
    two rows a thread up to 1024 features, then the CTA's two rows."""
    if N <= 1024:
        lanes = 8 if N <= 64 else 16 if N <= 128 else 32
        per_cta, threads = 256 // lanes * 2, 256
    else:
        per_cta, threads = 2, -(-N // 512) * 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return TURNS * sms * (2048 // threads) * per_cta + 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [31, 63, 64, 127, 128, 255, 256, 384, 511, 512, 513, 1001, 1022, 1023,
                               1024, 1600, 2047, 5118, 5119, 5120, 6143, 6144, 8191, 8192, 12001,
                               16384])
def test_six_turns_of_every_cta(N, dtype):
    rows = rows_for(N)
    x = randn(N, rows, N, dtype=dtype, scale=1.5, shift=0.3)
    dy = randn(N + 3, rows, N, dtype=dtype)
    w, b = randn(N + 1, N, scale=0.2, shift=1.0), randn(N + 2, N, scale=0.2)
    y, mean, rstd = binding.layer_norm(x, w, b)
    dx, dw, db = binding.layer_norm_bwd(dy, x, mean, rstd, w)
    sums = torch.zeros(4, N, dtype=torch.float64, device="cuda")   # dw, db, their magnitudes
    step = max(1, (1 << 25) // N)
    for r in range(0, rows, step):
        at = slice(r, r + step)
        check_fwd(x[at], w, b, 1e-6, y[at], mean[at], rstd[at])
        check_bwd(dy[at], x[at], mean[at], rstd[at], w, dx[at], None, None)
        g = dy[at].double()
        t = g * (x[at].double() - mean[at].double()[:, None]) * rstd[at].double()[:, None]
        sums += torch.stack([t.sum(0), g.sum(0), t.abs().sum(0), g.abs().sum(0)])
    for name, got, ref, mag in (("dweight", dw, sums[0], sums[2]), ("dbias", db, sums[1], sums[3])):
        e = (rows + 68) * U * mag   # as the bound of the sums over rows there
        within(got, ref, e + half_step(got.dtype) * (ref.abs() + e), name)


@pytest.mark.parametrize("N", [63, 1001, 5119])
def test_six_turns_in_place(N):
    """bf16 rows of odd length over themselves: neighbouring rows share words."""
    rows = rows_for(N)
    x, w, b = randn(N, rows, N, dtype=BF), randn(1, N), randn(2, N)
    y, mean, rstd = binding.layer_norm(x, w, b)
    dy = randn(3, rows, N, dtype=BF)
    dx, dw, db = binding.layer_norm_bwd(dy, x, mean, rstd, w)
    out = dy.clone()
    for s, t in zip(binding.layer_norm_bwd(out, x, mean, rstd, w, out=out), (dx, dw, db)):
        assert torch.equal(s, t)
    out = x.clone()
    for s, t in zip(binding.layer_norm_bwd(dy, out, mean, rstd, w, out=out), (dx, dw, db)):
        assert torch.equal(s, t)
    x2 = x.clone()
    binding.layer_norm(x2, w, b, out=x2)
    assert torch.equal(x2, y)
