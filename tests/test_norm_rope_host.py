"""Refusals of the layer norm and the scaled rotary embedding, at the C entry
points and in the binding, and host logic: no GPU."""
import ctypes
import math
import re

import pytest

from video_diffusion_transformer_non_b200 import binding

A = 1 << 20   # an aligned address that is never read


@pytest.fixture(scope="module")
def codes():
    with open(binding._HEADER) as f:
        return {n: int(v) for n, v in re.findall(r"VIDATTN_(?:ERR_)?(\w+) = (\d+)", f.read())}


def arr(v, t=ctypes.c_int64):
    return None if v is None else (t * len(v))(*v)


def ln(x=A, w=A, b=A, y=A, mean=A, rstd=A, B=2, H=3, S=10, N=64, sx=(1920, 640, 64),
       sy=(1920, 640, 64), xt=0, pt=1, eps=1e-6):
    return binding.load_library().vidattn_layernorm(x, w, b, y, mean, rstd, B, H, S, N, arr(sx),
                                                    arr(sy), xt, pt, eps, None)


def ln_bwd(dy=A, x=A, mean=A, rstd=A, w=A, dx=A, dw=A, db=A, B=2, H=3, S=10, N=64,
           sdy=(1920, 640, 64), sx=(1920, 640, 64), sdx=(1920, 640, 64), xt=0, pt=1, ws=A,
           n=1 << 30):
    return binding.load_library().vidattn_layernorm_bwd(
        dy, x, mean, rstd, w, dx, dw, db, B, H, S, N, arr(sdy), arr(sx), arr(sdx), xt, pt, ws, n,
        None)


SIZES = [(dict(B=0), "BAD_SHAPE"), (dict(H=0), "BAD_SHAPE"), (dict(S=-1), "BAD_SHAPE"),
         (dict(N=0), "BAD_SHAPE"), (dict(N=16385), "BAD_SHAPE"), (dict(xt=2), "BAD_SHAPE"),
         (dict(pt=-1), "BAD_SHAPE"), (dict(B=1 << 16, H=1 << 16), "BAD_SHAPE"),
         (dict(B=1 << 15, H=1 << 15, S=2), "BAD_SHAPE"), (dict(x=None), "NULL"),
         (dict(sx=None), "NULL"), (dict(x=A + 1), "MISALIGNED"), (dict(x=A + 2, xt=1), "MISALIGNED"),
         (dict(w=A + 2), "MISALIGNED"), (dict(mean=A + 2), "MISALIGNED"),
         (dict(rstd=A + 1), "MISALIGNED"), (dict(sx=(-1920, 640, 64)), "BAD_SHAPE")]


@pytest.mark.parametrize("kw,name", SIZES + [
    (dict(y=None), "NULL"), (dict(sy=None), "NULL"), (dict(b=A + 2), "MISALIGNED"),
    (dict(eps=-1.0), "BAD_SHAPE"), (dict(eps=math.nan), "BAD_SHAPE"),
    (dict(eps=math.inf), "BAD_SHAPE"),
    (dict(sy=(0, 640, 64)), "BAD_SHAPE"), (dict(sy=(1920, 640, 63)), "BAD_SHAPE"),
    (dict(sy=(1920, 64, 64)), "BAD_SHAPE"), (dict(sy=(1920, 640, -64)), "BAD_SHAPE")])
def test_norm_refusals(codes, kw, name):
    assert ln(**kw) == codes[name]


@pytest.mark.parametrize("kw,name", SIZES + [
    (dict(dy=None), "NULL"), (dict(dx=None), "NULL"), (dict(mean=None), "NULL"),
    (dict(rstd=None), "NULL"), (dict(ws=None), "NULL"), (dict(sdy=None), "NULL"),
    (dict(sdx=None), "NULL"), (dict(ws=A + 64), "MISALIGNED"), (dict(dw=A + 2), "MISALIGNED"),
    (dict(db=A + 1), "MISALIGNED"), (dict(dy=A + 1), "MISALIGNED"),
    (dict(sdx=(0, 640, 64)), "BAD_SHAPE"), (dict(sdy=(1920, -1, 64)), "BAD_SHAPE"),
    (dict(n=0), "SCRATCH_LIMIT"), (dict(n=255), "SCRATCH_LIMIT")])
def test_norm_gradient_refusals(codes, kw, name):
    assert ln_bwd(**kw) == codes[name]


def test_norm_of_no_rows_is_ok(codes):
    assert ln(S=0, x=None, y=None) == codes["OK"]
    assert ln_bwd(S=0, dw=None, db=None, ws=None, n=0) == codes["OK"]


def test_norm_workspace():
    """[CTAs][2][N] fp32: at most one CTA for every rows a CTA takes at once,
    at most 148 SMs x 2048 threads."""
    ws = binding.layernorm_bwd_workspace
    assert ws(1, 1, 1, 64, 0) == 512
    assert ws(1, 1, 10 ** 6, 128, 0) == 148 * 8 * 2 * 128 * 4
    assert ws(1, 1, 1000, 5120, 1) == 148 * (2048 // 320) * 2 * 5120 * 4
    assert ws(1, 1, 0, 64, 0) == 0
    assert ws(0, 1, 1, 64, 0) == -1 and ws(1, 1, 1, 64, 5) == -1 and ws(1, 1, 1, 20000, 0) == -1


def rope(q=A, k=A, qo=A, ko=A, B=1, H=2, S=60, D=64, si=(7680, 3840, 64), so=(7680, 3840, 64),
         T=3, Hg=4, Wg=5, off=0, bands=(16, 24, 24), freqs=None, pos=(1.0, 1.0, 1.0), amp=1.0,
         flags=0):
    freqs = [0.5] * 64 if freqs is None else freqs
    return binding.load_library().vidattn_rope3d_scaled(
        q, k, qo, ko, B, H, S, D, arr(si), arr(so), T, Hg, Wg, off, *bands,
        arr(freqs, ctypes.c_double) if freqs else None, arr(pos, ctypes.c_double), amp, flags, None)


@pytest.mark.parametrize("kw,name", [
    (dict(q=None), "NULL"), (dict(qo=None), "NULL"), (dict(k=None), "NULL"),
    (dict(ko=None), "NULL"), (dict(si=None), "NULL"), (dict(so=None), "NULL"),
    (dict(freqs=[]), "NULL"), (dict(pos=None), "NULL"),
    (dict(D=96), "UNSUPPORTED_D"), (dict(flags=4), "BAD_SHAPE"),
    (dict(B=0), "BAD_SHAPE"), (dict(S=0), "BAD_SHAPE"), (dict(T=0), "BAD_SHAPE"),
    (dict(off=1), "BAD_SHAPE"), (dict(off=-1), "BAD_SHAPE"),
    (dict(T=1 << 30, Hg=1 << 30, Wg=1 << 30), "BAD_SHAPE"),
    (dict(bands=(16, 24, 26)), "BAD_SHAPE"), (dict(bands=(15, 24, 24)), "BAD_SHAPE"),
    (dict(bands=(-2, 24, 24)), "BAD_SHAPE"),
    (dict(freqs=[math.nan] * 32), "BAD_SHAPE"), (dict(freqs=[1e300] * 32), "BAD_SHAPE"),
    (dict(pos=(math.inf, 1.0, 1.0)), "BAD_SHAPE"), (dict(amp=math.nan), "BAD_SHAPE"),
    (dict(amp=1e300), "BAD_SHAPE"), (dict(freqs=[2.0 ** 30] * 32), "BAD_SHAPE"),
    (dict(q=A + 8), "MISALIGNED"), (dict(ko=A + 2), "MISALIGNED"),
    (dict(si=(7680, 3840, 68)), "MISALIGNED"), (dict(so=(7680, 3844, 64)), "MISALIGNED"),
    (dict(si=(7680, 3840, -64)), "BAD_SHAPE"), (dict(so=(7680, 3840, 0)), "BAD_SHAPE"),
    (dict(so=(7680, 64, 64)), "BAD_SHAPE")])
def test_rope_refusals(codes, kw, name):
    assert rope(**kw) == codes[name]


def test_frequencies():
    """Plain ones; by parts: slow pairs divided by the factor, fast ones kept."""
    f = binding.rope3d_frequencies((4, 0, 6), 100.0)
    assert f == pytest.approx([1.0, 0.1, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)])
    g = binding.rope3d_frequencies((4, 0, 6), 100.0, extent=(63, 1, 6), factor=2.0)
    assert g[0] == 1.0                                      # 10 turns over the trained 63
    assert g[2] == 0.5                                      # less than one over 6
    turns = 63 * 0.1 / (2 * math.pi)                        # 1.003: a little is kept
    keep = (turns - 1) / 7
    assert g[1] == pytest.approx(0.1 * keep + 0.05 * (1 - keep))
    with pytest.raises(ValueError):
        binding.rope3d_frequencies((3, 0, 0))
    with pytest.raises(ValueError):
        binding.rope3d_frequencies((4, 0, 0), factor=0.0)


@pytest.fixture
def host(monkeypatch):
    import torch
    monkeypatch.setattr(binding, "_DEVICE_TYPE", "cpu")

    def never(*a, **k):
        raise AssertionError("a refused call reached the library")

    monkeypatch.setattr(binding, "load_library", never)
    return torch


@pytest.mark.parametrize("case", ["dtype", "ndim", "feature_stride", "weight_shape", "weight_dtype",
                                  "bias_dtype", "not_tensor", "weight_list"])
def test_layer_norm_checks(host, case):
    torch = host
    x, w, b = torch.zeros(4, 64), torch.zeros(64), torch.zeros(64)
    if case == "dtype":
        x = x.half()
    elif case == "ndim":
        x = torch.zeros(1, 1, 1, 4, 64)
    elif case == "feature_stride":
        x = torch.zeros(64, 4).t()
    elif case == "weight_shape":
        w = torch.zeros(65)
    elif case == "weight_dtype":
        w = b = w.double()
    elif case == "bias_dtype":
        b = b.bfloat16()
    elif case == "not_tensor":
        x = [1.0]
    elif case == "weight_list":
        w = [1.0] * 64
    with pytest.raises(ValueError):
        binding.layer_norm(x, w, b)


@pytest.mark.parametrize("case", ["dy_dtype", "dy_shape", "mean_shape", "mean_dtype", "dy_stride"])
def test_layer_norm_bwd_checks(host, case):
    torch = host
    x, dy, m, r = torch.zeros(4, 64), torch.zeros(4, 64), torch.zeros(4), torch.zeros(4)
    if case == "dy_dtype":
        dy = dy.bfloat16()
    elif case == "dy_shape":
        dy = torch.zeros(5, 64)
    elif case == "mean_shape":
        m = torch.zeros(5)
    elif case == "mean_dtype":
        r = r.double()
    elif case == "dy_stride":
        dy = torch.zeros(64, 4).t()
    with pytest.raises(ValueError):
        binding.layer_norm_bwd(dy, x, m, r, torch.zeros(64))


@pytest.mark.parametrize("case", ["dtype", "bands", "bands_odd", "freqs", "pos", "k_shape",
                                  "k_strides", "feature_stride", "out_k_alone"])
def test_rope_scaled_checks(host, case):
    torch = host
    q = k = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    kw = dict(grid=(1, 2, 4), bands=(8, 8, 8), freqs=[1.0] * 12)
    if case == "dtype":
        q = q.float()
    elif case == "bands":
        kw["bands"], kw["freqs"] = (32, 32, 2), [1.0] * 33
    elif case == "bands_odd":
        kw["bands"] = (7, 9, 8)
    elif case == "freqs":
        kw["freqs"] = [1.0] * 11
    elif case == "pos":
        kw["pos_scale"] = (1.0, 1.0)
    elif case == "k_shape":
        k = torch.zeros(1, 2, 9, 64, dtype=torch.bfloat16)
    elif case == "k_strides":
        k = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16).transpose(1, 2)
    elif case == "feature_stride":
        q = k = torch.zeros(1, 2, 64, 8, dtype=torch.bfloat16).transpose(2, 3)
    elif case == "out_k_alone":
        k, kw["out_k"] = None, q
    with pytest.raises(ValueError):
        binding.rope3d_scaled(q, k, **kw)
