"""Refusals of the attention's backward pass, at the C entry point and in the
binding, and its workspace's size: host logic, no GPU."""
import pytest

from video_diffusion_transformer_non_b200 import binding

A = 1 << 20   # an aligned address that is never read
OK, NULL, SEG_PAIR, BAD_D, BAD_SHAPE, MISALIGNED = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def codes():
    """The header's status values by name."""
    import re
    with open(binding._HEADER) as f:
        return {n: int(v) for n, v in re.findall(r"VIDATTN_(?:ERR_)?(\w+) = (\d+)", f.read())}


def call(q=A, k=A, v=A, out=A, dout=A, lse=A, dlse=None, sq=None, sk=None, dq=A, dk=A, dv=A, B=1,
         H=2, S_q=256, S_kv=256, D=128, scale=0.1, flags=0, ws=A, n=1 << 30):
    return binding.load_library().vidattn_bwd(q, k, v, out, dout, lse, dlse, sq, sk, dq, dk, dv, B,
                                              H, S_q, S_kv, D, scale, flags, ws, n, None)


@pytest.mark.parametrize("kw,name", [
    *((dict([(n, None)]), "NULL") for n in ("q", "k", "v", "out", "dout", "lse", "dq", "dk", "dv",
                                            "ws")),
    *((dict([(n, A + 8)]), "MISALIGNED") for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv",
                                                   "ws")),
    (dict(lse=A + 2), "MISALIGNED"), (dict(dlse=A + 1), "MISALIGNED"),
    (dict(sq=A + 2, sk=A), "MISALIGNED"),
    (dict(sq=A), "SEG_PAIR"), (dict(sk=A), "SEG_PAIR"),
    (dict(D=96), "UNSUPPORTED_D"), (dict(D=256), "UNSUPPORTED_D"),
    (dict(B=0), "BAD_SHAPE"), (dict(H=0), "BAD_SHAPE"), (dict(B=70000), "BAD_SHAPE"),
    (dict(S_q=-1), "BAD_SHAPE"), (dict(S_kv=-1), "BAD_SHAPE"),
    (dict(S_kv=2 ** 31 - 2), "BAD_SHAPE"),
    (dict(scale=float("nan")), "BAD_SHAPE"), (dict(scale=float("inf")), "BAD_SHAPE"),
    (dict(flags=2), "BAD_SHAPE"), (dict(flags=65 << 8), "BAD_SHAPE"),
    (dict(flags=1 << 16), "BAD_SHAPE"),
    (dict(n=0), "SCRATCH_LIMIT"), (dict(n=2047), "SCRATCH_LIMIT"),
])
def test_argument_errors_return_before_any_launch(codes, kw, name):
    assert call(**kw) == codes[name]


def test_nothing_to_do_is_ok(codes):
    assert call(S_q=0, S_kv=0, ws=None, n=0) == codes["OK"]


def test_workspace_bytes():
    """Row statistics (256 floats a 128-query tile and head), with ids 16
    bytes a tile, with splits the ranges' fp32 partial sums."""
    ws = binding.bwd_workspace
    up = lambda n: (n + 255) // 256 * 256
    S = binding.VIDATTN_SPLIT_KV
    stats = lambda BH, S_q: up(BH * -(-S_q // 128) * 1024)
    assert ws(False, 1, 2, 300, 500, 64, S(1)) == stats(2, 300)
    assert ws(True, 3, 2, 300, 500, 64, S(1)) == stats(6, 300) + up(16 * 3 * (3 + 4))
    assert ws(False, 1, 2, 300, 500, 64, S(2)) == \
        stats(2, 300) + up(2 * 2 * 2 * 500 * 64 * 4) + up(2 * 2 * 300 * 64 * 4)
    assert ws(False, 1, 40, 32760, 32760, 128) == stats(40, 32760)     # enough units: no splits
    assert ws(False, 1, 2, 300, 500, 96) == -1
    assert ws(False, 0, 2, 300, 500, 64) == -1
    assert ws(False, 1, 2, 300, 500, 64, S(65)) == -1


@pytest.fixture
def host(monkeypatch):
    """The binding's checks on CPU tensors; a call that passes them all fails
    in the library (no CUDA device here) or reaches it never."""
    import torch
    monkeypatch.setattr(binding, "_DEVICE_TYPE", "cpu")

    def never(*a, **k):
        raise AssertionError("a refused call reached the library")

    monkeypatch.setattr(binding, "vidattn_bwd", never)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    return torch, bf


@pytest.mark.parametrize("case", ["dout_dtype", "dout_shape", "dout_strided", "out_shape",
                                  "lse_dtype", "lse_shape", "dlse_shape", "seg_one", "seg_dtype",
                                  "seg_shape", "q_ndim", "kv_shape"])
def test_binding_checks(host, case):
    torch, bf = host
    q, k, v, out, dout = (bf(1, 2, 16, 64) for _ in range(5))
    lse = torch.zeros((1, 2, 16))
    kw = {}
    if case == "dout_dtype":
        dout = dout.float()
    elif case == "dout_shape":
        dout = bf(1, 2, 15, 64)
    elif case == "dout_strided":
        dout = bf(1, 16, 2, 64).transpose(1, 2)
    elif case == "out_shape":
        out = bf(1, 2, 16, 128)
    elif case == "lse_dtype":
        lse = lse.double()
    elif case == "lse_shape":
        lse = torch.zeros((1, 2, 17))
    elif case == "dlse_shape":
        kw["dlse"] = torch.zeros((1, 1, 16))
    elif case == "seg_one":
        kw["seg_q"] = torch.zeros((1, 16), dtype=torch.int32)
    elif case == "seg_dtype":
        kw["seg_q"] = kw["seg_kv"] = torch.zeros((1, 16), dtype=torch.int64)
    elif case == "seg_shape":
        kw["seg_q"] = kw["seg_kv"] = torch.zeros((1, 17), dtype=torch.int32)
    elif case == "q_ndim":
        q = q[0]
    elif case == "kv_shape":
        v = bf(1, 2, 17, 64)
    with pytest.raises(ValueError):
        binding.attention_bwd(dout, q, k, v, out, lse, **kw)
