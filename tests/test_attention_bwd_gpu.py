"""The attention's backward pass (vidattn_bwd) against its formula in 64 bits,
at sizes and masks where it can go wrong: one token, ragged tiles, other
numbers of queries than keys, the causal limit with rows that see nothing,
ids in any order, split units, gradients of lse, scales.  Bounds: _bwd_ref."""
import math

import pytest
import torch

import _bwd_ref as ref
from _gpu_helpers import GUARD, SENTINEL_BF16
from video_diffusion_transformer_non_b200 import binding

pytestmark = pytest.mark.gpu


def randn(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def make(B, H, S_q, S_kv, D, seed, ids=None, with_dlse=False, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = dict(q=randn(gen, B, H, S_q, D, scale=scale), k=randn(gen, B, H, S_kv, D),
             v=randn(gen, B, H, S_kv, D), dout=randn(gen, B, H, S_q, D), dlse=None,
             seg_q=None, seg_kv=None)
    if with_dlse:
        x["dlse"] = randn(gen, B, H, S_q, dtype=torch.float32)
    if ids == "runs":            # video, text and padding, cut anywhere
        cut = lambda S: (torch.arange(S, device="cuda")[None] * 3 // max(S, 1)).repeat(B, 1)
        x["seg_q"], x["seg_kv"] = cut(S_q).int(), cut(S_kv).int()
    elif ids == "any":           # any order; id 5 has queries but no keys, 7 keys but no queries
        x["seg_q"] = torch.randint(-2, 2, (B, S_q), generator=gen, device="cuda").int()
        x["seg_kv"] = torch.randint(-2, 2, (B, S_kv), generator=gen, device="cuda").int()
        x["seg_q"][:, ::5] = 5
        x["seg_kv"][:, ::7] = 7
    elif ids == "far":           # runs far apart: many tiles of a unit are not visited
        pat = lambda S: ((torch.arange(S, device="cuda") // 100) % 4)[None].repeat(B, 1)
        x["seg_q"], x["seg_kv"] = pat(S_q).int(), pat(S_kv).int()
        x["seg_q"][:, S_q // 2:] += 10
        x["seg_kv"][:, S_kv // 2:] += 10
    return x


class Guarded:
    def __init__(self, shape):
        n = math.prod(shape)
        self.buf = torch.full((n + 2 * GUARD,), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.buf.view(torch.int16)[:GUARD] = SENTINEL_BF16
        self.buf.view(torch.int16)[GUARD + n:] = SENTINEL_BF16
        self.t = self.buf[GUARD:GUARD + n].view(shape)

    def check(self):
        b = self.buf.view(torch.int16)
        n = self.t.numel()
        assert bool((b[:GUARD] == SENTINEL_BF16).all() and (b[GUARD + n:] == SENTINEL_BF16).all())
        assert not bool(self.t.isnan().any()), "an element was never written"


def call(x, out, lse, causal, scale, n_split=0):
    """The C entry point with guarded outputs and a workspace full of NaNs,
    guarded behind its last byte."""
    B, H, S_q, D = x["q"].shape
    S_kv = x["k"].shape[2]
    flags = int(causal) | binding.VIDATTN_SPLIT_KV(n_split)
    n = binding.bwd_workspace(x["seg_q"] is not None, B, H, S_q, S_kv, D, flags)
    assert n > 0 and n % 256 == 0
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    g = dict(dq=Guarded(x["q"].shape), dk=Guarded(x["k"].shape), dv=Guarded(x["v"].shape))
    st = binding.vidattn_bwd(x["q"], x["k"], x["v"], out, x["dout"], lse, x["dlse"], x["seg_q"],
                             x["seg_kv"], g["dq"].t, g["dk"].t, g["dv"].t, B, H, S_q, S_kv, D,
                             scale, flags, ws, n)
    assert st == 0, binding.status_string(st)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert bool((ws[n:] == 0xFF).all()), "written behind the workspace"
    for t in g.values():
        t.check()
    return {name: t.t for name, t in g.items()}


def run(x, causal=False, scale=None, n_split=0, what=""):
    D = x["q"].shape[3]
    scale = D ** -0.5 if scale is None else scale
    see = ref.visible(x["seg_q"], x["seg_kv"], x["q"].shape[2], x["k"].shape[2], causal, "cuda")
    out, lse = ref.forward(x["q"], x["k"], x["v"], see, scale)
    out, lse = out.to(torch.bfloat16), lse.float()
    got = call(x, out, lse, causal, scale, n_split)
    r = ref.backward(x["q"], x["k"], x["v"], out, x["dout"], lse, x["dlse"], see, scale)
    ref.check(got, r, what)
    # what no pair reaches is exactly zero
    none_q, none_k = ~see.any(3), ~see.any(2)
    shape = x["q"].shape
    assert bool((got["dq"][none_q.expand(shape[0], shape[1], -1)] == 0).all())
    for n in ("dk", "dv"):
        assert bool((got[n][none_k.expand(shape[0], shape[1], -1)] == 0).all())
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S_q,S_kv", [(1, 1), (1, 300), (300, 1), (2, 2), (127, 129), (128, 128),
                                      (129, 127), (640, 640), (1000, 333)])
def test_sizes(D, S_q, S_kv):
    run(make(1, 2, S_q, S_kv, D, 1000 + S_q))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S_q,S_kv", [(1, 1), (5, 300), (300, 5), (384, 384), (700, 700),
                                      (900, 260), (260, 900)])
def test_causal(D, S_q, S_kv):
    """S_q > S_kv: the first S_q - S_kv queries see nothing."""
    run(make(2, 1, S_q, S_kv, D, 2000 + S_q), causal=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ids", ["runs", "any", "far"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("S_q,S_kv", [(3, 2), (500, 500), (1100, 700)])
def test_ids(D, ids, causal, S_q, S_kv):
    run(make(2, 2, S_q, S_kv, D, 3000 + S_q, ids), causal=causal)


@pytest.mark.parametrize("D,ids,causal,n_split", [
    (128, None, False, 2), (128, None, True, 5), (64, "runs", False, 3), (64, "far", True, 64),
    (128, "any", True, 7), (64, None, False, 64)])
def test_split_units(D, ids, causal, n_split):
    """Ranges that are empty (more of them than tiles), or end anywhere."""
    run(make(2, 3, 1500, 900, D, 4000 + n_split, ids), causal=causal, n_split=n_split)


def test_split_is_chosen_for_few_units():
    """One head, many keys: the library's own choice splits (the workspace
    then holds partial sums)."""
    x = make(1, 1, 200, 20000, 128, 4500)
    assert binding.bwd_workspace(False, 1, 1, 200, 20000, 128) > 4 * 200 * 128
    run(x)


@pytest.mark.parametrize("D", [64, 128])
def test_gradient_of_lse(D):
    run(make(1, 2, 300, 450, D, 5000, with_dlse=True))
    run(make(1, 2, 450, 300, D, 5001, "any", with_dlse=True), causal=True)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-4])
def test_scales(scale):
    run(make(1, 2, 260, 390, 64, 6000), scale=scale)


def test_sharp_rows():
    """Large scores: most weights vanish, one of a row is near 1."""
    run(make(1, 2, 500, 500, 128, 6100, scale=12.0))


def test_joint_sequence():
    """The small joint sequence, two of its heads."""
    x = make(2, 2, 4389, 4389, 128, 7000)
    row = torch.zeros(4389, dtype=torch.int32, device="cuda")
    row[4096:], row[4352:] = 1, 2
    x["seg_q"] = x["seg_kv"] = row.expand(2, -1).contiguous()
    run(x)


def test_more_tiles_than_a_unit_lists():
    """With ids and more query tiles than a unit keeps as bits, it walks
    every tile of its range and masks them all."""
    S_q = 3100 * 128 + 5
    x = make(1, 1, S_q, 200, 64, 7500, "runs")
    run(x)
    run(x, causal=True)


def test_after_the_forward_kernel():
    """binding.attention's own out and lse, equal ids and strides; the same
    bits from a second call, from another stream, and with a head on its own."""
    x = make(2, 3, 700, 700, 128, 8000, "far")
    out, lse = binding.attention(x["q"], x["k"], x["v"], x["seg_q"], x["seg_kv"], causal=True)
    a = binding.attention_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, x["seg_q"],
                              x["seg_kv"], causal=True)
    see = ref.visible(x["seg_q"], x["seg_kv"], 700, 700, True, "cuda")
    ref.check(dict(zip(("dq", "dk", "dv"), a)),
              ref.backward(x["q"], x["k"], x["v"], out, x["dout"], lse, None, see, 128 ** -0.5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = binding.attention_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, x["seg_q"],
                              x["seg_kv"], causal=True, stream=side)
    side.synchronize()
    one = lambda t: t[:, 1:2].contiguous()
    c = binding.attention_bwd(one(x["dout"]), one(x["q"]), one(x["k"]), one(x["v"]), one(out),
                              one(lse), x["seg_q"], x["seg_kv"], causal=True)
    torch.cuda.synchronize()
    for s, t, u in zip(a, b, c):
        assert torch.equal(s, t)
        assert torch.equal(s[:, 1:2], u)


def test_differences():
    """Central differences of the loss sum(out * g) + sum(lse * h) in 64 bits
    along random directions; the gradients may be off by their bounds."""
    x = make(1, 2, 60, 90, 64, 9000, with_dlse=True)
    D = 64
    scale = D ** -0.5
    see = ref.visible(None, None, 60, 90, True, "cuda")
    out, lse = ref.forward(x["q"], x["k"], x["v"], see, scale)
    got = call(x, out.to(torch.bfloat16), lse.float(), True, scale)
    bounds = ref.backward(x["q"], x["k"], x["v"], out.to(torch.bfloat16), x["dout"], lse.float(),
                          x["dlse"], see, scale)
    # delta used the rounded out: |d delta| <= 2^-8 sum |dout out|, and lse
    # rounded to fp32 turns P by 2^-24 |lse|; both enter through P
    p = torch.where(see, (x["q"].double() @ x["k"].double().transpose(2, 3) * scale
                          - lse[..., None]).exp(), 0.0)
    dd = 2.0 ** -8 * (x["dout"].double() * out).abs().sum(-1, keepdim=True)
    extra = dict(dq=scale * (p * dd) @ x["k"].double().abs(),
                 dk=scale * (p * dd).transpose(2, 3) @ x["q"].double().abs(), dv=0.0)

    def loss(q, k, v):
        o, l = ref.forward(q, k, v, see, scale)
        return (o * x["dout"].double()).sum() + (l * x["dlse"].double()).sum()

    gen = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        u = torch.randn(x[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        at = {n: x[n].double() for n in "qkv"}
        h = 1e-4
        f = [loss(**{**at, name: at[name] + s * h * u}) for s in (1, -1)]
        slope = ((f[0] - f[1]) / (2 * h)).item()
        mine = (got[grad].double() * u).sum().item()
        tol = ((bounds[grad][1] + extra[grad] + 1e-6 * bounds[grad][0].abs()) * u.abs()).sum()
        # the third derivative's share of a central difference: h^2 |slope| order
        assert abs(mine - slope) <= tol.item() + 1e-4 * abs(slope), (name, mine, slope, tol.item())


@pytest.mark.parametrize("n_split", [0, 3])
def test_graph_replay(n_split):
    """Captured with its workspace; replayed on new inputs in the same buffers."""
    x, y = make(1, 2, 600, 600, 128, 9100, "far"), make(1, 2, 600, 600, 128, 9101, "far")
    scale = 128 ** -0.5

    def fwd(z):
        return binding.attention(z["q"], z["k"], z["v"], z["seg_q"], z["seg_kv"])

    names = ("q", "k", "v", "dout")
    buf = {n: x[n].clone() for n in names}
    out, lse = (t.clone() for t in fwd(x))
    args = lambda: (buf["dout"], buf["q"], buf["k"], buf["v"], out, lse, x["seg_q"], x["seg_kv"],
                    scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.attention_bwd(*args(), n_split=n_split)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        grads = binding.attention_bwd(*args(), n_split=n_split)
    for z in (y, x):
        for n in names:
            buf[n].copy_(z[n])
        o, l = fwd(z)
        out.copy_(o)
        lse.copy_(l)
        direct = binding.attention_bwd(*args(), n_split=n_split)
        for t in grads:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(grads, direct):
            assert torch.equal(a, b)


def test_no_tokens():
    """No keys: dq is zero; no queries: dk and dv are."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, e = randn(gen, 1, 2, 5, 64), randn(gen, 1, 2, 0, 64)
    lse = torch.full((1, 2, 5), -math.inf, device="cuda")
    dq, dk, dv = binding.attention_bwd(q, q, e, e, torch.zeros_like(q), lse)
    assert bool((dq == 0).all()) and dk.shape == e.shape
    dq, dk, dv = binding.attention_bwd(e, e, q, q, e, lse[:, :, :0])
    assert bool((dk == 0).all()) and bool((dv == 0).all()) and dq.numel() == 0
