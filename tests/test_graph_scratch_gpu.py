"""Captured graphs and the library's scratch (segment summaries, partial results
of split keys): a graph stays valid when the stream it was captured on later
needs more scratch, and graphs captured on streams of their own can be replayed
at the same time."""
import pytest
import torch

from video_diffusion_transformer_non_b200 import autograd, binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def randn(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(BF)


def ids(S, n):
    return (torch.arange(S, device="cuda") * n // S).int()[None].contiguous()


@pytest.mark.parametrize("with_ids,S_q,S_kv", [(True, 300, 300), (False, 200, 20000)])
def test_graph_outlives_its_scratch(with_ids, S_q, S_kv):
    """Ids, and keys split by the library's own choice."""
    D, H = 64, 2
    q, k, v = randn(1, 1, H, S_q, D), randn(2, 1, H, S_kv, D), randn(3, 1, H, S_kv, D)
    seg = (ids(S_q, 3), ids(S_kv, 3)) if with_ids else (None, None)
    want = binding.attention(q, k, v, *seg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.attention(q, k, v, *seg)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = binding.attention(q, k, v, *seg)
    for S in (70000, 140000):       # more scratch on that stream, twice
        x, big = randn(4, 1, 8, 300, D), randn(5, 1, 8, S, D)
        with torch.cuda.stream(side):
            binding.attention(x, big, big, ids(300, 2), ids(S, 2))
            binding.attention(x, big, big)
        torch.cuda.synchronize()
        for t in got:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert binding.device_status() == 0


def test_training_steps_replayed_at_once():
    """Two steps (norm, rotation, attention with ids, and back) captured on
    streams of their own, replayed together many times."""
    B, H, S, D = 1, 4, 500, 64
    turn = dict(grid=(5, 10, 10), bands=(16, 24, 24))
    w = [randn(20 + i, D) for i in range(4)]

    def step(x, seg, dout):
        x = x.detach().requires_grad_()
        p = [t.detach().requires_grad_() for t in w]
        q, k, v = (x[:, :, i].transpose(1, 2) for i in range(3))
        out, _ = autograd.qkv_attention(q, k, v, dict(q=p[:2], k=p[2:]), turn, seg, seg)
        return (out, *torch.autograd.grad(out, [x] + p, dout))

    graphs = []
    for n in (2, 5):
        x, seg, dout = randn(n, B, S, 3, H, D), ids(S, n), randn(10 + n, B, H, S, D)
        want = step(x, seg, dout)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x, seg, dout)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = step(x, seg, dout)
        graphs.append((g, torch.cuda.Stream(), got, want, (x, seg, dout)))
    for _ in range(5):
        for _, _, got, _, _ in graphs:
            for t in got:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(20):
            for g, stream, *_ in graphs:
                with torch.cuda.stream(stream):
                    g.replay()
        torch.cuda.synchronize()
        for _, _, got, want, _ in graphs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_operators_on_several_streams_at_once():
    """The backward pass, the norm with its gradients and the rotation, many calls
    on each of three streams that overlap."""
    D, H = 128, 3
    work = []
    for i, S in enumerate((700, 1300, 2100)):
        q, k, v, dout = (randn(30 + 10 * i + j, 1, H, S, D) for j in range(4))
        out, lse = binding.attention(q, k, v, ids(S, i + 1), ids(S, i + 1))
        w = randn(9, D)
        turn = dict(grid=(1, S // 10, 10), bands=(44, 42, 42),
                    freqs=binding.rope3d_frequencies((44, 42, 42)))

        def call(stream=None, q=q, k=k, v=v, dout=dout, out=out, lse=lse, w=w, turn=turn, S=S, i=i):
            grads = binding.attention_bwd(dout, q, k, v, out, lse, ids(S, i + 1), ids(S, i + 1),
                                          stream=stream, n_split=i + 1)
            y, m, r = binding.layer_norm(q, w, stream=stream)
            back = binding.layer_norm_bwd(dout, q, m, r, w, stream=stream)
            return (*grads, y, m, r, *back, *binding.rope3d_scaled(q, k, stream=stream, **turn))
        work.append((call, torch.cuda.Stream()))
    want = [call() for call, _ in work]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [None] * 3
        for _ in range(4):
            for i, (call, stream) in enumerate(work):
                with torch.cuda.stream(stream):
                    got[i] = call()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for s, t in zip(a, b):
                assert torch.equal(s, t)
