"""The q/k norm in sequence-parallel attention over two gloo ranks on the CPU: it
runs on each rank's shard ahead of the exchange, so the result is that of the
norm over the whole sequence.  The attention and the norm are plain fp64."""
import os
import socket

import numpy as np
import torch
import torch.multiprocessing as mp

from video_diffusion_transformer_non_b200.ulysses import ulysses_attention


def _attn(q, k, v, seg_q, seg_kv, scale, causal):
    s = q @ k.transpose(2, 3) * scale
    lse = s.logsumexp(-1)
    return (s - lse[..., None]).exp() @ v, lse


def _norm(x, weight, bias, eps):
    m = x.mean(-1, keepdim=True)
    y = (x - m) / ((x - m).square().mean(-1, keepdim=True) + eps).sqrt()
    return y if weight is None else y * weight + bias


def _rope(q, k, rope):
    """Marks every token by its global position."""
    t = torch.arange(q.shape[2], dtype=q.dtype)[None, None, :, None] * rope["by"]
    return q + t, k + t


def _data():
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((2, 4, 24, 8), generator=gen, dtype=torch.float64) for _ in range(3))
    return q, k, v, torch.randn(8, generator=gen, dtype=torch.float64), torch.ones(8).double()


def _main(rank, port, queue):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=2)
    try:
        q, k, v, w, b = _data()
        sl = slice(12 * rank, 12 * rank + 12)
        out, lse = ulysses_attention(q[:, :, sl], k[:, :, sl], v[:, :, sl], n_chunks=2,
                                     attn_fn=_attn, rope=dict(by=0.01), rope_fn=_rope,
                                     qk_norm=dict(q=(w, b), eps=1e-3), norm_fn=_norm)
        queue.put((rank, out.numpy(), lse.numpy()))
    finally:
        dist.destroy_process_group()


def test_norm_on_the_shards():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    queue = ctx.Queue()
    procs = [ctx.Process(target=_main, args=(r, port, queue)) for r in range(2)]
    for p in procs:
        p.start()
    res = sorted((queue.get(timeout=120) for _ in range(2)), key=lambda r: r[0])
    for p in procs:
        p.join(60)
    q, k, v, w, b = _data()
    qr, kr = _rope(_norm(q, w, b, 1e-3), _norm(k, None, None, 1e-3), dict(by=0.01))
    out, lse = _attn(qr, kr, v, None, None, 8 ** -0.5, False)
    np.testing.assert_allclose(np.concatenate([r[1] for r in res], 2), out.numpy(), rtol=1e-12,
                               atol=1e-12)
    np.testing.assert_allclose(np.concatenate([r[2] for r in res], 2), lse.numpy(), rtol=1e-12,
                               atol=1e-12)
