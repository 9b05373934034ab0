"""The library's calls as differentiable torch functions: the attention path of
a video DiT block for training.

    attention      binding.attention, differentiable in q, k, v through out and lse
    layer_norm     binding.layer_norm, differentiable in x, weight and bias
    rope3d         binding.rope3d_scaled, differentiable in q (and k)
    qkv_attention  projection -> norm of q and k -> rotary embedding -> attention
                   as one function: the intermediate gradients stay in place

Each runs the library's kernels in both directions on the current stream and
has first derivatives only.  Windows (binding.attention_window) have no
backward pass.

Inside a CUDA graph, capture forward and backward together, or use tensors
whose gradients no eager graph still holds: torch's accumulation of a leaf's
gradient runs on the stream that the leaf was first used on.  The attention's
forward pass keeps scratch per stream where it has ids or splits its keys: graphs
that may be replayed at the same time are captured on streams of their own.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding


def _grad(g, like):
    """The gradient of an output as the kernels take it: contiguous, zero where
    autograd has none."""
    return torch.zeros_like(like) if g is None else g.contiguous()


def _attention_on(q, k, v, seg_q, seg_kv, scale, causal):
    """binding.attention on q's device and its current stream, whichever device
    is current."""
    if not q.is_cuda or torch.cuda.current_device() == q.device.index:
        return binding.attention(q, k, v, seg_q, seg_kv, scale, causal=causal)
    with torch.cuda.device(q.device):
        return binding.attention(q, k, v, seg_q, seg_kv, scale, causal=causal)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, seg_q, seg_kv, scale, causal):
        out, lse = _attention_on(q, k, v, seg_q, seg_kv, scale, causal)
        ctx.save_for_backward(q, k, v, out, lse, seg_q, seg_kv)
        ctx.set_materialize_grads(False)
        ctx.scale, ctx.causal = scale, causal
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dlse):
        q, k, v, out, lse, seg_q, seg_kv = ctx.saved_tensors
        dq, dk, dv = binding.attention_bwd(
            _grad(dout, out), q, k, v, out, lse, seg_q, seg_kv, ctx.scale, ctx.causal,
            None if dlse is None else dlse.contiguous())
        return dq, dk, dv, None, None, None, None


def attention(q, k, v, seg_q=None, seg_kv=None, scale=None, causal=False):
    """binding.attention with gradients; returns (out, lse).  Where a query sees
    no key, out is 0, lse -inf, and both pass no gradient on: lse's may be an
    infinity or a NaN there, out's has to be finite as everywhere."""
    return _Attention.apply(q, k, v, seg_q, seg_kv, scale, causal)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = binding.layer_norm(x, weight, bias, eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        if dy.stride(-1) != 1:   # of a plain sum, or of a transposed use
            dy = dy.contiguous()
        dx, dw, db = binding.layer_norm_bwd(dy, x, mean, rstd, weight,
                                            params=any(ctx.needs_input_grad[1:3]))
        return dx, dw, db if ctx.needs_input_grad[2] else None, None


def _check_bias(weight, bias):
    if weight is None and bias is not None:
        raise ValueError("a bias goes with a weight")


def layer_norm(x, weight=None, bias=None, eps=1e-6):
    """binding.layer_norm with gradients; returns y."""
    _check_bias(weight, bias)
    return _LayerNorm.apply(x, weight, bias, eps)


_TURN = ("grid", "bands", "freqs", "pos_scale", "amplitude", "interleaved", "token_offset")


def rope_arguments(rope):
    """rope3d_scaled's arguments from a dict of them, in which ``freqs`` may be
    left out (theta's own frequencies, 10000 by default) and ``token_offset``
    may be called ``offset``; None stands for an option's default.  Sequences
    are copied: a backward pass turns by what the forward was given."""
    unknown = set(rope) - set(_TURN) - {"theta", "offset"}
    if unknown:
        raise ValueError(f"unknown rope options: {sorted(unknown)}")
    rope = {n: v for n, v in rope.items() if v is not None}
    if "offset" in rope:
        if "token_offset" in rope:
            raise ValueError("give offset or token_offset, not both")
        rope["token_offset"] = rope.pop("offset")
    for n in ("grid", "bands"):
        if n not in rope:
            raise ValueError(f"rope needs {n}")
    turn = {n: rope[n] for n in _TURN if n in rope}
    for n in ("grid", "bands", "pos_scale"):
        if n in turn:
            turn[n] = tuple(turn[n])
    if "freqs" not in turn:
        turn["freqs"] = binding.rope3d_frequencies(turn["bands"], rope.get("theta", 10000.0))
    elif "theta" in rope:
        raise ValueError("give freqs or theta, not both")
    else:
        turn["freqs"] = tuple(map(float, turn["freqs"]))
    return turn


def norm_arguments(qk_norm):
    """(weight, bias) of q, (weight, bias) of k and eps from a qk_norm dict."""
    unknown = set(qk_norm) - {"q", "k", "eps"}
    if unknown:
        raise ValueError(f"unknown qk_norm options: {sorted(unknown)}")
    eps = qk_norm.get("eps")
    return (qk_norm.get("q") or (None, None), qk_norm.get("k") or (None, None),
            1e-6 if eps is None else eps)


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, turn):
        ctx.turn = turn
        return binding.rope3d_scaled(q, k, **turn)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        dq, dk = binding.rope3d_scaled_bwd(dq.contiguous(), None if dk is None else dk.contiguous(),
                                           **ctx.turn)
        return dq, dk, None


def rope3d(q, k=None, **rope):
    """binding.rope3d_scaled of q (and k) with gradients (options: grid, bands,
    freqs or theta, pos_scale, amplitude, interleaved, token_offset); returns
    (q_rot, k_rot or None)."""
    return _Rope.apply(q, k, rope_arguments(rope))


class _QkvAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, wq, bq, wk, bk, eps, turn, seg_q, seg_kv, scale, causal, norm):
        ctx.set_materialize_grads(False)
        stats = (None,) * 4
        qn, kn = q, k
        if norm:
            qn, mq, rq = binding.layer_norm(q, wq, bq, eps)
            kn, mk, rk = binding.layer_norm(k, wk, bk, eps)
            stats = (mq, rq, mk, rk)
        if turn is not None:   # over the norm's results, which nothing else reads
            qn, kn = binding.rope3d_scaled(qn, kn, **turn,
                                           **(dict(out_q=qn, out_k=kn) if norm else {}))
        qn, kn, vn = qn.contiguous(), kn.contiguous(), v.contiguous()
        out, lse = _attention_on(qn, kn, vn, seg_q, seg_kv, scale, causal)
        ctx.save_for_backward(*((q, k) if norm else (None, None)), wq, wk, *stats, qn, kn, vn, out,
                              lse, seg_q, seg_kv)
        ctx.turn, ctx.scale, ctx.causal, ctx.norm = turn, scale, causal, norm
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dlse):
        q, k, wq, wk, mq, rq, mk, rk, qn, kn, vn, out, lse, seg_q, seg_kv = ctx.saved_tensors
        dq, dk, dv = binding.attention_bwd(
            _grad(dout, out), qn, kn, vn, out, lse, seg_q, seg_kv, ctx.scale, ctx.causal,
            None if dlse is None else dlse.contiguous())
        if ctx.turn is not None:
            binding.rope3d_scaled_bwd(dq, dk, out_q=dq, out_k=dk, **ctx.turn)
        dwq = dbq = dwk = dbk = None
        need = ctx.needs_input_grad
        if ctx.norm:
            _, dwq, dbq = binding.layer_norm_bwd(dq, q, mq, rq, wq, out=dq, params=any(need[3:5]))
            _, dwk, dbk = binding.layer_norm_bwd(dk, k, mk, rk, wk, out=dk, params=any(need[5:7]))
        return (dq, dk, dv, dwq, dbq if need[4] else None, dwk, dbk if need[6] else None,
                None, None, None, None, None, None, None)


def qkv_attention(q, k, v, qk_norm=None, rope=None, seg_q=None, seg_kv=None, scale=None,
                  causal=False):
    """A block's attention from its projections, with gradients.

    q, k, v: bf16 [B,H,S,D], any strides with a contiguous last dim (a
    [B,S,H,D] projection's ``transpose(1, 2)``); q and k of equal shape and
    strides where there is a rope.
    qk_norm: dict(q=(weight, bias), k=(weight, bias), eps=1e-6), weight and bias
    [D] or None: layer norm of q and k over each head; {} for one without
    parameters, None for no norm.
    rope: dict of rope3d's options, or None.
    Returns (out bf16 [B,H,S,D], lse fp32 [B,H,S]) as ``attention`` does."""
    wq = bq = wk = bk = None
    eps = 1e-6
    if qk_norm is not None:
        (wq, bq), (wk, bk), eps = norm_arguments(qk_norm)
        _check_bias(wq, bq)
        _check_bias(wk, bk)
    turn = None if rope is None else rope_arguments(rope)
    return _QkvAttention.apply(q, k, v, wq, bq, wk, bk, eps, turn, seg_q, seg_kv, scale, causal,
                               qk_norm is not None)
