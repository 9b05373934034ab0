"""The operators that train the attention path of a video diffusion transformer,
as they are measured: the attention's backward pass, the layer norm of q and k
(and of the hidden state) with its gradients, and the scaled or partial 3D
rotary embedding with its gradient.

``own`` False: the plain forms (elementary torch operations in 32 bits, rounded
once at the end); True: the calls a user makes of the framework.

Where the sizes come from: the 480p latent volume 21 x 30 x 52 (32760 tokens,
heads of 128), the small joint sequence (4096 video + 256 text + 37 padding),
the joint sequence with heads of 64 (17776 tokens + 16 padding) and the tiny
512-token call are the repository's own workloads; the other sizes are generic.
"""
import math

import torch

own = False

# bytes of one score matrix that a plain form or an exact one holds at a time
_CHUNK = 5 << 30


def listed():
    return [
        # latency: the tiny workload, 8 blocks of work
        dict(name="attn_bwd_tiny", op="attn_bwd", B=1, H=2, S_q=512, S_kv=512, D=64, ids="none",
             causal=False),
        # the small joint sequence: video, text and padding each see themselves
        dict(name="attn_bwd_joint_small", op="attn_bwd", B=2, H=12, S_q=4389, S_kv=4389, D=128,
             ids="joint", causal=False),
        # the 480p latent, one segment, 8 of its heads: the largest
        dict(name="attn_bwd_480p_h8", op="attn_bwd", B=1, H=8, S_q=32760, S_kv=32760, D=128,
             ids="none", causal=False),
        # heads of 64, text and video in one segment, padding in another
        dict(name="attn_bwd_d64_joint_h8", op="attn_bwd", B=1, H=8, S_q=17792, S_kv=17792, D=64,
             ids="pad", causal=False),
        # the causal pathway over half of the 480p volume
        dict(name="attn_bwd_causal", op="attn_bwd", B=1, H=8, S_q=16380, S_kv=16380, D=128,
             ids="none", causal=True),
        # cross attention of the 480p latent over 512 text tokens: few key blocks, long sums
        dict(name="attn_bwd_cross", op="attn_bwd", B=1, H=12, S_q=32760, S_kv=512, D=128,
             ids="none", causal=False),
        # the norm ahead of a block over a hidden state of 40 heads x 128
        dict(name="ln_hidden", op="ln_fwd", B=1, H=1, S=32760, N=5120, x="bf16", params="f32"),
        dict(name="ln_hidden_bwd", op="ln_bwd", B=1, H=1, S=32760, N=5120, x="bf16", params="f32"),
        # the norm of q over each head, straight from the projection's [B,S,H,D]
        dict(name="ln_head_bwd", op="ln_bwd", B=1, H=16, S=32760, N=128, x="bf16", params="bf16"),
        # latency: a prompt's tokens in fp32, an odd row length
        dict(name="ln_text_f32", op="ln_fwd", B=1, H=1, S=226, N=1001, x="f32", params="f32"),
        # q and k of the whole 480p latent, from the projection's [B,S,H,D], interleaved pairs,
        # frequencies stretched by parts for a volume twice the trained one
        dict(name="rope_480p", op="rope_fwd", B=1, H=40, T=21, Hg=30, Wg=52, text=0, D=128,
             d_t=44, d_h=42, d_w=42, theta=10000.0, factor=2.0, interleaved=True),
        # the gradient for heads of 64, half pairing, 44 of the 64 features turned, positions
        # interpolated, text behind the video; written into the projection's [B,S,H,D]
        dict(name="rope_d64_bwd", op="rope_bwd", B=2, H=8, T=13, Hg=30, Wg=45, text=242, D=64,
             d_t=12, d_h=16, d_w=16, theta=10000.0, factor=1.5, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_bwd", "attn_bwd", "attn_bwd", "ln_fwd", "ln_bwd", "rope_fwd", "rope_bwd"])
    if op == "attn_bwd":
        D = rng.choice([64, 128])
        ids = rng.choice(["none", "joint", "pad"])
        # at least 2 keys: with one, q and k have no gradient and only rounding is left
        S_q = _log_int(rng, 1, 32760)
        S_kv = S_q if ids != "none" or rng.random() < 0.5 else _log_int(rng, 2, 32760)
        S_q, S_kv = (2, 2) if S_kv < 2 else (S_q, S_kv)
        B, H = rng.randint(1, 2), rng.randint(1, 16)
        most = 8 * 32760 * 32760
        if B * H * S_q * S_kv > most:
            B = 1
            H = max(1, most // (S_q * S_kv))
        return dict(op=op, B=B, H=H, S_q=S_q, S_kv=S_kv, D=D, ids=ids,
                    causal=rng.random() < 0.35)
    if op in ("ln_fwd", "ln_bwd"):
        if rng.random() < 0.5:   # per head
            B, H, N = rng.randint(1, 2), rng.randint(1, 24), rng.choice([64, 128])
            S = _log_int(rng, 1, 32760)
        else:                    # per token
            B, H, N = 1, 1, _log_int(rng, 16, 8192)
            S = _log_int(rng, 1, 32760 if N <= 5120 else 16380)
        return dict(op=op, B=B, H=H, S=S, N=N, x=rng.choice(["bf16", "bf16", "f32"]),
                    params=rng.choice(["f32", "bf16", "none"]))
    D = rng.choice([64, 128])
    step = 2 if rng.random() < 0.5 else 4
    d_t = step * rng.randint(0, D // 8 // step * 2)
    d_h = step * rng.randint(1, D // 4 // step)
    d_w = step * rng.randint(1, (D - d_t - d_h) // step)
    T, Hg, Wg = _log_int(rng, 1, 33), _log_int(rng, 1, 40), _log_int(rng, 1, 52)
    return dict(op=op, B=rng.randint(1, 2), H=rng.randint(1, 16), T=T, Hg=Hg, Wg=Wg,
                text=rng.choice([0, 0, 1, 77, 226, 256]), D=D, d_t=d_t, d_h=d_h, d_w=d_w,
                theta=rng.choice([256.0, 10000.0]), factor=rng.choice([1.0, 1.5, 2.0, 4.0]),
                interleaved=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs


def _randn(gen, shape, dtype, scale=1.0, shift=0.0):
    """N(shift, scale^2) values of `dtype` on the GPU."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(shift, scale, generator=gen)


def _segments(case):
    """int32 [B,S] ids of a joint sequence: "joint" gives video, text and
    padding their own ids, "pad" one id to video and text and one to padding."""
    if case["ids"] == "none":
        return None
    S = case["S_q"]
    pad = min(37, S // 16) if case["ids"] == "joint" else min(16, S // 16)
    text = min(256, S // 8) if case["ids"] == "joint" else 0
    row = torch.zeros(S, dtype=torch.int32)
    row[S - pad - text:] = 1
    row[S - pad:] = 2 if case["ids"] == "joint" else 1
    return row.expand(case["B"], S).contiguous().cuda()


def _visible(case, seg):
    """Which keys each query sees, bool [B,1,S_q,S_kv], or None for all."""
    see = None
    if seg is not None:
        see = (seg[:, :, None] == seg[:, None, :])[:, None]
    if case["causal"]:
        i = torch.arange(case["S_q"], device="cuda")[:, None]
        j = torch.arange(case["S_kv"], device="cuda")[None]
        lim = (j <= i + (case["S_kv"] - case["S_q"]))[None, None]
        see = lim if see is None else see & lim
    return see


def _head_groups(case, item):
    """Heads taken at a time, so that one score matrix stays below _CHUNK."""
    per = case["B"] * case["S_q"] * case["S_kv"] * item
    n = max(1, min(case["H"], _CHUNK // per))
    return [slice(h, min(case["H"], h + n)) for h in range(0, case["H"], n)]


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _bands(case):
    return case["d_t"], case["d_h"], case["d_w"]


def _frequencies(case):
    """Per pair, theta^(-2k/d) of its band, stretched for volumes beyond the
    trained one: interleaved cases by parts (a pair that turns fewer than 1
    times over the trained extent is interpolated by `factor`, more than 8
    times kept, linear in between), with the amplitude 0.1 ln(factor) + 1;
    the others keep them and interpolate the positions.
    Returns (frequencies, position scales, amplitude)."""
    f, out = case["factor"], []
    for d, extent in zip(_bands(case), (case["T"], case["Hg"], case["Wg"])):
        for k in range(d // 2):
            w = case["theta"] ** (-2.0 * k / d)
            if case["interleaved"]:
                turns = max(1.0, extent / f) * w / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - 1.0) / 7.0))
                w = w * keep + w / f * (1.0 - keep)
            out.append(w)
    if case["interleaved"]:
        return out, [1.0, 1.0, 1.0], 0.1 * math.log(f) + 1.0
    return out, [1.0 / f, 1.0 / f, 1.0 / f], 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "attn_bwd":
        B, H, S_q, S_kv, D = (case[n] for n in ("B", "H", "S_q", "S_kv", "D"))
        bf = torch.bfloat16
        q, dout = _randn(gen, (B, H, S_q, D), bf), _randn(gen, (B, H, S_q, D), bf)
        k, v = _randn(gen, (B, H, S_kv, D), bf), _randn(gen, (B, H, S_kv, D), bf)
        seg = _segments(case)
        # what the forward pass left behind
        out = torch.empty_like(q)
        lse = torch.empty((B, H, S_q), dtype=torch.float32, device="cuda")
        see = _visible(case, seg)
        for h in _head_groups(case, 4):
            s = q[:, h].float() @ k[:, h].float().transpose(2, 3) * D ** -0.5
            if see is not None:
                s.masked_fill_(~see, -math.inf)
            lse[:, h] = s.logsumexp(-1)
            p = s.sub_(lse[:, h, :, None]).exp_().nan_to_num_(0.0)
            out[:, h] = (p @ v[:, h].float()).to(bf)
        return dict(case=case, q=q, k=k, v=v, dout=dout, out=out, lse=lse, seg=seg)
    if op in ("ln_fwd", "ln_bwd"):
        B, H, S, N = (case[n] for n in ("B", "H", "S", "N"))
        t = _dtype(case["x"])
        # the projection's [B,S,H,N], seen as [B,H,S,N]
        x = _randn(gen, (B, S, H, N), t, 1.5, 0.3).transpose(1, 2)
        st = dict(case=case, x=x, weight=None, bias=None, eps=1e-6)
        if case["params"] != "none":
            st["weight"] = _randn(gen, (N,), _dtype(case["params"]), 0.2, 1.0)
            st["bias"] = _randn(gen, (N,), _dtype(case["params"]), 0.2)
        if op == "ln_bwd":
            st["dy"] = _randn(gen, (B, H, S, N), t)
            xd = x.double() if x.numel() < 1 << 26 else x.float()
            mean = xd.mean(-1)
            st["mean"] = mean.float()
            st["rstd"] = ((xd - mean[..., None]).square_().mean(-1) + st["eps"]).rsqrt().float()
        return st
    B, H, D = case["B"], case["H"], case["D"]
    S = case["T"] * case["Hg"] * case["Wg"] + case["text"]
    freqs, pos_scale, amplitude = _frequencies(case)
    shape = (B, S, H, D) if op == "rope_fwd" else (B, H, S, D)
    q, k = _randn(gen, shape, torch.bfloat16), _randn(gen, shape, torch.bfloat16)
    if op == "rope_fwd":
        q, k = q.transpose(1, 2), k.transpose(1, 2)
    return dict(case=case, q=q, k=k, freqs=freqs, pos_scale=pos_scale, amplitude=amplitude)


# ------------------------------------------------------------- the plain forms


def _plain_attn_bwd(st):
    case, dt = st["case"], st["q"].dtype
    scale = case["D"] ** -0.5
    see = _visible(case, st["seg"])
    dq, dk, dv = torch.empty_like(st["q"]), torch.empty_like(st["k"]), torch.empty_like(st["v"])
    # the score matrices of all heads at once would not fit the card
    for h in _head_groups(case, 4):
        q, k, v, do, o = (st[n][:, h].float() for n in ("q", "k", "v", "dout", "out"))
        p = q @ k.transpose(2, 3)
        p.mul_(scale).sub_(st["lse"][:, h, :, None])
        if see is not None:
            p.masked_fill_(~see, -math.inf)
        p.exp_()
        dv[:, h] = (p.transpose(2, 3) @ do).to(dt)
        ds = do @ v.transpose(2, 3)
        ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        dq[:, h] = (ds @ k * scale).to(dt)
        dk[:, h] = (ds.transpose(2, 3) @ q * scale).to(dt)
    return dict(dq=dq, dk=dk, dv=dv)


def _plain_ln_fwd(st):
    x = st["x"].float()
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = ((d * d).mean(-1) + st["eps"]).rsqrt()
    y = d * rstd[..., None]
    if st["weight"] is not None:
        y = y * st["weight"].float() + st["bias"].float()
    return dict(y=y.to(st["x"].dtype), mean=mean, rstd=rstd)


def _plain_ln_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    xh = (x - st["mean"][..., None]) * st["rstd"][..., None]
    g = dy if st["weight"] is None else dy * st["weight"].float()
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = (g - c1 - xh * c2) * st["rstd"][..., None]
    if st["weight"] is None:
        return dict(dx=dx.to(st["x"].dtype))
    pt = st["weight"].dtype
    return dict(dx=dx.to(st["x"].dtype), dweight=(dy * xh).sum((0, 1, 2)).to(pt),
                dbias=dy.sum((0, 1, 2)).to(pt))


def _angles(st):
    """fp64 [S, pairs] angles; tokens behind the video volume have none."""
    case = st["case"]
    T, Hg, Wg = case["T"], case["Hg"], case["Wg"]
    n = torch.arange(T * Hg * Wg + case["text"], device="cuda")
    coords = [torch.div(n, Hg * Wg, rounding_mode="floor"),
              torch.div(n, Wg, rounding_mode="floor") % Hg, n % Wg]
    axis = torch.tensor([a for a in range(3) for _ in range(_bands(case)[a] // 2)], device="cuda")
    pos = torch.stack(coords).double() * torch.tensor(st["pos_scale"], dtype=torch.float64,
                                                      device="cuda")[:, None]
    w = torch.tensor(st["freqs"], dtype=torch.float64, device="cuda")
    a = pos[axis] * w[:, None]
    a[:, T * Hg * Wg:] = 0.0
    return a.T, n < T * Hg * Wg


def _pairs(case):
    """Feature indices of the first and the second member of every pair."""
    first, second, start = [], [], 0
    for d in _bands(case):
        k = range(d // 2)
        first += [start + (2 * i if case["interleaved"] else i) for i in k]
        second += [start + (2 * i + 1 if case["interleaved"] else i + d // 2) for i in k]
        start += d
    return first, second


def _plain_rope(st, sign):
    case = st["case"]
    a, video = _angles(st)
    amp = torch.where(video, st["amplitude"], 1.0)[:, None]
    cos, sin = (a.cos() * amp).float(), (a.sin() * amp * sign).float()
    first, second = _pairs(case)
    q, k = st["q"].float(), st["k"].float()
    qo, ko = q.clone(), k.clone()
    qo[..., first] = q[..., first] * cos - q[..., second] * sin
    qo[..., second] = q[..., first] * sin + q[..., second] * cos
    ko[..., first] = k[..., first] * cos - k[..., second] * sin
    ko[..., second] = k[..., first] * sin + k[..., second] * cos
    return dict(q=qo.to(st["q"].dtype), k=ko.to(st["k"].dtype))


# -------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op == "attn_bwd":
        return _plain_attn_bwd(state)
    if op == "ln_fwd":
        return _plain_ln_fwd(state)
    if op == "ln_bwd":
        return _plain_ln_bwd(state)
    return _plain_rope(state, 1.0 if op == "rope_fwd" else -1.0)


def _run_own(st, case, op):
    from video_diffusion_transformer_non_b200 import binding
    if op == "attn_bwd":
        dq, dk, dv = binding.attention_bwd(st["dout"], st["q"], st["k"], st["v"], st["out"],
                                           st["lse"], st["seg"], st["seg"], causal=case["causal"])
        return dict(dq=dq, dk=dk, dv=dv)
    if op == "ln_fwd":
        y, mean, rstd = binding.layer_norm(st["x"], st["weight"], st["bias"], eps=st["eps"])
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "ln_bwd":
        dx, dw, db = binding.layer_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"],
                                            st["weight"])
        return dict(dx=dx) if dw is None else dict(dx=dx, dweight=dw, dbias=db)
    turn = dict(grid=(case["T"], case["Hg"], case["Wg"]), bands=_bands(case),
                freqs=st["freqs"], pos_scale=tuple(st["pos_scale"]), amplitude=st["amplitude"],
                interleaved=case["interleaved"])
    if op == "rope_fwd":
        q, k = binding.rope3d_scaled(st["q"], st["k"], **turn)
        return dict(q=q, k=k)
    B, H, S, D = st["q"].shape
    dq, dk = (torch.empty((B, S, H, D), dtype=st["q"].dtype, device="cuda").transpose(1, 2)
              for _ in range(2))
    binding.rope3d_scaled_bwd(st["q"], st["k"], out_q=dq, out_k=dk, **turn)
    return dict(q=dq, k=dk)


# ------------------------------------------------------- what it cannot do without


def _pairs_seen(case):
    """(query, key) pairs that the masks leave, per head."""
    S_q, S_kv = case["S_q"], case["S_kv"]
    if case["ids"] == "none":
        if not case["causal"]:
            return case["B"] * S_q * S_kv
        # row i sees min(S_kv, i + 1 + S_kv - S_q) keys, none below zero
        lo = max(0, S_q - S_kv)
        first = max(0, S_kv - S_q) + 1
        n = S_q - lo
        return case["B"] * (n * first + n * (n - 1) // 2)
    pad = min(37, S_q // 16) if case["ids"] == "joint" else min(16, S_q // 16)
    text = min(256, S_q // 8) if case["ids"] == "joint" else 0
    runs = (S_q - pad - text, text, pad)
    return case["B"] * sum(n * (n + 1) // 2 if case["causal"] else n * n for n in runs)


def work(case):
    op = case["op"]
    if op == "attn_bwd":
        B, H, S_q, S_kv, D = (case[n] for n in ("B", "H", "S_q", "S_kv", "D"))
        rows = B * H * (4 * S_q * D * 2 + 4 * S_kv * D * 2 + 4 * S_q)
        ids = 0 if case["ids"] == "none" else 4 * B * S_q
        # S, dP, dV, dQ and dK: five products of 2 D flops a visible pair
        return {"bytes": rows + ids, "flops": 10 * D * H * _pairs_seen(case)}
    if op in ("ln_fwd", "ln_bwd"):
        n = case["B"] * case["H"] * case["S"]
        item = 2 if case["x"] == "bf16" else 4
        par = {"bf16": 2, "f32": 4, "none": 0}[case["params"]] * case["N"]
        if op == "ln_fwd":
            return {"bytes": n * (2 * item * case["N"] + 8) + 2 * par, "flops": 8 * n * case["N"]}
        return {"bytes": n * (3 * item * case["N"] + 8) + 3 * par, "flops": 14 * n * case["N"]}
    S = case["T"] * case["Hg"] * case["Wg"] + case["text"]
    values = 2 * case["B"] * case["H"] * S * case["D"]
    return {"bytes": 2 * 2 * values, "flops": 3 * values}


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    return {"attn_bwd": _exact_attn, "ln_fwd": _exact_ln, "ln_bwd": _exact_ln_bwd,
            "rope_fwd": _exact_rope, "rope_bwd": _exact_rope}[case["op"]](case, st)


def _exact_attn(case, st):
    """The gradients of sum(out * dout) with out = softmax(scale q k^T) v, from
    q, k, v and dout alone, a block of query rows of one head at a time."""
    B, H, S_q, S_kv, D = (case[n] for n in ("B", "H", "S_q", "S_kv", "D"))
    dq = torch.zeros((B, H, S_q, D), dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros((B, H, S_kv, D), dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, min(S_q, (1 << 28) // S_kv))
    keys = torch.arange(S_kv, device="cuda")
    for b in range(B):
        for h in range(H):
            K, V = st["k"][b, h].double(), st["v"][b, h].double()
            for r in range(0, S_q, step):
                rows = slice(r, min(S_q, r + step))
                Q, G = st["q"][b, h, rows].double(), st["dout"][b, h, rows].double()
                w = torch.einsum("id,jd->ij", Q, K) / math.sqrt(D)
                hidden = torch.zeros_like(w, dtype=torch.bool)
                if st["seg"] is not None:
                    hidden |= st["seg"][b, rows, None] != st["seg"][b, None, :]
                if case["causal"]:
                    last = torch.arange(r, rows.stop, device="cuda") + S_kv - S_q
                    hidden |= keys[None, :] > last[:, None]
                w = torch.where(hidden, 0.0, torch.exp(
                    w - torch.where(hidden, -math.inf, w).amax(1, keepdim=True).clamp_min(-1e300)))
                total = w.sum(1, keepdim=True)
                w = w / torch.where(total > 0, total, 1.0)
                g = torch.einsum("id,jd->ij", G, V)
                g = w * (g - (w * g).sum(1, keepdim=True))
                dv[b, h] += torch.einsum("ij,id->jd", w, G)
                dk[b, h] += torch.einsum("ij,id->jd", g, Q) / math.sqrt(D)
                dq[b, h, rows] = torch.einsum("ij,jd->id", g, K) / math.sqrt(D)
    return dict(dq=dq, dk=dk, dv=dv)


def _exact_ln(case, st):
    x = st["x"].double()
    var, mean = torch.var_mean(x, -1, correction=0)
    rstd = 1.0 / torch.sqrt(var + st["eps"])
    y = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
    if st["weight"] is not None:
        y = torch.addcmul(st["bias"].double(), y, st["weight"].double())
    return dict(y=y, mean=mean, rstd=rstd)


def _exact_ln_bwd(case, st):
    """Sample by sample: row sums by matrix products with ones and with the row."""
    n = case["N"]
    x, dy = st["x"].double(), st["dy"].double()
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    r = 1.0 / torch.sqrt(var + st["eps"])
    xh = (x - mean) * r
    del x
    w = torch.ones(n, dtype=torch.float64, device="cuda") if st["weight"] is None \
        else st["weight"].double()
    c1 = (dy @ w / n).unsqueeze(-1)
    c2 = ((dy * xh) @ w / n).unsqueeze(-1)
    out = dict(dx=r * (dy * w - c1 - xh * c2))
    if st["weight"] is not None:
        out["dweight"] = torch.einsum("bhsn,bhsn->n", dy, xh)
        out["dbias"] = torch.einsum("bhsn->n", dy)
    return out


def _exact_rope(case, st):
    """As products of complex numbers: feature pairs times amplitude e^(+-i angle)."""
    T, Hg, Wg = case["T"], case["Hg"], case["Wg"]
    S = T * Hg * Wg + case["text"]
    t, h, w = torch.meshgrid(*(torch.arange(n, dtype=torch.float64, device="cuda")
                               for n in (T, Hg, Wg)), indexing="ij")
    sign = 1.0 if case["op"] == "rope_fwd" else -1.0
    outs = {}
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        start = at = 0
        for a, (d, c) in enumerate(zip(_bands(case), (t, h, w))):
            half = d // 2
            for i in range(half):
                one, two = (start + 2 * i, start + 2 * i + 1) if case["interleaved"] \
                    else (start + i, start + half + i)
                turn = torch.polar(torch.full((T * Hg * Wg,), st["amplitude"],
                                              dtype=torch.float64, device="cuda"),
                                   sign * st["pos_scale"][a] * st["freqs"][at + i] * c.reshape(-1))
                z = torch.complex(x[:, :, :T * Hg * Wg, one], x[:, :, :T * Hg * Wg, two]) * turn
                y[:, :, :T * Hg * Wg, one], y[:, :, :T * Hg * Wg, two] = z.real, z.imag
            start, at = start + d, at + half
        assert y.shape[2] == S
        outs[name] = y
    return outs
