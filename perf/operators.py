"""The token-wise operators around the attention layer, as cases to measure: the
linear product with its epilogue, the norms around a residual branch, and the
loss taken straight from the hidden states.

``run`` computes a case in elementary torch operations in 32 bits (``own`` is
false) or through the library's entry points (``own`` is true); ``exact`` is the
operator's definition in 64 bits, its gradients by differentiating it.

  linear       z = x W^T + b,  y = act(z) + residual;  swiglu: W holds the gate's
               rows, then the other factor's, y = silu(z_gate) * z_up + residual
  linear_bwd   dx, dW, db of sum(y * dy), from the saved z
  norm         r = res_scale * x + gate * rmsnorm(h; w_post),  u = rmsnorm(r; w_pre)
  norm_bwd     the gradients of sum(r * dr) + sum(u * du), from the saved r
  loss         S_s = sum over shard s of logsumexp(x W^T) - (x W^T)[label],
               C_s its counted tokens, L = sum S / sum C
  loss_bwd     the same, and dL/dx, dL/dW
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-6


def listed():
    return [
        # one decoded token through a gated feed-forward input product: bound by the weights' bytes
        {"name": "linear_token", "op": "linear", "tokens": 1, "k": 2560, "n": 10240, "act": "swiglu",
         "bias": False, "residual": False, "save": False},
        # a small decode batch through the product back to the residual stream
        {"name": "linear_batch_residual", "op": "linear", "tokens": 24, "k": 10240, "n": 2560, "act": "none",
         "bias": False, "residual": True, "save": False},
        # a ragged prompt through a biased gelu product with a width that fills no tile
        {"name": "linear_ragged_gelu", "op": "linear", "tokens": 1003, "k": 1032, "n": 1544, "act": "gelu",
         "bias": True, "residual": True, "save": True},
        # training forward of the 8K sequence's gated product, z kept for the backward
        {"name": "linear_train_8k", "op": "linear", "tokens": 8192, "k": 2560, "n": 10240, "act": "swiglu",
         "bias": False, "residual": False, "save": True},
        # its backward
        {"name": "linear_bwd_8k", "op": "linear_bwd", "tokens": 8192, "k": 2560, "n": 10240, "act": "swiglu",
         "bias": False},
        # one decoded token between two blocks: launch latency
        {"name": "norm_token", "op": "norm", "world": 1, "batch": 1, "tokens": 1, "d": 2560, "dtype": "bf16",
         "gate": "channel", "post": True},
        # 64K tokens between two blocks, gated by channel: memory traffic
        {"name": "norm_64k", "op": "norm", "world": 4, "batch": 1, "tokens": 65536, "d": 2560, "dtype": "bf16",
         "gate": "channel", "post": True},
        # its backward, two sequences, each with a gate of its own
        {"name": "norm_bwd_64k", "op": "norm_bwd", "world": 4, "batch": 2, "tokens": 65536, "d": 2560,
         "dtype": "bf16", "gate": "sequence", "post": True},
        # exact type, a gate for every token, an odd token count and width
        {"name": "norm_bwd_f32", "op": "norm_bwd", "world": 3, "batch": 1, "tokens": 2997, "d": 1028,
         "dtype": "f32", "gate": "token", "post": True},
        # scoring a short answer: bound by the vocabulary's bytes
        {"name": "loss_few", "op": "loss", "world": 1, "tokens": 37, "d": 2560, "vocab": 151936, "ignored": 0.0},
        # ragged shards, an odd vocabulary, a fifth of the labels ignored
        {"name": "loss_bwd_ragged", "op": "loss_bwd", "world": 3, "tokens": 1503, "d": 520, "vocab": 32003,
         "ignored": 0.2},
        # the training step's loss at 8K tokens over the whole vocabulary
        {"name": "loss_bwd_8k", "op": "loss_bwd", "world": 4, "tokens": 8192, "d": 2560, "vocab": 151936,
         "ignored": 0.1},
    ]


def _spread(rng, lo, hi, step=1):
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return min(hi, max(lo, v // step * step))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "norm", "norm_bwd", "loss", "loss_bwd"])
    if op in ("linear", "linear_bwd"):
        act = rng.choice(["none", "gelu", "silu", "swiglu"])
        k, n = _spread(rng, 64, 10240, 8), _spread(rng, 64, 10240, 8)
        tokens = _spread(rng, 1, 8192)
        while tokens * k * n > 8192 * 2560 * 10240:
            k = max(64, k // 16 * 8)
        case = {"op": op, "tokens": tokens, "k": k, "n": n, "act": act, "bias": rng.random() < 0.5}
        if op == "linear":
            case |= {"residual": rng.random() < 0.5, "save": rng.random() < 0.5}
        return case
    world = rng.choice([1, 2, 3, 4, 8])
    if op in ("norm", "norm_bwd"):
        batch = rng.choice([1, 2, 3])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = _spread(rng, 64, 8192, 8 if dtype == "bf16" else 4)
        shard = _spread(rng, 1, max(1, 65536 * 2560 // (d * world * batch * 2)))
        return {"op": op, "world": world, "batch": batch, "tokens": world * batch * shard, "d": d, "dtype": dtype,
                "gate": rng.choice(["none", "channel", "sequence", "token"]), "post": rng.random() < 0.7}
    d, vocab = _spread(rng, 64, 2560, 8), _spread(rng, 1000, 151936)
    shard = _spread(rng, 1, 8192 // world)
    return {"op": op, "world": world, "tokens": world * shard, "d": d, "vocab": vocab,
            "ignored": rng.choice([0.0, 0.1, 0.5])}


def work(case):
    t = case["tokens"]
    if case["op"] in ("linear", "linear_bwd"):
        k, n = case["k"], case["n"]
        nw = 2 * n if case["act"] == "swiglu" else n
        bias = 2 * nw if case["bias"] else 0
        if case["op"] == "linear":
            out = t * n * (2 if case["residual"] else 1) + (t * nw if case["save"] else 0)
            return {"bytes": 2 * (t * k + nw * k + out) + bias, "flops": 2 * t * k * nw}
        saved = 0 if case["act"] == "none" else t * nw
        return {"bytes": 2 * (2 * t * k + 2 * nw * k + t * n + saved) + 2 * bias, "flops": 4 * t * k * nw}
    if case["op"] in ("norm", "norm_bwd"):
        d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
        gate = t * d if case["gate"] == "token" else 0
        if case["op"] == "norm":
            return {"bytes": e * (4 * t * d + gate), "flops": 10 * t * d}
        return {"bytes": e * (6 * t * d + 2 * gate), "flops": 25 * t * d}
    d, v = case["d"], case["vocab"]
    both = 2 if case["op"] == "loss_bwd" else 1
    return {"bytes": both * 2 * (t * d + v * d) + 4 * t, "flops": (6 if both == 2 else 2) * t * d * v}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).add_(mean).to(dtype)

    s, t = dict(case), case["tokens"]
    if case["op"] in ("linear", "linear_bwd"):
        k, n = case["k"], case["n"]
        nw = 2 * n if case["act"] == "swiglu" else n
        s["x"], s["w"] = rnd(t, k), rnd(nw, k, scale=k ** -0.5)
        s["b"] = rnd(nw, scale=0.5) if case["bias"] else None
        if case["op"] == "linear":
            s["res"] = rnd(t, n) if case["residual"] else None
        else:
            # z as the forward saved it
            s["z"] = rnd(t, nw) if case["act"] != "none" else None
            s["dy"] = rnd(t, n)
    elif case["op"] in ("norm", "norm_bwd"):
        p, b, d = case["world"], case["batch"], case["d"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        shape = (p, b, t // (p * b), d)
        s["h"] = rnd(*shape, dtype=dt)
        s["w_post"] = rnd(d, scale=0.1, mean=1.0, dtype=dt) if case["post"] else None
        s["w_pre"] = rnd(d, scale=0.1, mean=1.0, dtype=dt)
        s["g"] = {"none": lambda: None, "channel": lambda: rnd(d, scale=0.5, dtype=dt),
                  "sequence": lambda: rnd(b, d, scale=0.5, dtype=dt),
                  "token": lambda: rnd(*shape, scale=0.5, dtype=dt)}[case["gate"]]()
        if case["op"] == "norm":
            s["x"] = rnd(*shape, dtype=dt)
        else:
            s["r"], s["dr"], s["du"] = rnd(*shape, scale=1.5, dtype=dt), rnd(*shape, dtype=dt), rnd(*shape, dtype=dt)
    else:
        s["x"], s["w"] = rnd(t, case["d"]), rnd(case["vocab"], case["d"], scale=2.0 * case["d"] ** -0.5)
        y = torch.randint(0, case["vocab"], (t,), generator=g, device="cuda", dtype=torch.int32)
        drop = torch.rand(t, generator=g, device="cuda") < case["ignored"]
        drop[0] = False
        s["y"] = y.masked_fill_(drop, IGNORE)
    return s


RES_SCALE = 0.75   # the residual stream's factor in the norm cases


# ------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "none":
        return z
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    gate, up = z.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return [y.bfloat16(), z.bfloat16()] if s["save"] else [y.bfloat16()]


def _plain_linear_bwd(s):
    dy = s["dy"].float()
    if s["act"] == "none":
        dz = dy
    else:
        z = s["z"].float()
        if s["act"] == "gelu":
            c = math.sqrt(2 / math.pi)
            th = torch.tanh(c * (z + 0.044715 * z * z * z))
            dz = dy * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z))
        elif s["act"] == "silu":
            sg = 1 / (1 + torch.exp(-z))
            dz = dy * sg * (1 + z * (1 - sg))
        else:
            gate, up = z.chunk(2, dim=-1)
            sg = 1 / (1 + torch.exp(-gate))
            dz = torch.cat([dy * up * sg * (1 + gate * (1 - sg)), dy * gate * sg], dim=-1)
    out = [(dz @ s["w"].float()).bfloat16(), (dz.t() @ s["x"].float()).bfloat16()]
    return out + [dz.sum(0)] if s["bias"] else out


def _gate(s, dtype):
    g = s["g"]
    if g is None:
        return 1.0
    g = g.to(dtype)
    return g[:, None, :] if s["gate"] == "sequence" else g


def _unit(v):
    """v over its root mean square, and one over that."""
    i = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * i, i


def _plain_norm(s):
    h = s["h"].float()
    if s["w_post"] is not None:
        h = _unit(h)[0] * s["w_post"].float()
    r = RES_SCALE * s["x"].float() + _gate(s, torch.float32) * h
    u = _unit(r)[0] * s["w_pre"].float()
    return [r.to(s["x"].dtype), u.to(s["x"].dtype)]


def _plain_norm_bwd(s):
    dt = s["r"].dtype
    rn, ri = _unit(s["r"].float())
    du, g = s["du"].float(), _gate(s, torch.float32)
    a = du * s["w_pre"].float()
    dr = s["dr"].float() + ri * (a - rn * (a * rn).mean(-1, keepdim=True))
    out = {"dx": (RES_SCALE * dr).to(dt), "dw_pre": (du * rn).sum((0, 1, 2))}
    h = s["h"].float()
    dn = dr * g
    if s["w_post"] is not None:
        hn, hi = _unit(h)
        n = hn * s["w_post"].float()
        b = dn * s["w_post"].float()
        out["dh"] = (hi * (b - hn * (b * hn).mean(-1, keepdim=True))).to(dt)
        out["dw_post"] = (dn * hn).sum((0, 1, 2))
    else:
        n = h
        out["dh"] = dn.to(dt)
    if s["gate"] == "token":
        out["dgate"] = (dr * n).to(dt)
    elif s["gate"] == "sequence":
        out["dgate"] = (dr * n).sum((0, 2))
    elif s["gate"] == "channel":
        out["dgate"] = (dr * n).sum((0, 1, 2))
    return out


def _plain_loss(s):
    p, y = s["world"], s["y"].long()
    z = s["x"].float() @ s["w"].float().t()
    keep = y != IGNORE
    at = torch.where(keep, y, 0)[:, None]
    m = z.max(-1, keepdim=True).values
    e = torch.exp(z - m)
    tot = e.sum(-1, keepdim=True)
    per = torch.where(keep, (m + torch.log(tot) - z.gather(1, at))[:, 0], 0.0)
    shard, count = per.double().view(p, -1).sum(1), keep.view(p, -1).sum(1)
    loss = shard.sum() / count.sum()
    out = {"shard_sum": shard.float(), "shard_count": count, "loss": loss.float().view(1)}
    if s["op"] == "loss_bwd":
        dz = e.div_(tot).scatter_add_(1, at, torch.full_like(tot, -1.0))
        dz = dz.mul_(torch.where(keep, 1.0 / count.sum(), 0.0)[:, None])
        out["dx"] = (dz @ s["w"].float()).bfloat16()
        out["dw"] = (dz.t() @ s["x"].float()).bfloat16()
    return out


# ------------------------------------------------- the library's own calls

def _own(s):
    from long_context_sequence_all_b200 import ulysses as U
    op = s["op"]
    if op in ("linear", "linear_bwd"):
        act = {"none": U.ACT_NONE, "gelu": U.ACT_GELU, "silu": U.ACT_SILU, "swiglu": U.ACT_SWIGLU}[s["act"]]
        if op == "linear":
            out = U.ulysses_linear(s["x"], s["w"], bias=s["b"], residual=s["res"], activation=act,
                                   save_pre=s["save"])
            return list(out) if s["save"] else [out]
        dx, dw, db = U.ulysses_linear_bwd(s["x"], s["w"], s["dy"], pre=s["z"], activation=act,
                                          bias_grad=s["bias"], grad_dtype=torch.bfloat16)
        return [dx, dw, db] if s["bias"] else [dx, dw]
    if op in ("norm", "norm_bwd"):
        mode = {"none": U.GATE_NONE, "channel": U.GATE_CHANNEL, "sequence": U.GATE_SEQUENCE,
                "token": U.GATE_TOKEN}[s["gate"]]
        if op == "norm":
            return list(U.ulysses_residual_norm(s["x"], s["h"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["g"],
                                                gate_mode=mode, res_scale=RES_SCALE, eps=EPS))
        got = U.ulysses_residual_norm_bwd(s["r"], s["h"], dr=s["dr"], du=s["du"], w_pre=s["w_pre"],
                                          w_post=s["w_post"], gate=s["g"], gate_mode=mode, res_scale=RES_SCALE,
                                          eps=EPS)
        return {k: v for k, v in zip(("dx", "dh", "dw_pre", "dw_post", "dgate"), got) if v is not None}
    if op == "loss":
        got = U.ulysses_linear_loss(s["x"], s["w"], s["y"], s["world"], ignore_index=IGNORE)
    else:
        got = U.ulysses_linear_loss_bwd(s["x"], s["w"], s["y"], s["world"], ignore_index=IGNORE,
                                        grad_dtype=torch.bfloat16)
    return dict(zip(("shard_sum", "shard_count", "loss", "dx", "dw"), got))


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd, "loss": _plain_loss, "loss_bwd": _plain_loss}[state["op"]](state)


# ------------------------------------------------------ 64-bit definitions

def _def_linear(x, w, b, act):
    z = torch.einsum("tk,nk->tn", x, w)
    z = z if b is None else z + b
    if act == "swiglu":
        n = w.shape[0] // 2
        return z, torch.sigmoid(z[:, :n]) * z[:, :n] * z[:, n:]
    return z, {"none": lambda: z, "silu": lambda: z * torch.sigmoid(z),
               "gelu": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[act]()


def _def_rms(v, w):
    v = v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS)
    return v if w is None else v * w


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op == "linear":
        z, y = _def_linear(s["x"], s["w"], s["b"], s["act"])
        y = y if s["res"] is None else y + s["res"]
        return [y, z] if s["save"] else [y]
    if op == "linear_bwd":
        if s["z"] is None:
            dz = s["dy"]
        else:
            z = s["z"].requires_grad_()
            # the activation alone: the product with one row of the unit matrix a feature
            n = s["dy"].shape[1]
            if s["act"] == "swiglu":
                y = torch.sigmoid(z[:, :n]) * z[:, :n] * z[:, n:]
            elif s["act"] == "silu":
                y = z * torch.sigmoid(z)
            else:
                y = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            dz, = torch.autograd.grad((y * s["dy"]).sum(), z)
        out = [torch.einsum("tn,nk->tk", dz, s["w"]), torch.einsum("tn,tk->nk", dz, s["x"])]
        return out + [torch.einsum("tn->n", dz)] if s["bias"] else out
    if op in ("norm", "norm_bwd"):
        leaves = {k: s[k].requires_grad_() for k in ("h", "w_post", "w_pre", "g") if s[k] is not None}
        branch = s["h"] if s["w_post"] is None else _def_rms(s["h"], s["w_post"])
        if s["gate"] == "sequence":
            branch = torch.einsum("pbsd,bd->pbsd", branch, s["g"])
        elif s["gate"] != "none":
            branch = branch * s["g"]
        if op == "norm":
            with torch.no_grad():
                r = s["x"] * RES_SCALE + branch
                return [r, _def_rms(r, s["w_pre"])]
        r = s["r"].requires_grad_()
        dr, dw_pre = torch.autograd.grad((r * s["dr"]).sum() + (_def_rms(r, s["w_pre"]) * s["du"]).sum(),
                                         [r, s["w_pre"]])
        names = [k for k in ("h", "w_post", "g") if k in leaves]
        got = torch.autograd.grad((branch * dr).sum(), [leaves[k] for k in names])
        named = {"h": "dh", "w_post": "dw_post", "g": "dgate"}
        return {"dx": dr * RES_SCALE, "dw_pre": dw_pre, **{named[k]: v for k, v in zip(names, got)}}
    x, w, p = s["x"], s["w"], s["world"]
    y = s["y"].long()
    keep = y.ne(IGNORE)
    z = torch.einsum("td,vd->tv", x, w)
    lse = torch.logsumexp(z, 1)
    own_logit = torch.einsum("td,td->t", x, w[y.clamp(min=0)])
    per = (lse - own_logit) * keep
    sums, counts = per.reshape(p, -1).sum(1), keep.reshape(p, -1).sum(1)
    out = {"shard_sum": sums, "shard_count": counts, "loss": (sums.sum() / counts.sum()).reshape(1)}
    if op == "loss_bwd":
        dz = z.sub_(lse[:, None]).exp_()
        dz[torch.arange(len(y), device=y.device)[keep], y[keep]] -= 1
        dz *= (keep / counts.sum())[:, None]
        out["dx"], out["dw"] = torch.einsum("tv,vd->td", dz, w), torch.einsum("tv,td->vd", dz, x)
    return out
