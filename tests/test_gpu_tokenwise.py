"""The token-wise operators (linear product with its epilogue, residual norm,
linear loss; forward and backward) against plain implementations in 64 bits.

Element-wise bounds, from the arithmetic of the GPU path:
- a product of bf16 operands is exact, its fp32 accumulation errs by at most one
  fp32 ulp an addition: K 2^-23 of the sum of |terms|;
- a value stored in bf16 moves by half a step, 2^-8 |value|; an operand rounded
  to bf16 before a product (dz) carries 2^-8 into it; the loss's exponentials
  are held in fp16 in between, 2^-11 more;
- the activations' exponential and quotient are good to a few fp32 ulps: 2^-20
  of a sigmoid, so an activation or its derivative errs by 2^-18 (2 + |z|);
- a sum of D squares errs by D 2^-24, its inverse root by half of that.
First-order terms only; the factor 1.05 covers products of two of them.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

from helpers import LOSS_REL
from long_context_sequence_all_b200 import ulysses as U

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -23
HALF = 2.0 ** -8
MORE = 1.05
ACTS = {"none": U.ACT_NONE, "gelu": U.ACT_GELU, "silu": U.ACT_SILU, "swiglu": U.ACT_SWIGLU}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    U.lib()
    U.ulysses_read_error()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rnd(g, *shape, scale=1.0, mean=0.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale + mean).to(dtype)


def _within(got, ref, bound, what):
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    worst = ((g - ref).abs() / bound.clamp_min(1e-30)).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: worst err/bound {worst:.3f}"


# ------------------------------------------------------------------- linear

def _act64(z, act):
    """(act(z), its derivatives by z, or by the gate's and the other factor's z)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    a, b = z.chunk(2, -1)
    s = torch.sigmoid(a)
    return a * s * b, torch.cat([b * s * (1 + a * (1 - s)), a * s], -1)


LINEAR = [  # tokens, K, N, act, bias, residual
    (1, 2560, 1024, "swiglu", False, False),     # one token: the product is cut along K
    (1, 64, 8, "none", True, True),              # the smallest: a single k-step
    (7, 72, 136, "gelu", True, False),           # a ragged k-step, a column tile and 8 columns
    (130, 520, 264, "silu", False, True),        # two CTAs' rows, a ragged column tile
    (257, 1032, 520, "swiglu", True, True),      # a second row tile of one row; the gate's last tile ends inside
    (1000, 256, 2048, "gelu", True, True),
    (4100, 640, 2560, "none", False, True),      # many tiles, each SM pair several
    (2300, 8192, 2304, "silu", True, True),      # 81 tiles: a turn of 74 and the other 7 cut along K
    (600, 4096, 3320, "swiglu", True, True),     # the same, gated, with a ragged tile among the cut ones
    (128, 1032, 520, "gelu", True, True),        # the most tokens of the kernel for few, and one more
    (129, 1032, 520, "gelu", True, True),
    (33, 4096, 136, "swiglu", False, True),      # a tile's k-steps shared by a cluster
]


@pytest.mark.parametrize("T,K,N,act,bias,residual", LINEAR)
def test_linear_forward(T, K, N, act, bias, residual):
    g = _gen(T + K + N)
    nz = 2 * N if act == "swiglu" else N
    x, w = _rnd(g, T, K), _rnd(g, nz, K, scale=K ** -0.5)
    b = _rnd(g, nz, scale=0.5) if bias else None
    r = _rnd(g, T, N) if residual else None
    y, pre = U.ulysses_linear(x, w, bias=b, residual=r, activation=ACTS[act], save_pre=True)
    y2 = U.ulysses_linear(x, w, bias=b, residual=r, activation=ACTS[act])
    assert torch.equal(y, y2)
    xd, wd = x.double(), w.double()
    z = xd @ wd.t() + (b.double() if bias else 0)
    ez = (K + 2) * U32 * (xd.abs() @ wd.abs().t() + (b.double().abs() if bias else 0))
    _within(pre, z, HALF * z.abs() + MORE * ez + 1e-30, "pre")
    a, _ = _act64(z, act)
    if act == "swiglu":
        (zg, zu), (eg, eu) = z.chunk(2, -1), ez.chunk(2, -1)
        ea = 1.1 * eg * zu.abs() + (zg * torch.sigmoid(zg)).abs() * eu + 2.0 ** -18 * (2 + zg.abs()) * zu.abs()
    else:
        ea = 1.13 * ez + (2.0 ** -18 * (2 + z.abs()) if act != "none" else 0)
    ref = a + (r.double() if residual else 0)
    _within(y, ref, HALF * ref.abs() + MORE * ea + U32 * (a.abs() + ref.abs()) + 1e-30, "y")
    assert U.ulysses_read_error() == 0


@pytest.mark.parametrize("T,K,N,act,bias,residual", LINEAR)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_backward(T, K, N, act, bias, residual, dtype):
    g = _gen(2 * T + K + N)
    nz = 2 * N if act == "swiglu" else N
    x, w, dy = _rnd(g, T, K), _rnd(g, nz, K, scale=K ** -0.5), _rnd(g, T, N)
    pre = _rnd(g, T, nz, scale=1.5) if act != "none" else None
    dx, dw, db = U.ulysses_linear_bwd(x, w, dy, pre=pre, activation=ACTS[act], bias_grad=bias, grad_dtype=dtype)
    again = U.ulysses_linear_bwd(x, w, dy, pre=pre, activation=ACTS[act], bias_grad=bias, grad_dtype=dtype)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and dw.dtype == dtype
    dyd, xd, wd = dy.double(), x.double(), w.double()
    if act == "none":
        dz, e32 = dyd, torch.zeros_like(dyd)
        edz = e32
    else:
        z = pre.double()
        _, d = _act64(z, act)
        if act == "swiglu":
            a, u = z.chunk(2, -1)
            dz = torch.cat([dyd, dyd], -1) * d
            f = 2.0 ** -18 * (2 + a.abs()) * dyd.abs()
            e32 = torch.cat([f * u.abs(), f], -1)
        else:
            dz, e32 = dyd * d, 2.0 ** -18 * (2 + z.abs()) * dyd.abs()
        edz = HALF * dz.abs() + e32
    ref = dz @ wd
    _within(dx, ref, HALF * ref.abs() + MORE * ((edz + nz * U32 * dz.abs()) @ wd.abs()) + 1e-30, "dx")
    ref = dz.t() @ xd
    bound = MORE * ((edz + T * U32 * dz.abs()).t() @ xd.abs()) + 1e-30
    _within(dw, ref, bound + (HALF * ref.abs() if dtype == torch.bfloat16 else 0), "dw")
    if bias:
        assert torch.equal(db, again[2])
        _within(db, dz.sum(0), MORE * (e32 + T * U32 * dz.abs()).sum(0) + 1e-30, "dbias")
    assert U.ulysses_read_error() == 0


def test_linear_gradient_against_differences():
    """dx along a direction against the forward's own differences, in fp32 steps
    wide enough for bf16 inputs: y is linear in x, so the difference is exact but
    for the roundings of the two forwards (2^-8 |y| each)."""
    g = _gen(5)
    T, K, N = 64, 256, 128
    x, w, dy, v = _rnd(g, T, K), _rnd(g, N, K, scale=K ** -0.5), _rnd(g, T, N), _rnd(g, T, K)
    dx, _, _ = U.ulysses_linear_bwd(x, w, dy)
    lo, hi = (x.float() - v.float()).bfloat16(), (x.float() + v.float()).bfloat16()
    y0, y1 = U.ulysses_linear(lo, w).double(), U.ulysses_linear(hi, w).double()
    want = ((y1 - y0) * dy.double()).sum()
    have = (dx.double() * (hi.double() - lo.double())).sum()
    slack = (HALF * (y0.abs() + y1.abs()) * dy.double().abs()).sum() + \
        (HALF * dx.double().abs() * (hi.double() - lo.double()).abs()).sum()
    assert abs(want - have) <= slack
    # and of a sum over many entries the roundings largely cancel: their spread is sqrt(count) of one
    assert abs(want - have) <= slack / math.sqrt(T) + 1.0


def test_linear_activation_limits():
    """Large, infinite and tiny products: the exponentials overflow to 0 or 1, never to NaN."""
    w = torch.eye(8, device="cuda", dtype=torch.bfloat16)
    v = torch.tensor([0.0, -0.0, 1e-30, -1e30, 1e30, -200.0, 200.0, 3e38], device="cuda").bfloat16()
    x = torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16)
    x[range(8), range(8)] = v
    for act in ("gelu", "silu"):
        y = U.ulysses_linear(x, w, activation=ACTS[act])
        want = torch.where(v > 0, v, torch.zeros_like(v))
        want[2] = (v[2].float() * 0.5).bfloat16()
        assert torch.equal(y.diagonal(), want), (act, y.diagonal())
        dx, _, _ = U.ulysses_linear_bwd(x, w, torch.ones_like(x), pre=x.clone(), activation=ACTS[act])
        slope = torch.tensor([0.5, 0.5, 0.5, 0, 1, 0, 1, 1], device="cuda").bfloat16()
        assert torch.equal(dx.diagonal(), slope), (act, dx.diagonal())
    assert U.ulysses_read_error() == 0


def test_linear_in_place_leading_dims_and_guards():
    """residual may be y; the seq layout's dims are kept; nothing behind the last row is written."""
    g = _gen(9)
    P, B, s, K, N = 2, 3, 37, 128, 264
    x, w = _rnd(g, P, B, s, K), _rnd(g, N, K, scale=K ** -0.5)
    buf = _rnd(g, P * B * s + 5, N)
    before = buf.clone()
    y = buf[:P * B * s].view(P, B, s, N)
    want = U.ulysses_linear(x, w, residual=before[:P * B * s].view(P, B, s, N))
    got = U.ulysses_linear(x, w, residual=y, y=y)
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)
    assert torch.equal(buf[P * B * s:], before[P * B * s:])
    T = P * B * s
    dxb = _rnd(g, T + 3, K)
    keep = dxb.clone()
    U.ulysses_linear_bwd(x.view(T, K), w, before[:T], dx=dxb[:T])
    assert torch.equal(dxb[T:], keep[T:])


def test_linear_no_tokens():
    x, w = torch.empty(0, 64, device="cuda").bfloat16(), torch.ones(16, 64, device="cuda").bfloat16()
    assert U.ulysses_linear(x, w).shape == (0, 16)
    dx, dw, db = U.ulysses_linear_bwd(x, w, torch.empty(0, 16, device="cuda").bfloat16(), bias_grad=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


# ------------------------------------------------------------ residual norm

def _rms64(v, w, eps):
    i = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * i * (1 if w is None else w), i


def _norm_inputs(g, P, B, s, D, dtype, gate, post):
    shape = (P, B, s, D)
    mk = lambda *sh, **kw: _rnd(g, *sh, dtype=dtype, **kw)
    gates = {"none": None, "channel": (D,), "sequence": (B, D), "token": shape}[gate]
    return dict(x=mk(*shape), h=mk(*shape, scale=2.0), w_post=mk(D, scale=0.2, mean=1.0) if post else None,
                w_pre=mk(D, scale=0.2, mean=1.0), gate=None if gates is None else mk(*gates, scale=0.7))


def _gate64(gate, mode):
    if gate is None:
        return 1.0
    return gate.double()[:, None, :] if mode == "sequence" else gate.double()


MODES = {"none": U.GATE_NONE, "channel": U.GATE_CHANNEL, "sequence": U.GATE_SEQUENCE, "token": U.GATE_TOKEN}
NORMS = [  # P, B, s, D, dtype, gate, post
    (1, 1, 1, 2560, torch.bfloat16, "channel", True),
    (1, 1, 1, 8, torch.bfloat16, "none", False),           # one vector
    (2, 3, 5, 72, torch.bfloat16, "sequence", True),       # a few lanes of a warp, several rows a CTA
    (3, 2, 7, 1028, torch.float32, "token", True),
    (2, 2, 33, 520, torch.float32, "sequence", False),
    (4, 1, 150, 2560, torch.bfloat16, "token", True),
    (1, 2, 40, 4104, torch.bfloat16, "channel", True),     # the last threads' vectors absent
    (1, 1, 9, 12288, torch.bfloat16, "sequence", True),
    (1, 2, 3, 8192, torch.float32, "channel", True),       # the widest rows
    (2, 1, 150, 16384, torch.bfloat16, "none", True),
    (1, 1, 155, 16384, torch.bfloat16, "token", True),     # one stage only
    (1, 700, 2, 64, torch.bfloat16, "sequence", True),     # more sequences than CTAs in flight
    (3, 2, 701, 256, torch.bfloat16, "channel", True),     # several rows a group, its ring refilled
    (2, 3, 611, 2560, torch.bfloat16, "sequence", True),
    (2, 3, 500, 160, torch.bfloat16, "sequence", True),    # short rows, several a warp, runs that end inside one
    (1, 1, 5000, 8, torch.bfloat16, "channel", True),
    (2, 2, 777, 24, torch.float32, "token", True),
    (1, 3, 1999, 204, torch.float32, "sequence", True),
    (2, 2, 450, 1280, torch.bfloat16, "token", False),
    (1, 1, 1801, 1028, torch.float32, "none", True),
    (1, 2, 611, 640, torch.float32, "channel", True),
]


@pytest.mark.parametrize("P,B,s,D,dtype,gate,post", NORMS)
def test_residual_norm_forward(P, B, s, D, dtype, gate, post):
    a, eps = 0.75, 1e-6
    t = _norm_inputs(_gen(B * s + D), P, B, s, D, dtype, gate, post)
    r, u = U.ulysses_residual_norm(t["x"], t["h"], w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"],
                                   gate_mode=MODES[gate], res_scale=a, eps=eps)
    half = HALF if dtype == torch.bfloat16 else 2.0 ** -24
    esum = (D / 2 + 8) * 2.0 ** -24
    branch = t["h"].double() if not post else _rms64(t["h"].double(), t["w_post"].double(), eps)[0]
    branch = branch * _gate64(t["gate"], gate)
    ref = a * t["x"].double() + branch
    er = (esum if post else 0) * branch.abs() + 4 * U32 * (branch.abs() + (a * t["x"].double()).abs())
    _within(r, ref, half * ref.abs() + MORE * er + 1e-30, "r")
    wp = t["w_pre"].double()
    un, i = _rms64(ref, wp, eps)
    # the mean square moves with r: by 2 sum |r| er / D, relative to itself
    em = (ref.abs() * er).mean(-1, keepdim=True) * i * i
    eu = er * i * wp.abs() + (esum + em + 4 * U32) * un.abs()
    _within(u, un, half * un.abs() + MORE * eu + 1e-30, "u")


@pytest.mark.parametrize("P,B,s,D,dtype,gate,post", NORMS)
def test_residual_norm_backward(P, B, s, D, dtype, gate, post):
    a, eps = 0.75, 1e-6
    g = _gen(3 * B * s + D)
    t = _norm_inputs(g, P, B, s, D, dtype, gate, post)
    r, dr, du = (_rnd(g, P, B, s, D, dtype=dtype) for _ in range(3))
    kw = dict(dr=dr, du=du, w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], gate_mode=MODES[gate], res_scale=a,
              eps=eps)
    got = U.ulysses_residual_norm_bwd(r, t["h"], **kw)
    again = U.ulysses_residual_norm_bwd(r, t["h"], **kw)
    assert all((p is None) == (q is None) and (p is None or torch.equal(p, q)) for p, q in zip(got, again))
    dx, dh, dw_pre, dw_post, dgate = got
    # the formula's gradient, by differentiating the definition in 64 bits
    leaf = {k: v.double().requires_grad_() for k, v in t.items() if v is not None and k != "x"}
    rr = r.double().requires_grad_()
    u, i = _rms64(rr, leaf["w_pre"], eps)
    gr, gw = torch.autograd.grad((u * du.double()).sum() + (rr * dr.double()).sum(), [rr, leaf["w_pre"]])
    n, ih = (leaf["h"], torch.ones(1, device="cuda").double()) if not post else _rms64(leaf["h"], leaf["w_post"], eps)
    gate64 = _gate64(leaf.get("gate"), gate)
    names = [k for k in ("h", "w_post", "gate") if k in leaf]
    grads = dict(zip(names, torch.autograd.grad((n * gate64 * gr).sum(), [leaf[k] for k in names])))
    half = HALF if dtype == torch.bfloat16 else 2.0 ** -24
    e = (2 * D + 32) * 2.0 ** -24          # a row's two sums and the few products behind them
    with torch.no_grad():
        aw = (du.double() * t["w_pre"].double()).abs()
        rn = (rr * i).abs()
        m1 = dr.double().abs() + i * (aw + rn * (aw * rn).mean(-1, keepdim=True))      # sum of |terms| of dR
        _within(dx, a * gr, half * (a * gr).abs() + e * a * m1 + 1e-30, "dx")
        T = P * B * s
        es = e + (T + 8) * 2.0 ** -24
        _within(dw_pre, gw, es * (du.double().abs() * rn).sum((0, 1, 2)) + 1e-30, "dw_pre")
        g64 = gate64.abs() if gate != "none" else 1.0
        if post:
            wp, hn = t["w_post"].double().abs(), (leaf["h"] * ih).abs()
            b = m1 * g64 * wp
            mh = ih * (b + hn * (b * hn).mean(-1, keepdim=True))
            _within(dw_post, grads["w_post"], 2 * es * (m1 * g64 * hn).sum((0, 1, 2)) + 1e-30, "dw_post")
        else:
            mh = m1 * g64
            assert dw_post is None
        _within(dh, grads["h"], half * grads["h"].abs() + 2 * e * mh + 1e-30, "dh")
        if gate == "none":
            assert dgate is None
        else:
            mg = m1 * n.abs()
            if gate == "token":
                _within(dgate, grads["gate"], half * grads["gate"].abs() + 2 * e * mg + 1e-30, "dgate")
            else:
                mg = mg.sum((0, 2)) if gate == "sequence" else mg.sum((0, 1, 2))
                _within(dgate, grads["gate"], 2 * es * mg + 1e-30, "dgate")


def test_residual_norm_partial_calls():
    """The first block (no branch), a branch without a following norm, and gradients of one side only."""
    g = _gen(77)
    P, B, s, D = 2, 1, 19, 256
    x, h, w = _rnd(g, P, B, s, D), _rnd(g, P, B, s, D), _rnd(g, D, mean=1.0, scale=0.1)
    r, u = U.ulysses_residual_norm(x, w_pre=w)
    assert r is None
    want, _ = _rms64(x.double(), w.double(), 1e-6)
    _within(u, want, (HALF + 1e-4) * want.abs() + 1e-30, "first norm")
    r2, u2 = U.ulysses_residual_norm(x, w_pre=w, r=torch.empty_like(x))
    assert torch.equal(r2, x) and torch.equal(u2, u)
    r3, none = U.ulysses_residual_norm(x, h)
    assert none is None and torch.equal(r3, (x.float() + h.float()).bfloat16())
    dr = _rnd(g, P, B, s, D)
    dx, dh, dw_pre, dw_post, dgate = U.ulysses_residual_norm_bwd(x, h, dr=dr)
    assert torch.equal(dx, dr) and torch.equal(dh, dr) and dw_pre is None and dw_post is None and dgate is None
    both = U.ulysses_residual_norm_bwd(x, du=dr, w_pre=w)
    zero = U.ulysses_residual_norm_bwd(x, du=dr, dr=torch.zeros_like(dr), w_pre=w)
    assert torch.equal(both[0], zero[0]) and torch.equal(both[2], zero[2]) and both[1] is None
    # in place: r over x or h, u over h
    want_r, want_u = U.ulysses_residual_norm(x, h, w_pre=w)
    for target in ("x", "h"):
        xc, hc = x.clone(), h.clone()
        rr, uu = U.ulysses_residual_norm(xc, hc, w_pre=w, r=xc if target == "x" else hc,
                                         u=hc if target == "x" else None)
        assert torch.equal(rr, want_r) and torch.equal(uu, want_u)
    drc = dr.clone()
    want_b = U.ulysses_residual_norm_bwd(x, h, dr=dr, du=h, w_pre=w)
    got_b = U.ulysses_residual_norm_bwd(x, h, dr=drc, du=h, w_pre=w, dx=drc)
    assert torch.equal(want_b[0], got_b[0]) and torch.equal(want_b[1], got_b[1])


# -------------------------------------------------------------- linear loss

def _loss64(x, w, y, P, ignore):
    z = x.double() @ w.double().t()
    keep = (y != ignore) & (y >= 0) & (y < w.shape[0])
    at = torch.where(keep, y, torch.zeros_like(y)).long()[:, None]
    lse = torch.logsumexp(z, 1)
    per = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    C = keep.sum()
    dz = torch.exp(z - lse[:, None]).scatter_add(1, at, -torch.ones_like(lse)[:, None])
    dz = torch.where(keep[:, None], dz / C, torch.zeros_like(dz))
    return per.view(P, -1).sum(1), keep.view(P, -1).sum(1), per.sum() / C, dz


LOSSES = [  # P, T, D, V, spread of the logits, ignored share, piece
    (1, 1, 64, 100, 1.0, 0.0, 0),
    (1, 3, 8, 1, 1.0, 0.0, 0),                 # a vocabulary of one: loss 0, gradient 0
    (4, 256, 128, 8192, 1.0, 0.2, 0),
    (3, 303, 136, 1003, 3.0, 0.5, 0),          # odd vocabulary, ragged rows
    (2, 1100, 256, 513, 1.0, 0.1, 256),        # five pieces, the last one short
    (2, 514, 64, 2049, 2.0, 0.0, 257),         # pieces that end inside a tile
    (2, 1026, 72, 4099, 2.0, 0.3, 1024),       # a last piece of two rows
    (11, 319, 64, 300, 1.0, 0.2, 0),           # more shards than are summed in one go
    (5, 16395, 8, 40, 1.0, 0.2, 0),            # more tokens than are
    (7, 63, 64, 300, 1.0, 0.2, 0),
    (1, 130, 64, 3000, 60.0, 0.0, 0),          # logits hundreds apart
]


@pytest.mark.parametrize("P,T,D,V,spread,ignored,piece", LOSSES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_loss(P, T, D, V, spread, ignored, piece, dtype):
    g = _gen(T + V)
    x, w = _rnd(g, T, D), _rnd(g, V, D, scale=spread * D ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[torch.rand(T, generator=g, device="cuda") < ignored] = -100
    y[0] = V - 1
    S, C, L = U.ulysses_linear_loss(x, w, y, P)
    S2, C2, L2, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, P, grad_dtype=dtype, piece_tokens=piece)
    again = U.ulysses_linear_loss_bwd(x, w, y, P, grad_dtype=dtype, piece_tokens=piece)
    assert all(torch.equal(p, q) for p, q in zip((S2, C2, L2, dx, dw), again))
    Sr, Cr, Lr, dz = _loss64(x, w, y, P, -100)
    ez = D * U32 * (x.double().abs() @ w.double().abs().t()).amax(1, keepdim=True)   # one logit's error
    es = 2 * ez.max() * Cr.max()
    for a, b, c in ((S, C, L), (S2, C2, L2)):
        assert torch.equal(b, Cr)
        assert ((a.double() - Sr).abs() <= LOSS_REL * Sr.abs() + es + 1e-30).all()
        assert abs(c.double() - Lr) <= LOSS_REL * Lr.abs() + 2 * ez.max() + 1e-30
    xd, wd = x.double().abs(), w.double().abs()
    soft = dz.abs()
    ref = dz @ w.double()
    _within(dx, ref, HALF * ref.abs() + MORE * (((HALF + 2.0 ** -11 + 2 * ez + V * U32) * soft) @ wd) + 1e-12, "dx")
    ref = dz.t() @ x.double()
    bound = MORE * (((HALF + 2.0 ** -11 + 2 * ez + T * U32) * soft).t() @ xd) + 1e-12
    _within(dw, ref, bound + (HALF * ref.abs() if dtype == torch.bfloat16 else 0), "dw")
    assert U.ulysses_read_error() == 0


def test_linear_loss_agrees_with_the_loss_from_logits():
    """The same labels through ulysses_linear and ulysses_loss_aggregate: the
    logits are rounded to bf16 there, 2^-8 of the largest at most."""
    g = _gen(21)
    P, T, D, V = 4, 512, 256, 4096
    x, w = _rnd(g, T, D), _rnd(g, V, D, scale=D ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[::9] = -100
    logits = U.ulysses_linear(x, w)
    S, C, L = U.ulysses_loss_aggregate(logits, y, P)
    S2, C2, L2 = U.ulysses_linear_loss(x, w, y, P)
    assert torch.equal(C, C2)
    assert abs(L.item() - L2.item()) <= 2 * HALF * logits.abs().max().item()


def test_linear_loss_ignored_rows_and_bad_labels():
    """Rows that do not count may hold NaN and infinities; a label outside the
    vocabulary is reported and not counted; no counted token: NaN and zeros."""
    g = _gen(31)
    P, T, D, V = 2, 300, 64, 700
    x, w = _rnd(g, T, D), _rnd(g, V, D, scale=0.3)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    clean = x.clone()
    y[5:150:3] = -100
    clean[5:150:3] = 0
    x[5:150:6] = float("nan")
    x[8:150:6] = float("inf")
    want = U.ulysses_linear_loss_bwd(clean, w, y, P)
    got = U.ulysses_linear_loss_bwd(x, w, y, P)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    assert not got[3][5:150:3].any()
    assert U.ulysses_read_error() == 0
    y[7], y[8] = V, -3
    S, C, L, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, P)
    assert C.sum().item() == (((y >= 0) & (y < V)).sum()).item() and not dx[7:9].any()
    assert U.ulysses_read_error() == 1 << 8
    U.ulysses_linear_loss(x, w, y, P)
    assert U.ulysses_read_error() == 1 << 8
    y.fill_(-100)
    S, C, L, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, P)
    assert torch.isnan(L).all() and not C.any() and not S.any() and not dx.any() and not dw.any()
    e = U.ulysses_linear_loss_bwd(x[:0], w, y[:0], P)
    assert torch.isnan(e[2]).all() and not e[1].any() and not e[4].any()


def test_linear_loss_masked_vocabulary():
    """Columns of the vocabulary at -inf or at the type's lowest value get no weight and no gradient."""
    g = _gen(41)
    T, D, V = 64, 64, 900
    x = _rnd(g, T, D).abs() + 0.125          # positive, so that w's sign decides the logit's
    w = _rnd(g, V, D, scale=0.2)
    dead = torch.zeros(V, dtype=torch.bool, device="cuda")
    dead[:300] = True                        # the whole of the first columns among them
    dead[850:] = True
    w[dead] = -1e30
    y = torch.randint(300, 850, (T,), generator=g, device="cuda", dtype=torch.int32)
    S, C, L, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, 1)
    Sr, Cr, Lr, dz = _loss64(x, w[300:850], y - 300, 1, -100)
    assert abs(L.double() - Lr) <= 1e-4 * Lr
    assert not dw[dead].any()
    ref = dz @ w[300:850].double()
    bound = HALF * ref.abs() + MORE * (((HALF + 2.0 ** -11 + 2e-4 + V * U32) * dz.abs()) @ w[300:850].double().abs()) + 1e-12
    _within(dx, ref, bound, "dx")


# ------------------------------------------------------ streams, graphs, run

def _block(x, p, P):
    """A feed-forward block and the loss behind it, forward and backward."""
    lead = x.shape[:-1]
    _, u = U.ulysses_residual_norm(x, w_pre=p["n1"])
    f, zf = U.ulysses_linear(u, p["w1"], activation=U.ACT_SWIGLU, save_pre=True)
    h, _ = U.ulysses_linear(f, p["w2"], bias=p["b2"], save_pre=True)
    r, v = U.ulysses_residual_norm(x, h, w_pre=p["n3"], w_post=p["n2"], gate=p["gate"], gate_mode=U.GATE_SEQUENCE,
                                   res_scale=0.9)
    flat = v.view(-1, v.shape[-1])
    S, C, L, dv, dhead = U.ulysses_linear_loss_bwd(flat, p["head"], p["labels"], P)
    dxr, dh, dn3, dn2, dgate = U.ulysses_residual_norm_bwd(r, h, du=dv.view(v.shape), w_pre=p["n3"], w_post=p["n2"],
                                                           gate=p["gate"], gate_mode=U.GATE_SEQUENCE, res_scale=0.9)
    df, dw2, db2 = U.ulysses_linear_bwd(f, p["w2"], dh, bias_grad=True)
    du, dw1, _ = U.ulysses_linear_bwd(u, p["w1"], df, pre=zf, activation=U.ACT_SWIGLU)
    dx, _, dn1, _, _ = U.ulysses_residual_norm_bwd(x, dr=dxr, du=du, w_pre=p["n1"])
    assert dx.shape == (*lead, x.shape[-1])
    return dict(L=L, x=dx, w1=dw1, w2=dw2, b2=db2, n1=dn1, n2=dn2, n3=dn3, gate=dgate, head=dhead)


def _block_inputs(g, P, B, s, D, N, V):
    p = dict(n1=_rnd(g, D, mean=1.0, scale=0.1), n2=_rnd(g, D, mean=1.0, scale=0.1),
             n3=_rnd(g, D, mean=1.0, scale=0.1), gate=_rnd(g, B, D), w1=_rnd(g, 2 * N, D, scale=D ** -0.5),
             w2=_rnd(g, D, N, scale=N ** -0.5), b2=_rnd(g, D, scale=0.1), head=_rnd(g, V, D, scale=D ** -0.5))
    p["labels"] = torch.randint(0, V, (P * B * s,), generator=g, device="cuda", dtype=torch.int32)
    p["labels"][::7] = -100
    return _rnd(g, P, B, s, D), p


def test_a_block_and_its_loss_together():
    """The operators as a training step runs them, against 64-bit automatic
    differentiation of the whole chain.  Each gradient passes at most eight
    bf16 roundings (activations and gradients between the operators, operands
    inside them); one is uniform within half a step, 2^-8 / sqrt(3) relative L2;
    eight of them, even all in line, stay below 2e-2."""
    P, B, s, D, N, V = 2, 2, 75, 256, 320, 1000
    x, p = _block_inputs(_gen(51), P, B, s, D, N, V)
    got = _block(x, p, P)
    q = {k: v.double().requires_grad_() for k, v in p.items() if k != "labels"}
    xd = x.double().requires_grad_()
    u, _ = _rms64(xd, q["n1"], 1e-6)
    a, b = (u @ q["w1"].t()).chunk(2, -1)
    h = (a * torch.sigmoid(a) * b) @ q["w2"].t() + q["b2"]
    r = 0.9 * xd + q["gate"][:, None, :] * _rms64(h, q["n2"], 1e-6)[0]
    v, _ = _rms64(r, q["n3"], 1e-6)
    L = torch.nn.functional.cross_entropy((v @ q["head"].t()).view(-1, V), p["labels"].long(), ignore_index=-100)
    names = [k for k in got if k not in ("L", "x")]
    grads = torch.autograd.grad(L, [xd] + [q[k] for k in names])
    assert abs(got["L"].item() - L.item()) <= 2e-2 * L.item()
    for k, ref in zip(["x"] + names, grads):
        rel = ((got[k].double() - ref).norm() / ref.norm()).item()
        assert rel <= 2e-2, f"{k}: relative L2 {rel:.3e}"
    assert U.ulysses_read_error() == 0


def test_block_on_another_stream_and_in_a_graph():
    """The same bits on a side stream, in a captured graph replayed on new
    inputs, and in two graphs replayed in turn."""
    P, B, s, D, N, V = 2, 1, 60, 128, 136, 600
    xa, p = _block_inputs(_gen(61), P, B, s, D, N, V)
    xb = _rnd(_gen(62), P, B, s, D)
    want = [_block(v, p, P) for v in (xa, xb)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _block(xa, p, P)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(want[0][k], got[k]) for k in got)
    x = xa.clone()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, _block(x, p, P)))
    for src, ref in ((xb, want[1]), (xa, want[0])):
        x.copy_(src)
        for gr, out in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(ref[k], out[k]) for k in ref)
    # an explicit stream argument, two calls at once on two streams with workspaces of their own
    w = p["head"]
    flat = xa.view(-1, D)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a = U.ulysses_linear_loss_bwd(flat, w, p["labels"], P, stream=s1)
    b = U.ulysses_linear_loss_bwd(flat, w, p["labels"], P, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(i, j) for i, j in zip(a, b))
    assert U.ulysses_read_error() == 0


def test_products_report_a_wait_that_ran_out():
    """A pipeline wait cut short is reported in the error word, the launch ends
    and frees its tensor memory: the next call is right again."""
    g = _gen(71)
    calls = []
    for T, K, N in ((600, 512, 512), (9, 2048, 256)):        # a pair of CTAs a tile; the clusters for few tokens
        x, w = _rnd(g, T, K), _rnd(g, N, K, scale=K ** -0.5)
        calls.append((x, w, U.ulysses_linear(x, w)))
    torch.cuda.synchronize()
    for x, w, want in calls:
        assert U.lib().ulysses_set_wait_limit(300) == 0
        try:
            U.ulysses_linear(x, w)
            torch.cuda.synchronize()
        finally:
            U.lib().ulysses_set_wait_limit(0)
        assert U.ulysses_read_error() & (1 << 9)
        assert torch.equal(U.ulysses_linear(x, w), want)
        assert U.ulysses_read_error() == 0


@pytest.mark.parametrize("op", ["linear", "norm", "loss"])
def test_first_call_of_a_process_may_be_captured(op):
    """Nothing an operator sets up on its first call is forbidden in a capture."""
    code = f"""
import torch
from long_context_sequence_all_b200 import ulysses as U
torch.cuda.init()
m = lambda *s: torch.ones(*s, device="cuda", dtype=torch.bfloat16)
x, w, y = m(300, 64), m(512, 64), torch.zeros(300, device="cuda", dtype=torch.int32)
q, v = m(1, 1, 300, 64), m(64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    if "{op}" == "linear":
        out = U.ulysses_linear(x, w)
        back = U.ulysses_linear_bwd(x, w, out)
    elif "{op}" == "norm":
        out, _ = U.ulysses_residual_norm(q, q, w_pre=v)
        back = U.ulysses_residual_norm_bwd(q, q, du=q, w_pre=v)
    else:
        out = U.ulysses_linear_loss(x, w, y, 2)[2]
        back = U.ulysses_linear_loss_bwd(x, w, y, 2)
g.replay()
torch.cuda.synchronize()
want = {{"linear": 64.0, "norm": 2.0}}.get("{op}")
print(out.flatten()[0].item())
assert want is None or out.flatten()[0].item() == want
assert want is not None or abs(out.item() - 6.238325) < 1e-4      # log(512): all logits equal
assert U.ulysses_read_error() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


# ------------------------------------------- tiles, parts and folds at their edges

@pytest.mark.parametrize("T,K,N,act,bias,residual", [
    (300, 64, 72, "swiglu", True, True),        # narrow gated tiles, the last one of 8 features
    (2050, 64, 1000, "swiglu", False, True),    # wide ones, a residual that ends inside the last
    (700, 72, 200, "none", True, True),
    (5000, 128, 2600, "gelu", True, True),      # the residual asked for a tile ahead, several tiles an SM pair
    (4099, 8, 4104, "silu", False, True),       # one k-step a tile
    (1, 8, 40000, "none", True, False),         # dx of few tokens over a long sum, cut over the SM pairs
    (17, 72, 30000, "gelu", True, False),
    (128, 200, 20000, "silu", False, False),
    (390, 72, 808, "gelu", True, False),        # dz of few tokens in strips of two rows
    (20000, 16, 72, "none", True, False),       # a bias gradient of many partials and few columns
])
def test_linear_at_the_edges(T, K, N, act, bias, residual):
    test_linear_forward(T, K, N, act, bias, residual)
    test_linear_backward(T, K, N, act, bias, residual, torch.float32)


@pytest.mark.parametrize("P,T,D,V", [(1, 1, 136, 50001), (3, 33, 72, 30011), (8, 128, 72, 20000), (2, 1502, 72, 4003),
                                     (8, 16384, 8, 72), (1, 700, 1000, 264)])
def test_linear_loss_at_the_edges(P, T, D, V):
    test_linear_loss(P, T, D, V, 1.0, 0.2, 0, torch.bfloat16)


@pytest.mark.parametrize("P,B,s,D,gate", [(1, 1, 30000, 64, "channel"), (2, 3, 5000, 64, "sequence"), (1, 2, 9000, 512, "channel")])
def test_residual_norm_of_many_short_rows(P, B, s, D, gate):
    test_residual_norm_backward(P, B, s, D, torch.bfloat16, gate, True)


@pytest.mark.parametrize("tokens", [48, 300])
def test_linear_loss_count_is_no_rounding(tokens):
    """w = 0: softmax = 1/V.  A label's dz, 1/V - 1, rounds to -1 (off by 1/V), the
    others', 1/V, are off by half a step (2^-8 of themselves) and 2^-11; 1/C, no
    power of two, is applied in fp32 (two roundings) and is no part of it."""
    V, D = 65536, 64
    w = torch.zeros(V, D, device="cuda", dtype=torch.bfloat16)
    x = torch.ones(tokens, D, device="cuda", dtype=torch.bfloat16)
    y = (torch.arange(tokens, device="cuda", dtype=torch.int32) * 211) % V
    _, _, loss, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, 1, grad_dtype=torch.float32)
    ref = torch.full((V, D), 1.0 / V, device="cuda", dtype=torch.float64)
    ref[y.long()] -= 1.0 / tokens
    bound = (1 + tokens * (HALF + 2.0 ** -11)) / V / tokens + 2 * U32 * ref.abs()
    _within(dw, ref, MORE * bound, "dw")
    assert not dx.any() and abs(loss.item() - math.log(V)) <= 4 * U32 * math.log(V)


def test_linear_loss_does_not_read_what_it_padded():
    """Scratch rows are longer than the vocabulary and the hidden size: what lies behind is NaN and not used."""
    g = _gen(90)
    for T, D, V in ((20, 72, 1001), (300, 72, 1001)):
        x, w = _rnd(g, T, D), _rnd(g, V, D, scale=D ** -0.5)
        y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        n = U.ulysses_linear_loss_bwd_workspace_size(1, T, D, V, torch.float32)
        got = []
        for fill in (0, 255):   # bytes 255: NaN in every type
            ws = torch.full((n,), fill, device="cuda", dtype=torch.uint8)
            got.append(U.ulysses_linear_loss_bwd(x, w, y, 1, workspace=ws))
        assert all(torch.equal(a, b) for a, b in zip(*got)) and torch.isfinite(got[1][4]).all()
    T, K, N = 300, 72, 136
    x, w, dy, pre = _rnd(g, T, K), _rnd(g, N, K), _rnd(g, T, N), _rnd(g, T, N)
    n = U.ulysses_linear_bwd_workspace_size(T, K, N, U.ACT_GELU)
    a, b = (U.ulysses_linear_bwd(x, w, dy, pre=pre, activation=U.ACT_GELU, bias_grad=True,
                                 workspace=torch.full((n,), f, device="cuda", dtype=torch.uint8)) for f in (0, 255))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("P,T,D,V", [(1, 1, 64, 1003), (3, 3, 64, 20001), (1, 5, 72, 300), (8, 16, 64, 5000), (7, 28, 72, 2049),
                                     (1, 33, 64, 1003), (2, 64, 128, 4099), (1, 65, 64, 1003), (9, 63, 64, 777)])
def test_linear_loss_of_few_tokens(P, T, D, V):
    test_linear_loss(P, T, D, V, 1.0, 0.3, 0, torch.float32)


@pytest.mark.parametrize("P,T,D,V", [(1, 100, 1000, 1103), (3, 33, 2560, 5000), (8, 128, 648, 300), (1, 12, 2536, 1103),
                                     (2, 66, 4096, 100), (1, 1, 4096, 130)])
def test_linear_loss_of_tiles_shared_by_clusters(P, T, D, V):
    test_linear_loss(P, T, D, V, 1.0, 0.3, 0, torch.float32)


# ------------------------------------------------------ offsets past 32 bits

def test_linear_past_32_bit_offsets():
    """2.5e9 elements in y, pre, residual and dz: the first, middle and last rows, and the sums over all."""
    g = _gen(101)
    T, K, N = 600001, 64, 4096
    x, w, b = _rnd(g, T, K), _rnd(g, N, K, scale=K ** -0.5), _rnd(g, N, scale=0.5)
    r = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    for t in range(0, T, 65536):
        r[t:t + 65536] = _rnd(g, min(65536, T - t), N)
    y, pre = U.ulysses_linear(x, w, bias=b, residual=r, activation=U.ACT_GELU, save_pre=True)
    dx, dw, db = U.ulysses_linear_bwd(x, w, r, pre=pre, activation=U.ACT_GELU, bias_grad=True)
    wd = w.double()
    dw_ref, dw_bound = (torch.zeros(N, K, device="cuda", dtype=torch.float64) for _ in range(2))
    db_ref, db_bound = (torch.zeros(N, device="cuda", dtype=torch.float64) for _ in range(2))
    for t in range(0, T, 40000):
        at = slice(t, min(t + 40000, T))
        xd, rd, zd = x[at].double(), r[at].double(), pre[at].double()
        z = xd @ wd.t() + b.double()
        ez = (K + 2) * U32 * (xd.abs() @ wd.abs().t() + b.double().abs())
        _within(pre[at], z, HALF * z.abs() + MORE * ez + 1e-30, "pre")
        a, _ = _act64(z, "gelu")
        ref = a + rd
        ea = 1.13 * ez + 2.0 ** -18 * (2 + z.abs())
        _within(y[at], ref, HALF * ref.abs() + MORE * ea + U32 * (a.abs() + ref.abs()) + 1e-30, "y")
        _, d = _act64(zd, "gelu")
        dz, e32 = rd * d, 2.0 ** -18 * (2 + zd.abs()) * rd.abs()
        ref = dz @ wd
        _within(dx[at], ref, HALF * ref.abs() + MORE * ((HALF * dz.abs() + e32 + N * U32 * dz.abs()) @ wd.abs()) + 1e-30, "dx")
        dw_ref += dz.t() @ xd
        dw_bound += (HALF * dz.abs() + e32 + T * U32 * dz.abs()).t() @ xd.abs()
        db_ref += dz.sum(0)
        db_bound += (e32 + T * U32 * dz.abs()).sum(0)
    _within(dw, dw_ref, MORE * dw_bound + 1e-30, "dw")
    _within(db, db_ref, MORE * db_bound + 1e-30, "dbias")


def test_residual_norm_past_32_bit_offsets():
    """2.5e9 elements a tensor: every row against 64 bits in pieces, both directions."""
    g = _gen(102)
    P, B, s, D, a, eps = 2, 1, 150001, 8192, 0.75, 1e-6
    mk = lambda: torch.cat([_rnd(g, 1, B, s, D) for _ in range(P)])
    x, h, w1, w2 = mk(), mk(), _rnd(g, D, mean=1.0), _rnd(g, D, mean=1.0)
    r, u = U.ulysses_residual_norm(x, h, w_pre=w1, w_post=w2, res_scale=a, eps=eps)
    dx, dh, dw1, dw2, _ = U.ulysses_residual_norm_bwd(r, h, dr=x, du=h, w_pre=w1, w_post=w2, res_scale=a, eps=eps)
    esum, e = (D / 2 + 8) * 2.0 ** -24, (2 * D + 32) * 2.0 ** -24
    flat = lambda t: t.view(-1, D)
    w1d, w2d = w1.double(), w2.double()
    dw1_ref, dw1_terms, dw2_ref, dw2_terms = (torch.zeros(D, device="cuda", dtype=torch.float64) for _ in range(4))
    for t in range(0, P * s, 20000):
        at = slice(t, min(t + 20000, P * s))
        xd, hd, rd = (flat(v)[at].double() for v in (x, h, r))
        branch, ih = _rms64(hd, w2d, eps)
        ref = a * xd + branch
        er = esum * branch.abs() + 4 * U32 * (branch.abs() + (a * xd).abs())
        _within(flat(r)[at], ref, HALF * ref.abs() + MORE * er + 1e-30, "r")
        un, i = _rms64(ref, w1d, eps)
        em = (ref.abs() * er).mean(-1, keepdim=True) * i * i
        eu = er * i * w1d.abs() + (esum + em + 4 * U32) * un.abs()
        _within(flat(u)[at], un, HALF * un.abs() + MORE * eu + 1e-30, "u")
        # backward, from the stored r, with dr = x and du = h
        rn, i = _rms64(rd, None, eps)
        aw = hd * w1d
        dR = xd + i * (aw - rn * (aw * rn).mean(-1, keepdim=True))
        m1 = xd.abs() + i * (aw.abs() + rn.abs() * (aw * rn).abs().mean(-1, keepdim=True))
        _within(flat(dx)[at], a * dR, HALF * (a * dR).abs() + e * a * m1 + 1e-30, "dx")
        hn, b, bm = hd * ih, dR * w2d, m1 * w2d.abs()
        ref = ih * (b - hn * (b * hn).mean(-1, keepdim=True))
        mh = ih * (bm + hn.abs() * (bm * hn.abs()).mean(-1, keepdim=True))
        _within(flat(dh)[at], ref, HALF * ref.abs() + 2 * e * mh + 1e-30, "dh")
        dw1_ref += (hd * rn).sum(0)
        dw1_terms += (hd * rn).abs().sum(0)
        dw2_ref += (dR * hn).sum(0)
        dw2_terms += (m1 * hn.abs()).sum(0)
    es = e + (P * s + 8) * 2.0 ** -24
    _within(dw1, dw1_ref, es * dw1_terms + 1e-30, "dw_pre")
    _within(dw2, dw2_ref, 2 * es * dw2_terms + 1e-30, "dw_post")


def test_linear_loss_past_32_bit_offsets():
    """2.5e9 logits in one piece, their exponentials in 4.9 GB of the workspace."""
    g = _gen(103)
    T, D, V = 4097, 64, 600011
    x, w = _rnd(g, T, D), _rnd(g, V, D, scale=D ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[::7] = -100
    y[-1] = V - 1
    S, C, L, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, 1, piece_tokens=T)
    assert torch.equal(L, U.ulysses_linear_loss(x, w, y, 1)[2])
    keep = y != -100
    count = int(keep.sum())
    wd, xd = w.double(), x.double()
    ez = D * U32 * (xd.abs().max() * wd.abs().max() * D)   # above every logit's error
    total = 0.0
    dw_ref, dw_bound = (torch.zeros(V, D, device="cuda", dtype=torch.float64) for _ in range(2))
    for t in range(0, T, 500):
        at = slice(t, min(t + 500, T))
        z = xd[at] @ wd.t()
        lse = torch.logsumexp(z, 1)
        idx = torch.where(keep[at], y[at], 0).long()[:, None]
        total += ((lse - z.gather(1, idx)[:, 0]) * keep[at]).sum().item()
        dz = torch.exp_(z.sub_(lse[:, None]))
        dz.scatter_add_(1, idx, -torch.ones_like(idx, dtype=torch.float64))
        dz *= keep[at][:, None] / count
        soft = dz.abs()
        e = HALF + 2.0 ** -11 + 2 * ez
        ref = dz @ wd
        _within(dx[at], ref, HALF * ref.abs() + MORE * (e + V * U32) * (soft @ wd.abs()) + 1e-12, "dx")
        dw_ref += dz.t() @ xd[at]
        dw_bound += (e + T * U32) * (soft.t() @ xd[at].abs())
    assert C.item() == count and abs(L.item() - total / count) <= LOSS_REL * total / count + 2 * ez
    _within(dw, dw_ref, MORE * dw_bound + 1e-12, "dw")


@pytest.mark.parametrize("T,K,N,act,bias,residual", [
    (24, 8200, 264, "none", True, True),        # sixteen CTAs a tile
    (1, 8192, 72, "swiglu", True, True),
    (32, 12288 + 8, 136, "gelu", False, False),
    (33, 8192, 136, "silu", True, True),        # eight again
])
def test_linear_of_few_tokens_over_long_sums(T, K, N, act, bias, residual):
    test_linear_forward(T, K, N, act, bias, residual)
    test_linear_backward(T, N, K, act, bias, residual, torch.float32)   # dx over K


@pytest.mark.parametrize("P,B,s,D,dtype", [(1, 40, 30, 2560, torch.bfloat16), (1, 2000, 8, 512, torch.bfloat16), (2, 17, 1, 72, torch.bfloat16),
                                           (1, 300, 3, 204, torch.float32), (1, 16, 400, 64, torch.bfloat16)])
def test_residual_norm_of_many_sequences(P, B, s, D, dtype):
    test_residual_norm_backward(P, B, s, D, dtype, "sequence", True)


# --------------------------------------- slots of the vocabulary with nothing in them

@pytest.mark.parametrize("shift", [0.0, -250.0])
@pytest.mark.parametrize("fill", [-1e30, torch.finfo(torch.bfloat16).min, float("-inf")])
@pytest.mark.parametrize("T,piece", [(5, 0), (64, 0), (300, 0), (300, 130)])   # either product, whole and in pieces
def test_linear_loss_of_dead_vocabulary_blocks(T, piece, fill, shift):
    """Blocks of 128 columns whose logits are all -inf (the lowest value's sums
    overflow) have no weight and no gradient, also where every other logit of a
    row is far below zero: x's first column is one, w's is the shift.  The live
    columns against 64 bits, with the bounds of test_linear_loss."""
    g = _gen(43)
    D, V, lo, hi = 64, 1400, 300, 850
    x = _rnd(g, T, D).abs() + 0.125          # positive: the sign of w is the logit's
    w = _rnd(g, V, D, scale=0.2)
    x[:, 0], w[:, 0] = 1.0, shift
    dead = torch.ones(V, dtype=torch.bool, device="cuda")
    dead[lo:hi] = False                      # the first two blocks, parts of two, the last four
    w[dead] = fill
    y = torch.randint(lo, hi, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[1::4] = -100
    S, C, L, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, 1, piece_tokens=piece)
    assert torch.equal(U.ulysses_linear_loss(x, w, y, 1)[2], L)
    live, x64 = w[lo:hi], x.double()
    _, Cr, Lr, dz = _loss64(x, live, torch.where(y == -100, y, y - lo), 1, -100)
    ez = D * U32 * (x64 @ live.double().abs().t()).amax(1, keepdim=True)
    assert torch.equal(C, Cr) and abs(L.double() - Lr) <= LOSS_REL * Lr + 2 * ez.max()
    soft = dz.abs()
    assert not dw[dead].any()
    ref = dz.t() @ x64
    _within(dw[lo:hi], ref, MORE * (((HALF + 2.0 ** -11 + 2 * ez + T * U32) * soft).t() @ x64) + 1e-12, "dw")
    if fill != float("-inf"):                # the product's own 0 times infinity is NaN
        ref = dz @ live.double()
        terms = ((HALF + 2.0 ** -11 + 2 * ez + V * U32) * soft) @ live.double().abs()
        _within(dx, ref, HALF * ref.abs() + MORE * terms + 1e-12, "dx")
    assert U.ulysses_read_error() == 0


@pytest.mark.parametrize("T", [1, 70])
def test_linear_loss_keeps_nan(T):
    """A counted token without a softmax (a NaN logit, or every logit -inf) has a NaN loss and NaN
    in the whole of its gradient, the label's element among it."""
    for fill, V in ((float("nan"), 5), (float("nan"), 400), (float("-inf"), 400)):
        x = torch.ones(T, 64, device="cuda", dtype=torch.bfloat16)
        w = torch.full((V, 64), fill, device="cuda", dtype=torch.bfloat16)
        if fill != fill:
            w[1:] = 1.0
        y = torch.full((T,), V - 2, device="cuda", dtype=torch.int32)
        _, C, L, dx, dw = U.ulysses_linear_loss_bwd(x, w, y, 1)
        assert C.item() == T and torch.isnan(L).all() and torch.isnan(dx).all() and torch.isnan(dw).all()
        assert torch.isnan(U.ulysses_linear_loss(x, w, y, 1)[2]).all()


# ----------------------------------------------------- the norms' bounded waits

@pytest.mark.parametrize("P,B,s,D,dtype,gate", [
    (2, 1, 400, 64, torch.bfloat16, "channel"),      # rows that share a warp
    (2, 3, 90, 160, torch.bfloat16, "sequence"),     # the same, brought row by row in the backward
    (1, 1, 700, 2560, torch.bfloat16, "channel"),    # teams of several warps
    (1, 2, 300, 1028, torch.float32, "token"),
    (1, 1, 200, 16384, torch.bfloat16, "none"),      # a CTA a row
    (1, 1, 155, 16384, torch.bfloat16, "token"),     # one stage only
])
def test_residual_norm_reports_a_wait_that_ran_out(P, B, s, D, dtype, gate):
    """A wait for rows cut short is reported in the error word and the launch
    ends, in both directions; the next call is right again.  (Rows that L2 holds
    are there before a thread has sent for the whole ring and first looks.)"""
    g = _gen(81)
    t = _norm_inputs(g, P, B, s, D, dtype, gate, True)
    dr, du = (_rnd(g, P, B, s, D, dtype=dtype) for _ in range(2))
    kw = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], gate_mode=MODES[gate])
    for call in (lambda: U.ulysses_residual_norm(t["x"], t["h"], **kw),
                 lambda: U.ulysses_residual_norm_bwd(t["x"], t["h"], dr=dr, du=du, **kw)):
        want = call()
        torch.empty(1 << 28, device="cuda", dtype=torch.uint8).zero_()     # L2 holds something else
        torch.cuda.synchronize()
        assert U.ulysses_read_error() == 0
        U.ulysses_set_wait_limit(200)                # cycles; rows from memory take thousands
        try:
            call()
            torch.cuda.synchronize()
        finally:
            U.ulysses_set_wait_limit(0)
        info = U.ulysses_read_error_info()
        assert info[0] == 1 << 9 and info[1] == 1 and info[8] >= 1, info[:9]
        again = call()
        torch.cuda.synchronize()
        assert all((p is None) == (q is None) and (p is None or torch.equal(p, q)) for p, q in zip(want, again))
        assert U.ulysses_read_error() == 0


@pytest.mark.parametrize("T,K,N,act,bias", [
    (1, 64, 8, "none", True),              # few tokens
    (24, 8200, 264, "silu", False),        # the same, sixteen CTAs a tile
    (128, 520, 136, "swiglu", True),
    (222, 64, 72, "swiglu", True),         # narrow gated tiles
    (4100, 128, 2600, "gelu", False),      # several tiles an SM pair, the residual a tile ahead
    (600, 4096, 3320, "swiglu", True),     # the last tiles cut along K: joined by a second kernel
    (2300, 8192, 2304, "none", False),
])
def test_linear_residual_in_place(T, K, N, act, bias):
    """The residual may be y itself, in every kernel that adds it."""
    g = _gen(T + N)
    nz = 2 * N if act == "swiglu" else N
    x, w, r = _rnd(g, T, K), _rnd(g, nz, K, scale=K ** -0.5), _rnd(g, T, N)
    b = _rnd(g, nz, scale=0.5) if bias else None
    want = U.ulysses_linear(x, w, bias=b, residual=r, activation=ACTS[act])
    y = r.clone()
    got = U.ulysses_linear(x, w, bias=b, residual=y, activation=ACTS[act], y=y)
    assert got.data_ptr() == y.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("P,B,s,D,dtype,gate", [
    (1, 200, 60, 2560, torch.bfloat16, "sequence"),    # several sequences a CTA, each with its gate
    (2, 300, 100, 1280, torch.bfloat16, "sequence"),
    (1, 300, 20, 1280, torch.bfloat16, "sequence"),    # sequences too short for that
    (3, 160, 7, 520, torch.bfloat16, "sequence"),
    (1, 1, 444, 2560, torch.bfloat16, "channel"),      # the most rows that have a CTA each, and more
    (1, 1, 445, 2560, torch.bfloat16, "channel"),
    (1, 1, 1500, 2560, torch.bfloat16, "none"),
    (1, 2, 500, 8192, torch.bfloat16, "sequence"),
    (1, 1, 700, 8192, torch.bfloat16, "token"),        # two stages do not fit beside the weights
    (1, 1, 30, 8192, torch.bfloat16, "channel"),
    (1, 200, 50, 2056, torch.float32, "sequence"),
])
def test_residual_norm_backward_in_one_cta_or_several(P, B, s, D, dtype, gate):
    test_residual_norm_backward(P, B, s, D, dtype, gate, True)
