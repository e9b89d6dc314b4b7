"""Plain 64-bit forms of the last-layer operators (block norms, block
quantisation, the LM head on e4m3 operands) for the tests, with the error
bounds that follow from the kernels' roundings."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U = 2.0 ** -24               # half an fp32 step, relative
BLK = 128
AMAX_FLOOR = 2.0 ** -100
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


def blocks(n: int) -> int:
    return -(-n // BLK)


def rand(shape, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def spread_scales(s, rows, M, d):
    """Block scales [ceil(M / rows), ceil(d / 128)] as an [M, d] matrix."""
    return s.repeat_interleave(BLK, 1)[:, :d].repeat_interleave(rows, 0)[:M]


# ---------------------------------------------------------------- quantisation

def quantize_fp32(x, rows):
    """The documented steps in fp32 (each correctly rounded, so a kernel can
    match them bit for bit): values and scales."""
    M, d = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -d % BLK, 0, -M % rows))
    c = p.view(p.shape[0] // rows, rows, p.shape[1] // BLK, BLK)
    amax = c.abs().amax((1, 3))
    s = torch.maximum(amax, torch.tensor(AMAX_FLOOR)) / torch.tensor(448.0)
    v = x.float() * spread_scales(1.0 / s, rows, M, d)
    return torch.where(v.isnan(), v, v.clamp(-448, 448)).to(torch.float8_e4m3fn), s


# ---------------------------------------------------------------- the norms

def norm64(x, res, pre, post=None, gate=None, rs=1.0, bs=1.0, offset=0.0, eps=1e-6):
    """(h, r, bound of |h error|, bound of |r error|) in 64 bits, before the
    outputs' own rounding.  Per row of d values: a sum of squares is formed
    by fused adds of at most 64 terms in a lane, 5 levels of a warp sum and
    up to 16 warp sums, all positive: relative error <= 85 U; rsqrtf is
    within 2 steps (4 U)."""
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731  (the scalars are passed as fp32)
    rs, bs, offset, eps = f32(rs), f32(bs), f32(offset), f32(eps)
    x, res, pre = x.to(F64), res.to(F64), pre.to(F64)
    sum_err = 85 * U + 2 * U              # the sum, times 1/d (itself rounded), plus eps
    a, a_rel = x, 0.0
    if post is not None:
        a = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (post.to(F64) + offset)
        a_rel = sum_err / 2 + 4 * U + 3 * U   # rsqrt; w + offset, two products
    if gate is not None:
        g = gate.to(F64).reshape(-1, x.shape[-1])
        a = a * g.repeat_interleave(x.shape[0] // g.shape[0], 0)
        a_rel += U
    r = rs * res + bs * a
    er = (rs * res).abs() * U + (bs * a).abs() * a_rel + r.abs() * U
    er = er * 1.001                       # second-order terms
    ms = (r * r).mean(-1, keepdim=True)
    f = 1.0 / torch.sqrt(ms + eps)
    w = pre + offset
    h = r * f * w
    ms_rel = (2 * r.abs() * er).mean(-1, keepdim=True) / (ms + eps) + sum_err
    eh = ((w * f).abs() * er + h.abs() * (ms_rel / 2 + 4 * U + 3 * U)) * 1.001 + 1e-36
    return h, r, eh, er + 1e-36


def within(got, want, err, dtype):
    """|got - want| <= err + half a step of dtype around the value."""
    bound = err + HALF_STEP[dtype] * (want.abs() + err)
    return ((got.to(F64) - want).abs() <= bound).all()


# ---------------------------------------------------------------- the LM head

def head64(h, hs, w, ws):
    """Exact logits and the bound of their error before the rounding to bf16:
    the 128 products of a block are exact in fp32, and adding them costs at
    most a whole fp32 step (2 U) of the sum of magnitudes each; the scale's
    product and the multiply-add per block cost (nb + 2) U more."""
    M, d = h.shape
    V = w.shape[0]
    a = h.to(F64) * spread_scales(hs.to(F64), 1, M, d)
    b = w.to(F64) * spread_scales(ws.to(F64), BLK, V, d)
    z = a @ b.T
    mag = a.abs() @ b.abs().T
    return z, (2 * BLK + blocks(d) + 2) * U * mag + 1e-36


def head_operands(M, V, d, seed, dyadic=False):
    """e4m3 operands with block scales.  dyadic: entries 0 and +-1/2, scales
    powers of two, so that every partial sum is exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    if dyadic:
        pick = lambda *s: ((torch.randint(0, 3, s, generator=g) - 1) * 0.5).to(torch.float8_e4m3fn)  # noqa: E731
        pw = lambda *s: torch.tensor([0.5, 1.0, 2.0])[torch.randint(0, 3, s, generator=g)]  # noqa: E731
        return pick(M, d), pw(M, blocks(d)), pick(V, d), pw(blocks(V), blocks(d))
    h, hs = quantize_fp32(torch.randn(M, d, generator=g), 1)
    w, ws = quantize_fp32(torch.randn(V, d, generator=g) * (3.0 / math.sqrt(d)), BLK)
    return h, hs, w, ws
