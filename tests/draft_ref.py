"""Plain 64-bit forms of the draft step's operators (CPU, numpy): 4-bit
quantisation, the LM head on it, the draw of tokens."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_e2m1(x):
    """Nearest e2m1 value, ties to the even code, magnitudes over 6 to 6."""
    m = np.abs(x)
    best = np.zeros(x.shape)
    err = np.abs(m - E2M1[0])
    for i, g in enumerate(E2M1[1:], 1):
        e = np.abs(m - g)
        take = (e < err) | ((e == err) & (i % 2 == 0))
        best = np.where(take, g, best)
        err = np.where(take, e, err)
    return np.copysign(best, x)


def round_e4m3(x):
    """Nearest e4m3 value of 0 <= x <= 448, ties to even (halves of a step are exact in 64 bits)."""
    e = np.maximum(np.floor(np.log2(np.maximum(x, 2.0 ** -40))), -6.0)
    step = 2.0 ** (e - 3)
    return np.round(x / step) * step


def quantize(x, block):
    """(values, block scales [M, nb], row scales [M] or None) of a float64 [M, d]; the quotients are rounded to
    fp32, as defined.  NaN in the scales of blocks that hold a NaN or an infinity."""
    M, d = x.shape
    nb = -(-d // block)
    b = np.zeros((M, nb * block))
    b[:, :d] = x
    b = b.reshape(M, nb, block)
    bad = ~np.isfinite(b).all(-1)
    clean = np.where(bad[..., None], 0.0, b)
    amax = np.abs(clean).max(-1)
    if block == 16:
        top = amax.max(-1)
        k = np.array([max(-126, math.ceil(math.log2(t / 2688))) if t > 0 else 0 for t in top])
        for i, t in enumerate(top):  # log2 rounds: settle the least k by comparison
            while t > 0 and k[i] > -126 and t <= 2688 * 2.0 ** (k[i] - 1):
                k[i] -= 1
            while t > 2688 * 2.0 ** k[i]:
                k[i] += 1
        g = 2.0 ** k.astype(np.float64)
        q = (amax / g[:, None] / 6).astype(np.float32).astype(np.float64)
        s = np.where(amax > 0, np.maximum(round_e4m3(q), 2.0 ** -9), 0.0)
        step = s * g[:, None]
    else:
        g = None
        mant, e = np.frexp(amax)
        s = np.where(amax > 0, 2.0 ** np.maximum(e - 3.0, -127), 2.0 ** -127)
        step = s
    with np.errstate(invalid="ignore", divide="ignore"):
        v = np.where(step[..., None] > 0, (clean / step[..., None]).astype(np.float32).astype(np.float64), 0.0)
    v = round_e2m1(v)
    s = np.where(bad, np.nan, s)
    return v.reshape(M, -1)[:, :d], s, g


def tile(s, rows=None):
    """Scales [M, nb] in tiles [ceil(M / 128), ceil(nb / 4), 32, 4, 4] (0 behind the ends)."""
    M, nb = s.shape
    t = np.zeros((-(-M // 128) * 128, -(-nb // 4) * 4))
    t[:M, :nb] = s
    return t.reshape(-1, 4, 32, t.shape[1] // 4, 4).transpose(0, 3, 2, 1, 4)


def pack(v):
    """e2m1 values [M, d] as bytes."""
    code = np.searchsorted(E2M1, np.abs(v)).astype(np.uint8) | (np.signbit(v).astype(np.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(p):
    code = np.stack((p & 15, p >> 4), -1).reshape(p.shape[0], -1)
    return np.where(code > 7, -1.0, 1.0) * E2M1[code & 7]


def to_device(sv, v, s, g, block, dev="cuda:0", lead=None):
    """The Fp4Tensor of values v [M, d], scales s [M, nb] and row scales g."""
    lead = lead or (v.shape[0],)
    t = torch.from_numpy(np.ascontiguousarray(tile(s))).float()
    if block == 16:
        scales = t.to(torch.float8_e4m3fn)
    else:
        with np.errstate(divide="ignore"):
            e = np.where(tile(s) > 0, np.log2(np.where(tile(s) > 0, tile(s), 1.0)) + 127, 0)
        scales = torch.from_numpy(np.ascontiguousarray(e.astype(np.uint8))).view(torch.float8_e8m0fnu)
    return sv.Fp4Tensor(torch.from_numpy(pack(v)).reshape(*lead, -1).to(dev), scales.to(dev),
                        None if g is None else torch.from_numpy(np.asarray(g)).float().reshape(lead).to(dev))


def head(hv, hs, hg, wv, ws, wg, block):
    """(logits, sum of magnitudes) in 64 bits."""
    def full(v, s, g):
        f = v * np.repeat(s, block, 1)[:, :v.shape[1]]
        return f if g is None else f * np.asarray(g, np.float64)[:, None]
    a, b = full(hv, hs, hg), full(wv, ws, wg)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def sample(z, u, T, top_k=0, top_p=1.0, min_p=0.0):
    """One row in 64 bits: (token, kept mask, q, margin); margin: the least relative distance of a decision (a cut
    by mass, the draw) from an id's boundary."""
    T, top_p, min_p, u = (float(np.float32(v)) for v in (T, top_p, min_p, u))
    z = z.astype(np.float64)
    V = z.size
    w = np.exp((z - z.max()) / T)
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if top_k > 0:
        order = order[:top_k]
    margin = np.inf
    if top_p < 1:
        cum = np.cumsum(w[order])
        target = top_p * cum[-1]
        n = int((cum < target).sum()) + 1
        margin = min(margin, np.abs(cum - target).min() / cum[-1])
        order = order[:n]
    if min_p > 0:
        order = order[w[order] >= min_p]
    keep = np.zeros(V, bool)
    keep[order] = True
    w = np.where(keep, w, 0.0)
    cdf = np.cumsum(w)
    token = int((cdf <= u * cdf[-1]).sum())
    if u > 0:
        margin = min(margin, np.abs(cdf - u * cdf[-1]).min() / cdf[-1])
    return token, keep, w / w.sum(), margin
