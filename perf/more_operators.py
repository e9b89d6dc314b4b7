"""Cases of the operators of a draft step in 4-bit floating point: microscaled
quantisation and its reading back (sv_quantize_fp4, sv_dequantize_fp4), the LM
head on such operands (sv_lm_head_logits_fp4), and the draw of tokens from its
logits with temperature, top-k, top-p and min-p (sv_sample_logits), whose
probabilities the verification takes as q.

`own` False: each operator in elementary torch operations; True: the calls a
user makes.

The 4-bit form of a matrix [rows, d]: two e2m1 values a byte (the even column
in the low half), a scale for each block of 16 values (e4m3, beside a power of
two for each row) or of 32 (a power of two, e8m0).  The scales lie in tiles of
128 rows x 4 blocks: [rows / 128, blocks / 4, 32, 4, 4], element [i, j, l, a, b]
belonging to row 128 i + 32 a + l and block 4 j + b; zeros behind the ends.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a draft step's hidden states, 8 sequences x 5 positions: latency
        dict(name="quant16_m40_d4096", op="quant", block=16, M=40, d=4096, x="bf16"),
        # fp32 activations of many positions, ragged: a last block of 8 values
        dict(name="quant32_m2299_d1000_fp32", op="quant", block=32, M=2299, d=1000, x="fp32"),
        # an output embedding laid out at load time and read back
        dict(name="quant16_v128256_d4096", op="quant", block=16, M=128256, d=4096, x="bf16"),
        # one token: the weights' bytes
        dict(name="head16_m1_v32000_d4096", op="head", block=16, M=1, V=32000, d=4096),
        # a small draft model's head over a large vocabulary, 64 sequences
        dict(name="head32_m64_v128256_d2048", op="head", block=32, M=64, V=128256, d=2048),
        # odd sizes: rows, an odd vocabulary, a last step of 32 along d
        dict(name="head16_m131_v32003_d1056", op="head", block=16, M=131, V=32003, d=1056),
        # 256 sequences x 9 positions: the tensor cores' rate
        dict(name="head16_m2304_v151936_d4096", op="head", block=16, M=2304, V=151936, d=4096),
        # one sequence's draft token from fp32 logits with the usual chat settings, q kept for the verification
        dict(name="sample_b1_v32000_fp32", op="sample", rows=1, V=32000, x="fp32", sigma=3.0, bias=1.1, masked=0.0, T=0.8,
             top_k=50, top_p=0.95, min_p=0.0, probs=True),
        # 8 drafting sequences, nucleus sampling
        dict(name="sample_b8_v128256_topp", op="sample", rows=8, V=128256, x="bf16", sigma=3.0, bias=1.1, masked=0.0,
             T=1.0, top_k=0, top_p=0.9, min_p=0.0, probs=True),
        # odd sizes, min-p, a twentieth of the vocabulary masked; tokens only (no verification behind it)
        dict(name="sample_b133_v32003_minp", op="sample", rows=133, V=32003, x="fp32", sigma=4.0, bias=0.0, masked=0.05,
             T=0.9, top_k=0, top_p=1.0, min_p=0.05, probs=False),
        # a batch's drafts with every filter
        dict(name="sample_b256_v128256_all", op="sample", rows=256, V=128256, x="bf16", sigma=3.0, bias=1.1, masked=0.0,
             T=0.7, top_k=1000, top_p=0.9, min_p=0.01, probs=True),
        # a large batch at temperature alone: the bytes of logits and q
        dict(name="sample_b256_v151936", op="sample", rows=256, V=151936, x="bf16", sigma=4.0, bias=1.2, masked=0.0,
             T=0.7, top_k=0, top_p=1.0, min_p=0.0, probs=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["quant", "head", "head", "sample", "sample"])
    block = rng.choice([16, 32])
    if op == "quant":
        x = rng.choice(["bf16", "fp32"])
        return dict(op=op, block=block, M=_log(rng, 1, 128256 if x == "bf16" else 64128), d=2 * _log(rng, 30, 2048), x=x)
    if op == "head":
        return dict(op=op, block=block, M=_log(rng, 1, 2304), V=_log(rng, 500, 151936), d=32 * _log(rng, 2, 128))
    return dict(op=op, rows=_log(rng, 1, 256), V=_log(rng, 500, 128256), x=rng.choice(["bf16", "bf16", "fp32"]),
                sigma=rng.choice([2.0, 3.0, 4.0]), bias=rng.choice([0.0, 1.1]), masked=rng.choice([0.0, 0.0, 0.05]),
                T=rng.choice([0.6, 0.7, 0.8, 1.0]), top_k=rng.choice([0, 0, rng.randint(1, 64), rng.randint(65, 2000)]),
                top_p=rng.choice([1.0, 0.95, 0.9, round(rng.uniform(0.5, 0.99), 3)]),
                min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), probs=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def _operand(g, rows, d, std, block):
    """A matrix N(0, std^2) in 4-bit form, made in pieces of whole scale tiles."""
    values, scales, outer = [], [], []
    for r in range(0, rows, 16384):
        n = min(16384, rows - r)
        v, s, o = _quant_plain(_normal(g, (n, d), std), block)
        values.append(_pack(v))
        scales.append(_tile(s))
        outer.append(o)
    return dict(values=torch.cat(values), scales=torch.cat([s.view(torch.uint8) for s in scales]).view(scales[0].dtype),
                rows=torch.cat(outer) if block == 16 else None, block=block)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "quant":
        # values whose size varies from row to row, as activations' does
        s = dict(x=_normal(g, (c["M"], c["d"])).mul_(torch.exp(_normal(g, (c["M"], 1), 0.5))).to(DTYPES[c["x"]]))
    elif c["op"] == "head":
        s = dict(h=_operand(g, c["M"], c["d"], 1.0, c["block"]),
                 w=_operand(g, c["V"], c["d"], 3.0 / math.sqrt(c["d"]), c["block"]))
    else:
        z = _normal(g, (c["rows"], c["V"]), c["sigma"])
        z -= c["bias"] * torch.log(torch.arange(1, c["V"] + 1, device=DEV, dtype=torch.float32))
        if c["masked"]:
            z.masked_fill_(torch.rand(z.shape, generator=g, device=DEV) < c["masked"], -math.inf)
        s = dict(z=z.to(DTYPES[c["x"]]), u=torch.rand((c["rows"],), generator=g, device=DEV))
    s["case"] = c
    return s


# ------------------------------------------------------------------ plain forms

def _pow2(k):
    """2^k in fp32, for whole -127 <= k <= 127."""
    b = (k.int() + 127) << 23
    return torch.where(b > 0, b, 1 << 22).int().view(torch.float32)


def _quant_plain(x, block):
    """x [rows, d] as e2m1 values (in fp32), their scales [rows, blocks] and the rows' powers of two (block 16)."""
    rows, d = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -d % block)).view(rows, -1, block)
    amax = b.abs().amax(-1)
    if block == 16:
        # the least power of two that brings the row's largest block scale to 448 or below
        mant, e = torch.frexp(amax.amax(-1))
        k = torch.where(mant > 2688 / 4096, e - 11, e - 12).clamp(min=-126)
        outer = _pow2(torch.where(mant > 0, k, 0))
        s = (amax / (6.0 * outer)[:, None]).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
        s = torch.where(amax > 0, s, 0.0)
        step = (s * outer[:, None])[..., None]
        s = s.to(torch.float8_e4m3fn)
    else:
        outer = None
        e = (torch.frexp(amax)[1] - 3).clamp(min=-127)
        e = torch.where(amax > 0, e, -127)
        s = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        step = _pow2(e)[..., None]
    a = torch.where(step > 0, b / step, 0.0)
    m = a.abs()
    v = 0.5 * (m > 0.25) + 0.5 * (m >= 0.75) + 0.5 * (m > 1.25) + 0.5 * (m >= 1.75) + (m > 2.5) + (m >= 3.5) + 2.0 * (m > 5)
    return torch.copysign(v, a).view(rows, -1)[:, :d], s, outer


def _pack(v):
    """e2m1 values [rows, d] as bytes [rows, d / 2]."""
    m = v.abs()
    code = sum((m >= t).to(torch.uint8) for t in E2M1[1:]) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(p, dtype=torch.float32):
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=p.device)
    return torch.stack((t[(p & 15).int()], t[(p >> 4).int()]), -1).view(p.shape[0], -1)


def _tile(s):
    """Scales [rows, blocks] in tiles."""
    rows, nb = s.shape
    b = torch.nn.functional.pad(s.view(torch.uint8), (0, -nb % 4, 0, -rows % 128))
    b = b.view(-1, 4, 32, b.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return b.view(s.dtype)


def _untile(t, rows, nb, dtype=torch.float32):
    """The scales' values, [rows, nb]."""
    b = t.view(torch.uint8).permute(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, t.shape[1] * 4)[:rows, :nb].contiguous()
    if t.dtype == torch.float8_e4m3fn:
        return b.view(t.dtype).to(dtype)
    return _pow2(b.int() - 127).to(dtype)


def _dequant(o, dtype=torch.float32):
    """The values that an operand in 4-bit form stands for."""
    rows, d = o["values"].shape[0], 2 * o["values"].shape[1]
    s = _untile(o["scales"], rows, -(-d // o["block"]), dtype)
    if o["rows"] is not None:
        s = s * o["rows"][:, None].to(dtype)
    return _unpack(o["values"], dtype) * s.repeat_interleave(o["block"], 1)[:, :d]


def _sample_plain(s):
    c = s["case"]
    z = s["z"].double()
    T, top_p, min_p = (torch.tensor(c[k], dtype=torch.float32).double().item() for k in ("T", "top_p", "min_p"))
    w = torch.exp((z - z.amax(-1, keepdim=True)) / T)
    ranked, order = torch.sort(z, dim=-1, descending=True, stable=True)
    r = w.gather(-1, order)
    keep = ranked > -math.inf
    if c["top_k"] > 0:
        keep &= torch.arange(c["V"], device=DEV) < c["top_k"]
    if top_p < 1:
        cum = (r * keep).cumsum(-1)
        keep &= torch.nn.functional.pad(cum[:, :-1], (1, 0)) < top_p * cum[:, -1:]
    if min_p > 0:
        keep &= r >= min_p
    kept = keep.sum(-1)
    w = w * torch.zeros_like(keep).scatter_(-1, order, keep)
    cdf = w.cumsum(-1)
    tokens = (cdf <= s["u"].double()[:, None] * cdf[:, -1:]).sum(-1)
    p = (w / w.sum(-1, keepdim=True)).float()
    out = dict(tokens=tokens.int(), prob=p.gather(-1, tokens[:, None]).squeeze(-1), kept=kept.int())
    if c["probs"]:
        out["probs"] = p
    return out


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_sampling_gb300 as sv
        if c["op"] == "quant":
            t = sv.sv_quantize_fp4(s["x"], block=c["block"])
            back = sv.sv_dequantize_fp4(t)
            return [back] if t.row_scales is None else [back, t.row_scales]
        if c["op"] == "head":
            h, w = (sv.Fp4Tensor(o["values"], o["scales"], o["rows"]) for o in (s["h"], s["w"]))
            return sv.sv_lm_head_logits_fp4(h, w)
        r = sv.sv_sample_logits(s["z"], s["u"], c["T"], c["top_k"], c["top_p"], c["min_p"], want_probs=c["probs"])
        out = dict(tokens=r.tokens, prob=r.prob, kept=r.kept)
        if c["probs"]:
            out["probs"] = r.probs
        return out
    if c["op"] == "quant":
        v, sc, outer = _quant_plain(s["x"], c["block"])
        nb = sc.shape[1]
        f = _untile(_tile(sc), c["M"], nb) * (1.0 if outer is None else outer[:, None])
        back = (_unpack(_pack(v)) * f.repeat_interleave(c["block"], 1)[:, :c["d"]]).to(torch.bfloat16)
        return [back] if outer is None else [back, outer]
    if c["op"] == "head":
        return (_dequant(s["h"]) @ _dequant(s["w"]).T).to(torch.bfloat16)
    return _sample_plain(s)


def work(case):
    c = case
    if c["op"] == "quant":
        M, d = c["M"], c["d"]
        form = M * d // 2 + M * -(-d // c["block"]) + (4 * M if c["block"] == 16 else 0)
        # x in, the 4-bit form out and in again, bf16 out
        return {"bytes": M * d * ((2 if c["x"] == "bf16" else 4) + 2) + 2 * form, "flops": 3 * M * d}
    if c["op"] == "head":
        M, V, d = c["M"], c["V"], c["d"]
        form = (M + V) * (d // 2 + -(-d // c["block"]) + (4 if c["block"] == 16 else 0))
        return {"bytes": form + 2 * M * V, "flops": 2 * M * V * d}
    n = c["rows"] * c["V"]
    return {"bytes": n * ((2 if c["x"] == "bf16" else 4) + (4 if c["probs"] else 0)) + 16 * c["rows"], "flops": 4 * n}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f = torch.float64
    if c["op"] == "quant":
        return _exact_quant(s["x"], c["block"])
    if c["op"] == "head":
        h, w = s["h"], s["w"]
        a = _exact_values(h)
        out = torch.empty((c["M"], c["V"]), dtype=f, device=DEV)
        for v in range(0, c["V"], 8192):
            n = min(8192, c["V"] - v)
            part = dict(values=w["values"][v:v + n], scales=w["scales"][v // 128:-(-(v + n) // 128)],
                        rows=None if w["rows"] is None else w["rows"][v:v + n], block=w["block"])
            torch.matmul(a, _exact_values(part).T, out=out[:, v:v + n])
        return out
    probs = torch.zeros((c["rows"], c["V"]), dtype=f, device=DEV)
    prob = torch.empty((c["rows"],), dtype=f, device=DEV)
    T, top_p, min_p = (torch.tensor(c[k], dtype=torch.float32).double().item() for k in ("T", "top_p", "min_p"))
    for i in range(c["rows"]):
        z = s["z"][i].to(f)
        p = torch.exp((z - z.max()) / T)
        p /= p.sum()
        ids = torch.argsort(z, descending=True, stable=True)[:int((z > -math.inf).sum())]
        if c["top_k"] > 0:
            ids = ids[:c["top_k"]]
        if top_p < 1:
            mass = p[ids].cumsum(0)
            ids = ids[:int((mass < top_p * mass[-1]).sum()) + 1]
        if min_p > 0:
            ids = ids[p[ids] >= min_p * p.max()]
        probs[i, ids] = p[ids] / p[ids].sum()
        at = torch.searchsorted(probs[i].cumsum(0), s["u"][i:i + 1].to(f), right=True)
        prob[i] = probs[i, at.clamp(max=c["V"] - 1)]
    out = dict(tokens=None, prob=prob, kept=None)
    if c["probs"]:
        out["probs"] = probs
    return out


def _exact_values(o):
    """The values of an operand in 4-bit form, from its bits."""
    p = o["values"]
    code = torch.stack((p & 15, p >> 4), -1).flatten(1).int()
    e, m = (code >> 1) & 3, code & 1
    mag = torch.where(e > 0, torch.exp2((e - 1).double()) * (1 + 0.5 * m), 0.5 * m.double())
    v = torch.where(code > 7, -mag, mag)
    rows, d = v.shape
    r, b = torch.arange(rows, device=p.device)[:, None], torch.arange(d, device=p.device)[None] // o["block"]
    byte = o["scales"].view(torch.uint8)[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].int()
    if o["block"] == 32:
        return v * torch.exp2((byte - 127).double())
    big = torch.exp2(((byte >> 3) & 15).double() - 7) * (1 + (byte & 7).double() / 8)
    scale = torch.where((byte >> 3) & 15 > 0, big, (byte & 7).double() * 2.0 ** -9)
    return v * scale * o["rows"].double()[:, None]


def _exact_quant(x, block):
    """What the 4-bit form of x stands for, a column of blocks after the other."""
    rows, d = x.shape
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    top = x.abs().amax(1).double()
    half, e = torch.frexp(torch.where(top > 0, top, 2688.0) / 2688)
    outer = torch.exp2((e - (half == 0.5).int()).clamp(min=-126).double())
    out = torch.empty((rows, d), dtype=torch.float64, device=x.device)
    for b in range(0, d, block):
        v = x[:, b:b + block].double()
        a = v.abs().amax(1)
        if block == 16:
            t = a / outer / 6
            step = torch.exp2(torch.frexp(t.clamp(min=2.0 ** -6))[1].double() - 4)
            sc = (torch.round(t / step) * step).clamp(min=2.0 ** -9) * outer
        else:
            sc = torch.exp2(torch.frexp(a.clamp(min=2.0 ** -125))[1].double() - 3)
        t = v.abs() / sc[:, None]
        at = (t[..., None] > mids).sum(-1)
        # halfway cases go to the value with an even last bit
        at += ((at % 2 == 1) & (t == mids[at.clamp(max=6)])).long()
        out[:, b:b + block] = torch.copysign(grid[at], v) * sc[:, None]
    out = torch.where(out.abs() > 0, out, 0.0)
    return [out, outer] if block == 16 else [out]
