"""Cases of the last-layer operators for targets served in 8-bit floating point:
the norms around the last block (sv_block_norm), block quantisation
(sv_quantize_fp8), the LM head on e4m3 operands (sv_lm_head_logits_fp8) and
the verification fused behind it (spec_verify_lm_head_fp8).

`own` False: each operator in elementary torch operations; True: the calls a
user makes.  A case's M rows are the B (K+1) verified positions of a batch.
"""
import math

import torch

own = False

DEV = "cuda"
BLK = 128            # values along d (and, for weights, rows) that share a scale
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one sequence, four drafts: the plain last norm of a decode step
        dict(name="norm_m5_d4096", op="norm", M=5, d=4096, x="bf16", res="bf16", w="bf16", post=False, gate=0,
             rs=1.0, bs=1.0, offset=0.0, hidden="bf16"),
        # odd width, everything in fp32, norms on both sides and a gate for each sequence of 9 positions
        dict(name="norm_m153_d1021_fp32", op="norm", M=153, d=1021, x="fp32", res="fp32", w="fp32", post=True, gate=17,
             rs=0.5, bs=0.22, offset=0.0, hidden="fp32"),
        # 256 sequences x 9 positions: sandwich norms (weights stored less one), fp32 residual stream, e4m3 out
        dict(name="norm_m2304_d4096_e4m3", op="norm", M=2304, d=4096, x="bf16", res="fp32", w="bf16", post=True,
             gate=256, rs=1.0, bs=1.0, offset=1.0, hidden="e4m3"),
        # activations of 64 sequences x 6 positions, a scale for each row and 128 values
        dict(name="quant_m384_d4096", op="quant", M=384, d=4096, x="bf16", rows=1),
        # an output embedding laid out once at load time, ragged on both axes
        dict(name="quant_v32003_d4112_w", op="quant", M=32003, d=4112, x="bf16", rows=128),
        # a single token (no drafts): the weights' bytes
        dict(name="head_m1_v32000_d4096", op="head", M=1, V=32000, d=4096),
        # 8 sequences x 5 positions
        dict(name="head_m40_v32000_d4096", op="head", M=40, V=32000, d=4096),
        # odd sizes: rows, an odd vocabulary, a last block of 16 along d
        dict(name="head_m131_v32003_d1040", op="head", M=131, V=32003, d=1040),
        # 64 sequences x 6 positions
        dict(name="head_m384_v128256_d4096", op="head", M=384, V=128256, d=4096),
        # 256 sequences x 9 positions: the tensor cores' rate
        dict(name="head_m2304_v151936_d4096", op="head", M=2304, V=151936, d=4096),
        # the whole step, draft distributions given
        dict(name="verify_b8_k4_v32000", op="verify", B=8, K=4, V=32000, d=4096, T=0.8, dense=True),
        # the whole step with deterministic drafts, as from an n-gram lookup
        dict(name="verify_b64_k8_v128256_onehot", op="verify", B=64, K=8, V=128256, d=4096, T=0.7, dense=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "head", "head", "verify"])
    if op == "norm":
        M = _log(rng, 1, 2304)
        G = rng.choice([g for g in range(1, M + 1) if M % g == 0])
        x = rng.choice(["bf16", "fp32"])
        return dict(op=op, M=M, d=_log(rng, 60, 8192), x=x, res=rng.choice(["bf16", "fp32"]),
                    w=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.5, gate=rng.choice([0, 1, G]),
                    rs=rng.choice([1.0, 0.5]), bs=rng.choice([1.0, 0.22]), offset=rng.choice([0.0, 1.0]),
                    hidden=rng.choice(["bf16", "fp32", "e4m3"]))
    if op == "quant":
        rows = rng.choice([1, 128])
        return dict(op=op, M=_log(rng, 1, 2304) if rows == 1 else _log(rng, 100, 40000), d=_log(rng, 60, 8192),
                    x=rng.choice(["bf16", "fp32"]), rows=rows)
    if op == "head":
        M, V, d = _log(rng, 1, 2304), _log(rng, 500, 151936), 16 * _log(rng, 4, 512)
        while M * V * d > 2304 * 151936 * 4096:
            d = d // 32 * 16
        return dict(op=op, M=M, V=V, d=d)
    return dict(op=op, B=_log(rng, 1, 64), K=rng.randint(0, 8), V=_log(rng, 500, 128256), d=16 * _log(rng, 4, 256),
                T=rng.choice([0.7, 0.8, 1.0]), dense=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def _weights(g, V, d):
    """An output embedding N(0, 1/d) in e4m3 with a scale for each 128 x 128 block, made in pieces."""
    w = torch.empty((V, d), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((-(-V // BLK), -(-d // BLK)), device=DEV)
    step = 128 * BLK
    for v in range(0, V, step):
        n = min(step, V - v)
        w[v:v + n], s[v // BLK:-(-(v + n) // BLK)] = _quant_plain(_normal(g, (n, d), 3.0 / math.sqrt(d)), BLK)
    return w, s


def _low_bit_head(g, M, V, d):
    """Operands whose products add up exactly in 32 bits: small whole activations, weights of three values, scales
    that are powers of two, as low-bit checkpoints kept in e4m3 have them.  Logits then have one right value, and the
    tokens drawn from them can be compared one for one."""
    nb = -(-d // BLK)
    h = _normal(g, (M, d), 2.0).round_().clamp_(-8, 8).to(torch.float8_e4m3fn)
    w = torch.empty((V, d), dtype=torch.float8_e4m3fn, device=DEV)
    for v in range(0, V, 16384):
        n = min(16384, V - v)
        w[v:v + n] = (torch.randint(0, 4, (n, d), generator=g, device=DEV, dtype=torch.int8) - 1).clamp_(-1, 1).float() \
            .mul_(torch.randint(0, 2, (n, 1), generator=g, device=DEV).mul_(2).sub_(1).float()).to(torch.float8_e4m3fn)
    # logits of standard deviation about 3: each term is about 2 * 0.87 * the two scales
    e = round(math.log2(3.0 / (1.7 * math.sqrt(d))))
    hs = torch.tensor([0.5, 1.0], device=DEV)[torch.randint(0, 2, (M, nb), generator=g, device=DEV)]
    ws = torch.tensor([2.0 ** e, 2.0 ** (e + 1)], device=DEV)[
        torch.randint(0, 2, (-(-V // BLK), nb), generator=g, device=DEV)]
    return h, hs, w, ws


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "norm":
        M, d = c["M"], c["d"]
        s = dict(x=_normal(g, (M, d), 1.5, DTYPES[c["x"]]), res=_normal(g, (M, d), 4.0, DTYPES[c["res"]]),
                 pre=(1 - c["offset"] + _normal(g, (d,), 0.2)).to(DTYPES[c["w"]]), post=None, gate=None)
        if c["post"]:
            s["post"] = (1 - c["offset"] + _normal(g, (d,), 0.2)).to(DTYPES[c["w"]])
        if c["gate"]:
            s["gate"] = _normal(g, (c["gate"], d), 1.0, DTYPES[c["x"]])
    elif c["op"] == "quant":
        # values whose size varies from block to block, as activations and weights do
        spread = torch.exp(_normal(g, (c["M"], 1), 0.7 if c["rows"] == 1 else 0.1))
        s = dict(x=_normal(g, (c["M"], c["d"])).mul_(spread).to(DTYPES[c["x"]]))
    elif c["op"] == "head":
        h, hs = _quant_plain(_normal(g, (c["M"], c["d"])), 1)
        w, ws = _weights(g, c["V"], c["d"])
        s = dict(h=h, hs=hs, w=w, ws=ws)
    else:
        B, K, V, d = c["B"], c["K"], c["V"], c["d"]
        h, hs, w, ws = _low_bit_head(g, B * (K + 1), V, d)
        u = torch.rand((B, K + 1), generator=g, device=DEV)
        z = _head_plain(h, hs, w, ws, torch.float32).view(B, K + 1, V)[:, :K] / c["T"]
        if c["dense"]:
            q = torch.softmax(z + _normal(g, z.shape, 1.0), -1)
            cdf = q.double().cumsum(-1)
            t = torch.rand((B, K, 1), generator=g, device=DEV, dtype=torch.float64) * cdf[..., -1:]
            tok = (cdf <= t).sum(-1).clamp_(max=V - 1)
        else:
            q = None
            tok = torch.where(torch.rand((B, K), generator=g, device=DEV) < 0.6, z.argmax(-1),
                              torch.randint(0, V, (B, K), generator=g, device=DEV))
        s = dict(h=h.view(B, K + 1, d), hs=hs.view(B, K + 1, -1), w=w, ws=ws, q=q, tok=tok.int(), u=u)
    s["case"] = c
    return s


# ------------------------------------------------------------------ plain forms

def _rms(x, eps=1e-6):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)


def _norm_plain(s):
    c = s["case"]
    a = s["x"].float()
    if s["post"] is not None:
        a = _rms(a) * (s["post"].float() + c["offset"])
    if s["gate"] is not None:
        a = a * s["gate"].float().repeat_interleave(c["M"] // c["gate"], 0)
    r = c["rs"] * s["res"].float() + c["bs"] * a
    h = _rms(r) * (s["pre"].float() + c["offset"])
    r = r.to(s["res"].dtype)
    if c["hidden"] == "e4m3":
        v, sc = _quant_plain(h, 1)
        return [v, sc, r]
    return [h.to(DTYPES[c["hidden"]]), r]


def _blocks(x, rows):
    """x [M, d] padded with zeros to whole blocks: [M/rows, rows, d/128, 128]."""
    M, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % BLK, 0, -M % rows))
    return x.view(-1, rows, x.shape[1] // BLK, BLK)


def _quant_plain(x, rows):
    M, d = x.shape
    b = _blocks(x.float(), rows)
    s = b.abs().amax((1, 3), keepdim=True).clamp_(min=AMAX_FLOOR) / E4M3_MAX
    v = (b * (1.0 / s)).clamp_(-E4M3_MAX, E4M3_MAX).view(b.shape[0] * rows, -1)[:M, :d]
    return v.to(torch.float8_e4m3fn).contiguous(), s.view(s.shape[0], s.shape[2])


def _dequant(v, s, rows, dtype=torch.float32):
    """The values that e4m3 v and its block scales stand for."""
    f = v.to(dtype)
    s = s.to(dtype).repeat_interleave(BLK, 1)[:, :v.shape[1]]
    return f * (s if rows == 1 else s.repeat_interleave(rows, 0)[:v.shape[0]])


def _head_plain(h, hs, w, ws, dtype=torch.bfloat16):
    return (_dequant(h, hs, 1) @ _dequant(w, ws, BLK).T).to(dtype)


def _verify_plain(s):
    c = s["case"]
    B, K, V = c["B"], c["K"], c["V"]
    z = _head_plain(s["h"].flatten(0, 1), s["hs"].flatten(0, 1), s["w"], s["ws"]).view(B, K + 1, V)
    p = torch.softmax(z.double() / c["T"], -1)
    tok = s["tok"].long()
    px = p[:, :K].gather(-1, tok[..., None]).squeeze(-1)
    qx = s["q"].gather(-1, tok[..., None]).squeeze(-1).double() if c["dense"] else torch.ones_like(px)
    a = (px / qx).clamp(max=1.0)
    ok = s["u"][:, :K].double() < a
    n = ok.long().cumprod(-1).sum(-1)                       # accepted drafts
    pos = torch.arange(K + 1, device=z.device)
    p_row = p.gather(1, n[:, None, None].expand(B, 1, V)).squeeze(1)
    j = n.clamp(max=max(K - 1, 0))
    rejected = n < K
    w = p_row.clone()
    if K:
        if c["dense"]:
            q_row = s["q"].gather(1, j[:, None, None].expand(B, 1, V)).squeeze(1).double()
        else:
            q_row = torch.zeros_like(p_row).scatter_(1, tok.gather(1, j[:, None]), 1.0)
        w = torch.where(rejected[:, None], (p_row - q_row).clamp(min=0), w)
    mass = w.sum(-1)
    cdf = w.cumsum(-1)
    drawn = (cdf <= s["u"][:, K:].double() * cdf[:, -1:]).sum(-1).clamp(max=V - 1)
    drafts = torch.nn.functional.pad(tok, (0, 1), value=-1)
    out = torch.where(pos < n[:, None], drafts, -1)
    out = torch.where(pos == n[:, None], drawn[:, None], out)
    flags = torch.where(pos[:K] < n[:, None], 1, torch.where(pos[:K] == n[:, None], 0, -1))
    return dict(logits=z, tokens=out.int(), count=(n + 1).int(), flags=flags.to(torch.int8), prob=a.float(),
                mass=torch.where(rejected, mass, 0.0).float())


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_sampling_gb300 as sv
        if c["op"] == "norm":
            r = sv.sv_block_norm(s["x"], s["res"], s["pre"], post_weight=s["post"], gate=s["gate"],
                                 residual_scale=c["rs"], branch_scale=c["bs"], weight_offset=c["offset"], eps=1e-6,
                                 hidden_dtype=DTYPES[c["hidden"]])
            return [r.hidden, r.residual] if r.scales is None else [r.hidden, r.scales, r.residual]
        if c["op"] == "quant":
            return sv.sv_quantize_fp8(s["x"], block_rows=c["rows"])
        if c["op"] == "head":
            return sv.sv_lm_head_logits_fp8(s["h"], s["hs"], s["w"], s["ws"])
        res, logits = sv.spec_verify_lm_head_fp8(s["h"], s["hs"], s["w"], s["ws"], s["q"], s["tok"], s["u"], c["T"])
        return dict(logits=logits, tokens=res.out_tokens, count=res.num_emitted, flags=res.accept_flags,
                    prob=res.accept_prob, mass=res.residual_mass)
    if c["op"] == "norm":
        return _norm_plain(s)
    if c["op"] == "quant":
        return _quant_plain(s["x"], c["rows"])
    if c["op"] == "head":
        return _head_plain(s["h"], s["hs"], s["w"], s["ws"])
    return _verify_plain(s)


def work(case):
    c = case
    if c["op"] == "norm":
        M, d = c["M"], c["d"]
        size = {"bf16": 2, "fp32": 4, "e4m3": 1}
        b = M * d * (size[c["x"]] + 2 * size[c["res"]] + size[c["hidden"]])
        b += d * size[c["w"]] * (2 if c["post"] else 1) + c["gate"] * d * size[c["x"]]
        if c["hidden"] == "e4m3":
            b += 4 * M * -(-d // BLK)
        return {"bytes": b, "flops": M * d * (5 + (4 if c["post"] else 0))}
    if c["op"] == "quant":
        M, d = c["M"], c["d"]
        return {"bytes": M * d * ((2 if c["x"] == "bf16" else 4) + 1) + 4 * -(-M // c["rows"]) * -(-d // BLK),
                "flops": 3 * M * d}
    M = c["M"] if c["op"] == "head" else c["B"] * (c["K"] + 1)
    V, d = c["V"], c["d"]
    nb = -(-d // BLK)
    b = M * d + 4 * M * nb + V * d + 4 * -(-V // BLK) * nb + 2 * M * V
    if c["op"] == "verify":
        # the drafted entries of q, and each sequence's surviving row of q
        b += c["B"] * V * 4 if c["dense"] and c["K"] else 0
    return {"bytes": b, "flops": 2 * M * V * d}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f = torch.float64
    if c["op"] == "norm":
        def rms(v):
            return v / torch.sqrt((v * v).sum(-1, keepdim=True) / c["d"] + 1e-6)
        branch = s["x"].to(f)
        if s["post"] is not None:
            branch = rms(branch) * (s["post"].to(f) + c["offset"])
        if s["gate"] is not None:
            per = c["M"] // c["gate"]
            branch = (branch.view(c["gate"], per, -1) * s["gate"].to(f)[:, None]).view(c["M"], -1)
        r = s["res"].to(f) * c["rs"] + branch * c["bs"]
        h = rms(r) * (s["pre"].to(f) + c["offset"])
        if c["hidden"] != "e4m3":
            return [h, r]
        return [*_exact_quant(h, 1), r]
    if c["op"] == "quant":
        return tuple(_exact_quant(s["x"].to(f), c["rows"]))
    h, hs = s["h"].flatten(0, -2), s["hs"].flatten(0, -2)
    out = torch.empty((h.shape[0], c["V"]), dtype=f, device=DEV)
    hd = h.to(f)
    for b in range(hs.shape[1]):
        hd[:, b * BLK:(b + 1) * BLK] *= hs[:, b:b + 1].to(f)
    for v in range(0, c["V"], 8192):
        wd = s["w"][v:v + 8192].to(f)
        sc = s["ws"][v // BLK:-(-(v + wd.shape[0]) // BLK)].to(f)
        for i in range(sc.shape[0]):
            for b in range(sc.shape[1]):
                wd[i * BLK:(i + 1) * BLK, b * BLK:(b + 1) * BLK] *= sc[i, b]
        torch.matmul(hd, wd.T, out=out[:, v:v + wd.shape[0]])
    if c["op"] == "head":
        return out
    return _exact_verify(s, out)


def _exact_quant(x, rows):
    """x / scale before its rounding to e4m3, and the scales."""
    M, d = x.shape
    nr, nb = -(-M // rows), -(-d // BLK)
    big = torch.zeros((nr * rows, nb * BLK), dtype=x.dtype, device=x.device)
    big[:M, :d] = x
    cells = big.reshape(nr, rows, nb, BLK)
    s = torch.maximum(cells.abs().amax(3).amax(1), torch.tensor(AMAX_FLOOR, dtype=x.dtype, device=x.device)) / E4M3_MAX
    v = (cells / s[:, None, :, None]).reshape(nr * rows, nb * BLK)[:M, :d]
    return v, s


def _exact_verify(s, z):
    """The verification of the logits z rounded to bf16, sequence by sequence, for the computed numbers alone."""
    c = s["case"]
    B, K, V = c["B"], c["K"], c["V"]
    zb = z.to(torch.float32).to(torch.bfloat16).double().view(B, K + 1, V)
    prob = torch.zeros((B, K), dtype=torch.float64, device=DEV)
    mass = torch.zeros((B,), dtype=torch.float64, device=DEV)
    for b in range(B):
        e = torch.exp((zb[b] - zb[b].amax(-1, keepdim=True)) / c["T"])
        p = e / e.sum(-1, keepdim=True)
        done = False
        for k in range(K):
            x = int(s["tok"][b, k])
            qx = float(s["q"][b, k, x]) if c["dense"] else 1.0
            a = min(1.0, float(p[k, x]) / qx)
            prob[b, k] = a
            if not done and not float(s["u"][b, k]) < a:
                q = s["q"][b, k].double() if c["dense"] else torch.zeros(V, dtype=torch.float64, device=DEV)
                if not c["dense"]:
                    q[x] = 1.0
                mass[b] = (p[k] - q).clamp(min=0).sum()
                done = True
    return dict(logits=z.view(B, K + 1, V), tokens=None, count=None, flags=None, prob=prob, mass=mass)
