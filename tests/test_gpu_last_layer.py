"""The norms around the target's last block and block quantisation, through
the binding, against plain 64-bit forms."""
import pytest
import torch

import last_layer_ref as R
import speculative_decoding_sampling_gb300 as sv
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _bits(t):
    t = t.cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _check_e4m3(v, s, want, err):
    """Values and scales of a quantised h: the scale is amax / 448 of h
    within h's own error, and v * s is h within half an e4m3 step (of the
    value, or of the smallest step 2^-9) and h's error."""
    M, d = want.shape
    nb = R.blocks(d)
    pad = lambda t: torch.nn.functional.pad(t, (0, nb * 128 - d)).view(M, nb, 128)  # noqa: E731
    amax = pad(want.abs()).amax(-1)
    aerr = pad(err).amax(-1)
    s = s.to(R.F64)
    assert ((s - amax / 448).abs() <= aerr / 448 + 2 * R.U * amax / 448 + 1e-36).all()
    sc = R.spread_scales(s, 1, M, d)
    got = v.to(R.F64) * sc
    # the product x * (1 / s) and the reciprocal: 2 U each, before the rounding
    bound = (err + 4 * R.U * want.abs()) * 1.1 + 2.0 ** -4 * want.abs() + 2.0 ** -10 * sc
    assert ((got - want).abs() <= bound).all()


# (M, d): below one lane's 8 values, odd widths (single accesses), a width
# that is a multiple of 8 but not of 128, every count of warps per row and of
# segments per warp, the widest row
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 129), (7, 200), (4, 256), (9, 504), (33, 1021), (6, 1024), (5, 4096),
          (3, 4112), (2, 8200), (3, 12345), (2, 32768)]


@pytest.mark.parametrize("M,d", SHAPES, ids=[f"M{m}_d{d}" for m, d in SHAPES])
@pytest.mark.parametrize("hidden", [BF, FP, E4], ids=["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("xt,rt,wt", [(BF, BF, BF), (BF, FP, FP), (FP, FP, BF), (FP, BF, FP)])
def test_block_norm(M, d, hidden, xt, rt, wt):
    seed = 1000 * M + d
    x, res = R.rand((M, d), seed, xt, 1.5), R.rand((M, d), seed + 1, rt, 4.0)
    pre, post = R.rand((d,), seed + 2, wt, 0.3), R.rand((d,), seed + 3, wt, 0.3)
    sandwich = (M + d) % 2 == 0
    kw = dict(rs=0.5, bs=0.22, offset=1.0) if sandwich else {}
    gate = R.rand((M, d), seed + 4, xt) if sandwich else None
    h, r, eh, er = R.norm64(x, res, pre, post if sandwich else None, gate, **kw)
    got = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), post_weight=post.to(DEV) if sandwich else None,
                           gate=None if gate is None else gate.to(DEV), residual_scale=kw.get("rs", 1.0),
                           branch_scale=kw.get("bs", 1.0), weight_offset=kw.get("offset", 0.0), hidden_dtype=hidden)
    torch.cuda.synchronize()
    assert R.within(got.residual.cpu(), r, er, rt)
    assert got.hidden.dtype == hidden and (got.scales is None) == (hidden != E4)
    if hidden == E4:
        _check_e4m3(got.hidden.cpu(), got.scales.cpu(), h, eh)
    else:
        assert R.within(got.hidden.cpu(), h, eh, hidden)


# rows enough for CTAs that stay: whole warps of 512 columns and ragged ones, one
# warp a row and sixteen, runs of rows that begin and end inside a gate's rows
MANY = [(608, 512), (1001, 4096), (700, 1000), (611, 8), (640, 136), (616, 8192), (900, 5136), (1520, 1536)]


@pytest.mark.parametrize("M,d", MANY, ids=[f"M{m}_d{d}" for m, d in MANY])
@pytest.mark.parametrize("xt,rt,hidden", [(BF, FP, E4), (BF, BF, BF), (FP, FP, FP), (FP, BF, E4)])
@pytest.mark.parametrize("form", ["plain", "post", "gate", "both"])
def test_block_norm_many_rows(M, d, xt, rt, hidden, form):
    seed = 7 * M + d
    x, res = R.rand((M, d), seed, xt, 1.5), R.rand((M, d), seed + 1, rt, 4.0)
    wt = BF if form in ("plain", "both") else FP
    pre = R.rand((d,), seed + 2, wt, 0.3)
    post = R.rand((d,), seed + 3, wt, 0.3) if form in ("post", "both") else None
    G = next(g for g in (17, 16, 13, 11, 10, 9, 7) if M % g == 0)
    gate = R.rand((G, d), seed + 4, xt) if form in ("gate", "both") else None
    kw = dict(rs=0.5, bs=0.22, offset=1.0) if form == "both" else {}
    h, r, eh, er = R.norm64(x, res, pre, post, gate, **kw)
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    o = {k: Guarded(sh, t) for k, sh, t in (("out", (M, d), hidden), ("residual_out", (M, d), rt))}
    got = sv.sv_block_norm(dv(x), dv(res), dv(pre), post_weight=dv(post), gate=dv(gate),
                           residual_scale=kw.get("rs", 1.0), branch_scale=kw.get("bs", 1.0),
                           weight_offset=kw.get("offset", 0.0), hidden_dtype=hidden, **{k: g.t for k, g in o.items()})
    torch.cuda.synchronize()
    assert all(g.guards_intact() for g in o.values())
    assert R.within(got.residual.cpu(), r, er, rt)
    if hidden == E4:
        _check_e4m3(got.hidden.cpu(), got.scales.cpu(), h, eh)
    else:
        assert R.within(got.hidden.cpu(), h, eh, hidden)


def test_block_norm_many_rows_in_place_and_bad_rows():
    """In place, with rows of zeros, a NaN and an infinity among them: those
    stay in their rows."""
    M, d = 650, 1024
    x, res, pre = R.rand((M, d), 1, BF), R.rand((M, d), 2, BF), R.rand((d,), 3, BF)
    x[5], res[5] = 0, 0
    clean = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), hidden_dtype=E4)
    x[100, 17], x[300, 1000] = float("nan"), float("inf")
    buf = res.to(DEV)
    got = sv.sv_block_norm(x.to(DEV), buf, pre.to(DEV), hidden_dtype=E4, residual_out=buf)
    keep = torch.ones(M, dtype=torch.bool)
    keep[100] = keep[300] = False
    for k in ("hidden", "scales", "residual"):
        assert torch.equal(_bits(getattr(got, k))[keep], _bits(getattr(clean, k))[keep]), k
    assert (got.hidden[5].float() == 0).all() and (got.scales[5].cpu() == torch.tensor(R.AMAX_FLOOR) / 448).all()
    assert got.scales[100].isnan().all() and got.hidden[100].float().isnan().all()
    assert got.residual[300, 1000].isinf() and got.hidden[300].float()[1000].isnan()


@pytest.mark.parametrize("shape,gshape", [((4, 3, 96), (96,)), ((4, 3, 96), (4, 1, 96)), ((4, 3, 96), (4, 3, 96)),
                                          ((4, 3, 95), (4, 1, 95)), ((6, 64), (2, 64))])
def test_gate_rows_serve_consecutive_rows(shape, gshape):
    d = shape[-1]
    x, res, pre, gate = R.rand(shape, 1), R.rand(shape, 2), R.rand((d,), 3), R.rand(gshape, 4)
    h, r, eh, er = R.norm64(x.view(-1, d), res.view(-1, d), pre, None, gate)
    got = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), gate=gate.to(DEV), hidden_dtype=FP)
    assert got.hidden.shape == shape and got.residual.shape == shape
    assert R.within(got.residual.cpu().view(-1, d), r, er, FP)
    assert R.within(got.hidden.cpu().view(-1, d), h, eh, FP)


@pytest.mark.parametrize("d", [640, 641])
def test_block_norm_in_place_and_zero_rows(d):
    """residual_out may be residual; a row of zeros gives zeros (eps keeps
    the root from dividing by zero) and the smallest scale."""
    x, res, pre = R.rand((5, d), 1, BF), R.rand((5, d), 2, BF), R.rand((d,), 3, BF)
    x[2], res[2] = 0, 0
    ref = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), hidden_dtype=E4)
    buf = res.to(DEV)
    got = sv.sv_block_norm(x.to(DEV), buf, pre.to(DEV), hidden_dtype=E4, residual_out=buf)
    assert got.residual is buf
    for k in ("hidden", "scales", "residual"):
        assert torch.equal(_bits(getattr(got, k)), _bits(getattr(ref, k)))
    assert (got.hidden[2].float() == 0).all() and (got.residual[2] == 0).all()
    assert (got.scales[2].cpu() == torch.tensor(R.AMAX_FLOOR) / 448).all()


def test_block_norm_nan_stays_in_its_row():
    x, res, pre = R.rand((4, 300), 1), R.rand((4, 300), 2), R.rand((300,), 3)
    clean = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), hidden_dtype=E4)
    x[1, 17] = float("nan")
    x[2, 5] = float("inf")
    got = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), hidden_dtype=E4)
    for i in (0, 3):
        assert torch.equal(_bits(got.hidden[i]), _bits(clean.hidden[i]))
        assert torch.equal(_bits(got.scales[i]), _bits(clean.scales[i]))
    assert got.scales[1].isnan().all() and got.hidden[1].float().isnan().all()
    # an infinite r: the norm's factor is 0, so r * 0 is NaN there and 0 elsewhere
    assert got.residual[2, 5].isinf() and got.hidden[2].float()[5].isnan()


def test_block_norm_empty():
    e = torch.empty((0, 3, 64), device=DEV)
    got = sv.sv_block_norm(e, e, torch.ones(64, device=DEV), hidden_dtype=E4)
    assert got.hidden.shape == (0, 3, 64) and got.scales.shape == (0, 3, 1)


QSHAPES = [(1, 1), (5, 8), (3, 127), (4, 129), (130, 257), (128, 128), (129, 1040), (300, 999), (257, 4096)]


@pytest.mark.parametrize("M,d", QSHAPES, ids=[f"M{m}_d{d}" for m, d in QSHAPES])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize(M, d, dt, rows):
    """Bit for bit the documented fp32 steps, and within half an e4m3 step
    of the input in 64 bits."""
    x = (R.rand((M, d), M + d) * torch.exp(R.rand((M, 1), 5) * 3)).to(dt)
    v, s = sv.sv_quantize_fp8(x.to(DEV), rows)
    want_v, want_s = R.quantize_fp32(x, rows)
    assert torch.equal(_bits(s), _bits(want_s))
    assert torch.equal(_bits(v), _bits(want_v))
    sc = R.spread_scales(s.cpu().to(R.F64), rows, M, d)
    err = (v.cpu().to(R.F64) * sc - x.to(R.F64)).abs()
    assert (err <= 2.0 ** -4 * x.to(R.F64).abs() * (1 + 8 * R.U) + 2.0 ** -10 * sc).all()


@pytest.mark.parametrize("d", [384, 383])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_extremes(d, rows):
    """Zero, tiny, huge, infinite and NaN blocks."""
    x = R.rand((256, d), 9)
    x[:128, :128] = 0
    x[:128, 128:256] *= 1e-37
    x[128:, :128] = 3.0e38
    x[128:, 128:256] = float("nan")
    x[5, 300] = float("inf")
    v, s = sv.sv_quantize_fp8(x.to(DEV), rows)
    want_v, want_s = R.quantize_fp32(x, rows)
    v, s = v.cpu(), s.cpu()
    assert torch.equal(s.isnan(), want_s.isnan()) and torch.equal(s.nan_to_num(), want_s.nan_to_num())
    v, want_v = v.float(), want_v.float()
    assert torch.equal(v.isnan(), want_v.isnan()) and torch.equal(v.nan_to_num(), want_v.nan_to_num())


def test_quantize_shapes_and_empty():
    x = R.rand((3, 4, 200), 1).to(DEV)
    v, s = sv.sv_quantize_fp8(x)
    assert v.shape == x.shape and s.shape == (3, 4, 2)
    v2, s2 = sv.sv_quantize_fp8(x.view(12, 200))
    assert torch.equal(_bits(v).view(12, 200), _bits(v2)) and torch.equal(s.view(12, 2), s2)
    v, s = sv.sv_quantize_fp8(x[:0], 1)
    assert v.shape == (0, 4, 200) and s.shape == (0, 4, 2)


@pytest.mark.parametrize("d", [520, 523])
def test_only_the_outputs_are_written(d):
    """Guards around every output, on widths that end inside a segment."""
    M = 7
    x, res, pre = R.rand((M, d), 1, BF).to(DEV), R.rand((M, d), 2).to(DEV), R.rand((d,), 3, BF).to(DEV)
    nb = R.blocks(d)
    o = {k: Guarded(s, t) for k, s, t in (("out", (M, d), E4), ("scales", (M, nb), FP), ("residual_out", (M, d), FP))}
    sv.sv_block_norm(x, res, pre, hidden_dtype=E4, **{k: g.t for k, g in o.items()})
    q = {k: Guarded(s, t) for k, s, t in (("out", (M, d), E4), ("scales", (1, nb), FP))}
    sv.sv_quantize_fp8(x, 128, **{k: g.t for k, g in q.items()})
    torch.cuda.synchronize()
    assert all(g.guards_intact() for g in list(o.values()) + list(q.values()))


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows are the same as on their own."""
    M, d = 70001, 32768
    x = torch.zeros((M, d), dtype=BF, device=DEV)
    tail = R.rand((3, d), 4, BF).to(DEV)
    x[-3:] = tail
    v, s = sv.sv_quantize_fp8(x)
    tv, ts = sv.sv_quantize_fp8(tail)
    assert torch.equal(_bits(v[-3:]), _bits(tv)) and torch.equal(s[-3:].cpu(), ts.cpu())
    del v, s
    w = R.rand((d,), 5, BF).to(DEV)
    got = sv.sv_block_norm(x, x, w)
    ref = sv.sv_block_norm(tail, tail, w)
    assert torch.equal(_bits(got.hidden[-3:]), _bits(ref.hidden))
    assert torch.equal(_bits(got.residual[-3:]), _bits(ref.residual))


def test_many_rows_offsets_past_32_bits():
    """More than 2^31 values through the CTAs that stay."""
    M, d = 300001, 8192
    x = torch.zeros((M, d), dtype=BF, device=DEV)
    tail, w = R.rand((3, d), 4, BF), R.rand((d,), 5, BF)
    x[-3:] = tail.to(DEV)
    got = sv.sv_block_norm(x, x, w.to(DEV))
    h, r, eh, er = R.norm64(tail, tail, w)
    assert R.within(got.residual[-3:].cpu(), r, er, BF) and R.within(got.hidden[-3:].cpu(), h, eh, BF)
    assert int(got.hidden[:-3].count_nonzero()) == 0


def test_other_stream_and_captured_graph():
    x, res, pre = R.rand((6, 900), 1, BF).to(DEV), R.rand((6, 900), 2, BF).to(DEV), R.rand((900,), 3, BF).to(DEV)
    want = sv.sv_block_norm(x, res, pre, hidden_dtype=E4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.sv_block_norm(x, res, pre, hidden_dtype=E4, stream=side)
    qv, qs = sv.sv_quantize_fp8(x, stream=side)
    side.synchronize()
    assert torch.equal(_bits(got.hidden), _bits(want.hidden)) and torch.equal(got.scales, want.scales)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = sv.sv_block_norm(x, res, pre, hidden_dtype=E4)
        cv, cs = sv.sv_quantize_fp8(x)
    for k in range(2):
        x.copy_(R.rand((6, 900), 10 + k, BF))
        g.replay()
        want = sv.sv_block_norm(x, res, pre, hidden_dtype=E4)
        wv, ws = sv.sv_quantize_fp8(x)
        torch.cuda.synchronize()
        assert torch.equal(_bits(cap.hidden), _bits(want.hidden)) and torch.equal(cap.scales, want.scales)
        assert torch.equal(_bits(cap.residual), _bits(want.residual))
        assert torch.equal(_bits(cv), _bits(wv)) and torch.equal(cs, ws)
