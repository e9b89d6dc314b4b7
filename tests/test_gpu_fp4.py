"""Microscaled 4-bit floating point on the GPU: quantisation and reading back,
bit for bit, and the LM head on such operands."""
import numpy as np
import pytest
import torch

import draft_ref as R
import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _x(M, d, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, d), generator=g) * torch.exp(2 * torch.randn((M, 1), generator=g))
    return x.to(dtype)


def _check_quantized(x, block, t):
    v, s, g = R.quantize(x.double().numpy(), block)
    got = R.unpack(t.values.cpu().reshape(-1, x.shape[-1] // 2).numpy())
    bad = np.repeat(np.isnan(s), block, 1)[:, :x.shape[-1]]
    assert np.array_equal(got, np.where(bad, 0.0, v))
    want = R.tile(s)
    have = t.scales.cpu()
    if block == 32:
        byte = have.view(torch.uint8).numpy().astype(np.float64)
        have = np.where(byte == 255, np.nan, 2.0 ** (byte - 127))
        want = np.where(want == 0, 2.0 ** -127, want)       # a byte of 0 stands for 2^-127
    else:
        have = have.float().double().numpy()
    assert np.array_equal(have, want, equal_nan=True)
    if block == 16:
        assert np.array_equal(t.row_scales.cpu().double().numpy().reshape(-1), g)
    # read back: value * scale is exact in fp32, and so is its product with a power of two
    full = v * np.repeat(s, block, 1)[:, :x.shape[-1]]
    if block == 16:
        full = full * g[:, None]
    f32 = sv.sv_dequantize_fp4(t, F32).cpu().double().numpy().reshape(full.shape)
    assert np.array_equal(np.where(bad, 0, f32), np.where(bad, 0, full))
    assert np.isnan(f32[bad]).all()
    b16 = sv.sv_dequantize_fp4(t).cpu().double().numpy().reshape(full.shape)
    assert np.array_equal(np.where(bad, 0, b16), np.where(bad, 0, full))  # 6 significant bits


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,d", [(1, 2), (3, 16), (5, 30), (40, 4096), (129, 200), (7, 1000), (256, 64), (2, 9000),
                                 (130, 8192), (33, 514)])
def test_quantize_bits(block, dtype, M, d):
    x = _x(M, d, dtype, seed=M + d)
    _check_quantized(x, block, sv.sv_quantize_fp4(x.to(DEV), block))


@pytest.mark.parametrize("block", [16, 32])
def test_quantize_special_values(block):
    x = _x(140, 256, F32, seed=9)
    x[1] = 0
    x[2, :100] = 0
    x[3, 17] = float("nan")
    x[4, 40] = float("inf")
    x[5, 255] = -float("inf")
    x[6] = float("nan")
    x[7] *= 1e30
    x[8] *= 1e-30
    x[9] = 1e-40                 # below the normal range
    x[10] = 3e38
    x[11, :] = -0.0
    x[12] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]).repeat(32)   # ties of the e2m1 grid at scale 1
    x[13] = 2688.0
    x[14] = 2688.0 * 2 ** -3
    x[15, 0] = 1e20              # the others far below a scale's range
    x[16] = torch.tensor([1.0, 1.0625, 1.1875, 1.3125] * 64)
    _check_quantized(x, block, sv.sv_quantize_fp4(x.to(DEV), block))


def test_quantize_alignment_leading_dims_and_out():
    x = _x(3 * 5, 64, BF).view(3, 5, 64).to(DEV)
    t = sv.sv_quantize_fp4(x)
    assert t.values.shape == (3, 5, 32) and t.row_scales.shape == (3, 5) and t.scales.shape == (1, 1, 32, 4, 4)
    _check_quantized(x.cpu().view(15, 64), 16, t)
    # a base that is aligned to its elements only
    buf = torch.zeros(15 * 64 + 1, dtype=BF, device=DEV)
    odd = buf[1:].view(15, 64)
    odd.copy_(x.view(15, 64))
    assert torch.equal(sv.sv_quantize_fp4(odd).values, t.values.view(15, 32))
    # ... and so for rows that are no whole octets, in and out
    for dtype in (BF, F32):
        y = _x(9, 214, dtype, seed=2)
        buf = torch.zeros(9 * 214 + 1, dtype=dtype, device=DEV)
        odd = buf[1:].view(9, 214)
        odd.copy_(y)
        q = sv.sv_quantize_fp4(odd)
        _check_quantized(y, 16, q)
        shifted = torch.zeros(9 * 214 + 3, dtype=dtype, device=DEV)
        sv.sv_dequantize_fp4(q, dtype, out=shifted[1:-2].view(9, 214))
        assert torch.equal(shifted[1:-2].view(9, 214), sv.sv_dequantize_fp4(q, dtype))
        assert not shifted[0] and not shifted[-2:].any()
    again = sv.sv_quantize_fp4(2 * x, out=t)
    assert again is t
    _check_quantized(2 * x.cpu().view(15, 64), 16, t)
    back = torch.empty((3, 5, 64), dtype=F32, device=DEV)
    assert sv.sv_dequantize_fp4(t, F32, out=back) is back and torch.equal(back, sv.sv_dequantize_fp4(t, F32))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,d", [(5, 30), (130, 256), (3, 9000)])
def test_nothing_is_written_beside_the_outputs(block, M, d):
    x = _x(M, d, BF).to(DEV)
    n = -(-M // 128) * -(-d // (4 * block)) * 512
    v = torch.full((M * (d // 2) + 128,), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((n + 128,), 0xA5, dtype=torch.uint8, device=DEV)
    g = torch.full((M + 2,), 77.0, device=DEV)
    t = sv.Fp4Tensor(v[64:-64].view(M, d // 2),
                     s[64:-64].view(torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu).view(
                         -(-M // 128), -(-d // (4 * block)), 32, 4, 4), g[1:-1] if block == 16 else None)
    sv.sv_quantize_fp4(x, block, out=t)
    _check_quantized(x.cpu(), block, t)
    for b in (v, s):
        assert (b[:64] == 0xA5).all() and (b[-64:] == 0xA5).all()
    assert g[0] == 77 and g[-1] == 77
    out = torch.full((M * d + 16,), 77.0, dtype=BF, device=DEV)
    sv.sv_dequantize_fp4(t, out=out[8:-8].view(M, d))
    assert (out[:8] == 77).all() and (out[-8:] == 77).all()


def test_no_rows():
    for block in (16, 32):
        t = sv.sv_quantize_fp4(torch.empty((0, 64), device=DEV), block)
        assert t.values.shape == (0, 32) and sv.sv_dequantize_fp4(t).shape == (0, 64)
        w = sv.sv_quantize_fp4(torch.randn((9, 64), device=DEV), block)
        assert sv.sv_lm_head_logits_fp4(t, w).shape == (0, 9)


def test_row_scales_of_a_checkpoint():
    """Any fp32 row scales: one rounding in fp32, one to bf16."""
    x = _x(20, 96, F32, seed=3).to(DEV)
    t = sv.sv_quantize_fp4(x)
    u = sv.Fp4Tensor(t.values, t.scales, t.row_scales * 0.37)
    want = sv.sv_dequantize_fp4(sv.Fp4Tensor(t.values, t.scales, torch.ones_like(t.row_scales)), F32) * u.row_scales[:, None]
    assert torch.equal(sv.sv_dequantize_fp4(u, F32), want)
    assert torch.equal(sv.sv_dequantize_fp4(u), want.to(BF))


# ------------------------------------------------------------------ the LM head

def _operand(M, d, block, seed, exact=False):
    r = np.random.default_rng(seed)
    nb = -(-d // block)
    if exact:  # products and their sums are exact in fp32, in any order
        v = r.choice([-1.0, -0.5, 0.0, 0.5, 1.0], (M, d))
        s = r.choice([0.5, 1.0, 2.0], (M, nb))
        g = r.choice([0.25, 1.0, 2.0], M)
    else:
        v = R.E2M1[r.integers(0, 8, (M, d))] * r.choice([-1.0, 1.0], (M, d))
        s = R.round_e4m3(np.exp(r.normal(0, 1, (M, nb)))) if block == 16 else 2.0 ** r.integers(-4, 5, (M, nb))
        g = np.float32(np.exp(r.normal(0, 1, M))).astype(np.float64)
    return v, s, g if block == 16 else None


def _head(M, V, d, block, seed=0, exact=False):
    h, w = _operand(M, d, block, seed, exact), _operand(V, d, block, seed + 1, exact)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    z = sv.sv_lm_head_logits_fp4(R.to_device(sv, *h, block), R.to_device(sv, *w, block), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want, mag = R.head(*h, *w, block)
    return z.cpu().double().numpy(), want, mag


# tiles of 64, 128 and 192 ids, alone, in pairs and with two row tiles a pair; rows that fill no tile; vocabularies that end inside a tile and are
# no multiple of 8; a last stage of 32 to 224 dims
SHAPES = [(1, 100, 32), (1, 5000, 256), (5, 1, 64), (8, 777, 96), (17, 2048, 1024), (64, 4100, 288), (127, 300, 544),
          (128, 20000, 256), (129, 1000, 480), (131, 3203, 1056), (200, 30000, 128), (257, 4096, 512), (513, 515, 224),
          (300, 15001, 64), (600, 9000, 288), (1030, 21000, 64), (520, 30001, 512)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,V,d", SHAPES)
def test_head_exact(block, M, V, d):
    """Operands whose products add up exactly: the logits have one right value."""
    z, want, _ = _head(M, V, d, block, seed=M + V + d, exact=True)
    want = torch.from_numpy(want).to(BF).double().numpy()
    assert np.array_equal(z, want)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,V,d", [(3, 700, 4096), (131, 3203, 1056), (300, 2000, 2048)])
def test_head_random(block, M, V, d):
    z, want, mag = _head(M, V, d, block, seed=d)
    # half a bf16 step; fp32 sums of d products in any order and the two roundings of the factors, with a factor of
    # two for sums that the tensor cores cut off instead of rounding
    tol = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 2 * (d + 4) * 2.0 ** -24 * mag
    assert (np.abs(z - want) <= tol).all()


def test_head_leading_dims_out_and_unaligned_rows():
    h, w = _operand(12, 64, 16, 5, True), _operand(203, 64, 16, 6, True)
    want = torch.from_numpy(R.head(*h, *w, 16)[0]).to(BF)
    ht, wt = R.to_device(sv, *h, 16, lead=(3, 4)), R.to_device(sv, *w, 16)
    assert torch.equal(sv.sv_lm_head_logits_fp4(ht, wt).cpu(), want.view(3, 4, 203))
    buf = torch.zeros(12 * 203 + 9, dtype=BF, device=DEV)
    out = buf[1:1 + 12 * 203].view(3, 4, 203)
    assert sv.sv_lm_head_logits_fp4(ht, wt, out=out) is out
    assert torch.equal(out.cpu(), want.view(3, 4, 203)) and not buf[0] and not buf[1 + 12 * 203:].any()


def test_head_nan_and_overflow_stay_where_they_belong():
    M, V, d = 70, 400, 128
    h, w = _operand(M, d, 16, 7, True), _operand(V, d, 16, 8, True)
    want = torch.from_numpy(R.head(*h, *w, 16)[0]).to(BF)
    ht, wt = R.to_device(sv, *h, 16), R.to_device(sv, *w, 16)
    b = ht.scales.view(torch.uint8)
    b[0, 0, 33 % 32, 33 // 32, 2] = 0x7F          # row 33, block 2
    wt.scales.view(torch.uint8)[2, 1, 300 % 32, 300 % 128 // 32, 1] = 0x7F   # id 300, block 5
    ht.row_scales[50] = float("inf")
    wt.row_scales[7] = float("nan")
    ht.row_scales[60] = 3e38
    wt.row_scales[200] = 3e38                     # the product of the two leaves the range
    z = sv.sv_lm_head_logits_fp4(ht, wt).cpu()
    nan = torch.zeros((M, V), dtype=torch.bool)
    nan[33], nan[50], nan[:, 300], nan[:, 7], nan[60, 200] = True, True, True, True, True
    assert not torch.isinf(z[:60]).any() and torch.isnan(z[nan]).all()
    other = ~nan
    other[60], other[:, 200] = False, False
    assert torch.equal(z[other], want[other])


def test_head_graph_and_streams():
    h, w = _operand(40, 256, 16, 11, True), _operand(3001, 256, 16, 12, True)
    want = torch.from_numpy(R.head(*h, *w, 16)[0]).to(BF)
    ht, wt = R.to_device(sv, *h, 16), R.to_device(sv, *w, 16)
    sv.sv_lm_head_logits_fp4(ht, wt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = sv.sv_lm_head_logits_fp4(ht, wt, stream=side)
    b = sv.sv_lm_head_logits_fp4(ht, wt)
    torch.cuda.synchronize()
    assert torch.equal(a.cpu(), want) and torch.equal(b.cpu(), want)
    x = torch.randn((40, 256), device=DEV, dtype=BF)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = sv.sv_lm_head_logits_fp4(sv.sv_quantize_fp4(x), wt)
    for seed in (1, 2):
        x.copy_(_x(40, 256, BF, seed=seed))
        g.replay()
        assert torch.equal(z, sv.sv_lm_head_logits_fp4(sv.sv_quantize_fp4(x), wt))
