"""4-bit operands at the ends of the floating-point ranges: signs of zeros, logits that
bf16 cannot hold, row scales whose product leaves fp32's range."""
import numpy as np
import pytest
import torch

import draft_ref as R
import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "fp32"])
def test_zeros_keep_their_sign(block, dtype):
    """-0 and negative values that round to zero are e2m1's -0, in both kinds of blocks; reading back keeps it."""
    x = torch.randn((40, 96), generator=torch.Generator().manual_seed(8)).to(dtype)
    x[:, ::5] = 0.0
    x[:, ::7] = -0.0
    x[:, 3::11] = -1e-6
    x[5] = -0.0
    t = sv.sv_quantize_fp4(x.to(DEV), block)
    code = torch.stack((t.values & 15, t.values >> 4), -1).view(40, 96).cpu()
    assert torch.equal(code > 7, torch.signbit(x))
    v, _, _ = R.quantize(x.double().numpy(), block)
    assert np.array_equal(R.unpack(t.values.cpu().numpy()), v)
    for out in (BF, torch.float32):
        assert torch.equal(torch.signbit(sv.sv_dequantize_fp4(t, out).cpu()), torch.signbit(x))


def _single(products, gh, gw):
    """Operands of which row m's and id v's only product is products[m] (a sum of one e2m1 value and one scale), with
    row scales gh [M], gw [V]."""
    M, V, d = len(gh), len(gw), 64
    hv, hs, wv, ws = np.zeros((M, d)), np.ones((M, 4)), np.zeros((V, d)), np.ones((V, 4))
    hv[:, 5] = products
    wv[:, 5] = 1.0
    return R.to_device(sv, hv, hs, np.asarray(gh), 16), R.to_device(sv, wv, ws, np.asarray(gw), 16)


def test_logits_next_to_the_largest_are_never_infinite():
    """What bf16 cannot hold is NaN, from where it would round to an infinity on."""
    top = 2.0 ** 128 * (1 - 2.0 ** -9)              # halfway from bf16's largest value to 2^128
    below = float(np.nextafter(np.float32(top), np.float32(0)))
    gh = [top, below, 3.4028234e38, 3.39e38, 1.0, top / 2]
    # (9 ids: plain stores; 128: tensor stores)
    for V in (9, 128):
        gw = [1.0] * V
        gw[3] = -1.0
        ht, wt = _single([1.0] * 6, gh, gw)
        z = sv.sv_lm_head_logits_fp4(ht, wt).cpu().double().numpy()
        assert not np.isinf(z).any()
        assert np.isnan(z[[0, 2]]).all() and not np.isnan(z[[1, 3, 4, 5]]).any()
        sign = np.asarray(gw)
        big = float(torch.finfo(BF).max)
        assert np.array_equal(z[1], big * sign) and np.array_equal(z[4], sign) and np.array_equal(z[5], 2.0 ** 127 * sign)
        assert np.array_equal(z[3], float(torch.tensor(3.39e38).to(BF)) * sign)
        # an accepted row of logits is one that the draw accepts
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = sv.sv_sample_logits(torch.from_numpy(z).to(BF).to(DEV), torch.full((6,), 0.5, device=DEV), 1.0, status=status)
        assert (r.tokens.cpu()[[0, 2]] == -1).all() and (r.tokens.cpu()[[1, 3, 4, 5]] >= 0).all()
        assert int(status.item()) == sv.SV_BAD_ROW


def test_row_scales_whose_product_leaves_the_range():
    """The product of three factors is right wherever it is in range, whatever two of them come to: it is rounded to
    fp32 at most twice and once to bf16."""
    hv = np.array([0.0, 0.5, 1.0, -6.0, 2.0, 4.0])
    for V in (130, 136):
        gh = np.float32([3e38, 3e38, 1e-30, 1e-30, 1e38, 2.0 ** -140]).astype(np.float64)
        gw = np.ones(V)
        gw[:8] = np.float32([3e38, 4.0, 1e-15, 1e-10, 2.0 ** -130, 1e-38, 2.0 ** 120, 1e30]).astype(np.float64)
        ht, wt = _single(hv, gh, gw)
        z = sv.sv_lm_head_logits_fp4(ht, wt).cpu().double().numpy()
        want = hv[:, None] * gh[:, None] * gw[None]
        over = np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -9)
        assert np.isnan(z[over]).all() and not np.isnan(z[~over]).any()
        # half a bf16 step (2^-8 of the value; 2^-134 below the normal range) and two of fp32's
        tol = np.abs(want) * (2.0 ** -8 + 2.0 ** -22) + 2.0 ** -134 + 2.0 ** -148
        assert [(i, z[i], want[i]) for i in zip(*np.nonzero(~over)) if abs(z[i] - want[i]) > tol[i]] == []
    # sums of many products: the largest that operands in 4 bits have, with factors whose own product is subnormal
    d = 128
    v, s = np.full((3, d), 6.0), np.full((3, 8), 448.0)
    gh, gw = np.float64(np.float32([1e-30, 1e-30, 1e-38])), np.float64(np.float32([1e-15, 1e-12, 1e-7]))
    z = sv.sv_lm_head_logits_fp4(R.to_device(sv, v, s, gh, 16), R.to_device(sv, v, s, gw, 16)).cpu().double().numpy()
    want = d * (6.0 * 448) ** 2 * gh[:, None] * gw[None]
    assert (np.abs(z - want) <= want * (2.0 ** -8 + 2.0 ** -21) + 2.0 ** -134 + 2.0 ** -148).all()


def test_a_row_does_not_depend_on_others_row_scales():
    """Ordinary rows beside rows with extreme factors, and alone: bit for bit."""
    M, V, d = 40, 300, 256
    g = torch.Generator(device=DEV).manual_seed(6)
    ht, wt = (sv.sv_quantize_fp4(torch.randn((n, d), generator=g, device=DEV)) for n in (M, V))
    plain = sv.sv_lm_head_logits_fp4(ht, wt)
    odd_h, odd_w = ht.row_scales.clone(), wt.row_scales.clone()
    odd_h[7], odd_h[8], odd_h[33] = 3e38, 1e-44, float("nan")
    odd_w[5], odd_w[70], odd_w[299] = 1e-40, 2e38, float("inf")
    mixed = sv.sv_lm_head_logits_fp4(sv.Fp4Tensor(ht.values, ht.scales, odd_h), sv.Fp4Tensor(wt.values, wt.scales, odd_w))
    rows = [i for i in range(M) if i not in (7, 8, 33)]
    ids = [i for i in range(V) if i not in (5, 70, 299)]
    assert torch.equal(mixed[rows][:, ids], plain[rows][:, ids])
    assert not torch.isinf(mixed).any() and torch.isnan(mixed[33]).all() and torch.isnan(mixed[:, 299]).all()
