"""The 4-bit LM head at the ends of the floating-point ranges: what bf16 cannot
hold, row scales whose product leaves fp32's range."""
import numpy as np
import pytest
import torch

import draft_ref as R
import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


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
