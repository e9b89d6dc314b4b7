"""The draw of tokens where roundings of z - max would show, and at more
elements than 32 bits count: logits of very different size in one row, rows at
both sides of the largest max / T that is multiplied out, uniforms next to an
id's boundary."""
import numpy as np
import pytest
import torch

import draft_ref as R
import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# A mass is 2^27 2^(j / 32) e^x in whole numbers: half of one lost in the table, half in the product, and 2^-28.4 of
# the mass by r, the series and the table's fp32 entry: eps <= 1.4 * 2^-27.  A boundary's place c in the row moves by
# at most c (1 - c) 2 eps <= 0.7 * 2^-27.
NEAR = 2.0 ** -27       # of the mass: nearer to a boundary a draw may fall on either side
FAR = 2.0 ** -25


def _uniforms_at_boundaries(z, T, n, seed):
    """n uniforms whose u sum(w) lies NEAR to FAR from an id's boundary (or the nearest above NEAR), the ids spread
    over the row; the tokens in 64 bits.  The boundaries are those of the unfiltered row."""
    w = np.exp((z.astype(np.float64) - z.max()) / float(np.float32(T)))
    cdf = np.cumsum(w)
    cdf /= cdf[-1]
    r = np.random.default_rng(seed)
    at = np.concatenate([np.arange(1, min(9, z.size)), r.permutation(z.size - 1)])
    us, tokens = [], []
    for i in at:
        if not 2.0 ** -8 < cdf[i] < 1 - 2.0 ** -8:
            continue
        for u in (np.float32(cdf[i]), np.nextafter(np.float32(cdf[i]), np.float32(2)),
                  np.nextafter(np.float32(cdf[i]), np.float32(-1))):
            d = np.abs(cdf[max(0, i - 3):i + 4] - float(u)).min()
            if NEAR < d < FAR:
                us.append(u)
                tokens.append(int((cdf <= float(u)).sum()))
                break
        if len(us) == n:
            break
    return np.array(us, np.float32), np.array(tokens)


def _row(kind, V, dtype, seed=0):
    r = np.random.default_rng(seed)
    if kind == "large-max":         # one large logit, the others sixteen octaves and more below it
        z = r.uniform(3.5e-7, 4.5e-7, V)
        z[V // 2] = 10.5
    elif kind == "small-max":       # the maximum far below the others' size
        z = np.where(r.random(V) < 0.5, -3.0, -5.0)
        z[V // 3] = 3e-7
    elif kind == "both":            # ordinary logits, and many next to 0
        z = r.normal(0, 1.5, V)
        z[r.random(V) < 0.7] *= 1e-6
        z[V // 5] = 9.0
    else:
        z = r.normal(0, 2.0, V)
    return torch.from_numpy(z).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["large-max", "small-max", "both", "normal"])
def test_boundaries_of_logits_of_different_size(dtype, kind):
    """Masses are as right whatever the logits' exponents, so a uniform further than NEAR from a boundary draws the
    token of exact arithmetic."""
    V, T = 60000, 1.0
    z = _row(kind, V, dtype)
    u, tokens = _uniforms_at_boundaries(z.double().numpy(), T, 256, 1)
    assert len(u) >= 200
    rows = z.to(DEV).expand(len(u), V).contiguous()
    ud = torch.from_numpy(u).to(DEV)
    r = sv.sv_sample_logits(rows, ud, T)
    assert np.array_equal(r.tokens.cpu().numpy(), tokens)
    few = sv.sv_sample_logits(rows[:7], ud[:7], T, 0, 1.0, 1e-30)    # (min-p takes nothing away)
    assert np.array_equal(few.tokens.cpu().numpy(), tokens[:7])


@pytest.mark.parametrize("mx", [45.0, 45.3, 45.5, 60.0, -45.3, -60.0, 1000.0, 2.0 ** -20, 0.0])
def test_boundaries_at_large_max_over_T(mx):
    """32 log2(e) max / T on both sides of 2^21 (max / T = 45426), positive and negative."""
    V, T = 5000, 1e-3
    r = np.random.default_rng(3)
    z = (mx - T * np.abs(r.normal(0, 3.0, V))).astype(np.float32)
    z[77] = mx
    u, tokens = _uniforms_at_boundaries(z, T, 64, 2)
    assert len(u) >= 48
    rows = torch.from_numpy(z).to(DEV).expand(len(u), V).contiguous()
    assert np.array_equal(sv.sv_sample_logits(rows, torch.from_numpy(u).to(DEV), T).tokens.cpu().numpy(), tokens)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("filt", [dict(top_k=50, top_p=0.9), dict(top_p=0.95), dict(min_p=0.01), dict()],
                         ids=lambda f: ",".join(f) or "none")
def test_rows_are_compared(dtype, filt):
    """Cuts, q and draws of rows of mixed sizes; nine rows of ten at least are decided and compared."""
    V, n = 12000, 24
    z = torch.stack([_row(k, V, dtype, s) for s in range(n // 4) for k in ("large-max", "small-max", "both", "normal")])
    u = np.random.default_rng(5).random(n, dtype=np.float32)
    r = sv.sv_sample_logits(z.to(DEV), torch.from_numpy(u).to(DEV), 0.9, filt.get("top_k", 0), filt.get("top_p", 1.0),
                            filt.get("min_p", 0.0), want_probs=True)
    compared = 0
    for i in range(n):
        token, keep, q, margin = R.sample(z[i].double().numpy(), float(u[i]), 0.9, **filt)
        if margin < NEAR:
            continue
        compared += 1
        assert int(r.kept[i]) == keep.sum() and int(r.tokens[i]) == token
        p = r.probs[i].cpu().double().numpy()
        # exp2 in fp32 of a rounded argument of up to 64, and three roundings
        assert (np.abs(p - q) <= 2.0 ** -17 * q + 2.0 ** -126).all() and not p[~keep].any()
        assert abs(float(r.prob[i]) - q[token]) <= 2.0 ** -23 * q[token] + 2.0 ** -40 * q.max()
    assert compared >= 0.9 * n


def test_more_elements_than_32_bits_count():
    """17000 rows of 131072: rows behind element 2^31 of logits and of q, against calls of those rows alone."""
    rows, V = 17000, 131072
    z = torch.empty((rows, V), dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for i in range(0, rows, 1000):
        z[i:i + 1000] = torch.randn((1000, V), generator=g, device=DEV) * 3
    u = torch.rand(rows, generator=g, device=DEV)
    r = sv.sv_sample_logits(z, u, 0.8, 100, 0.9, want_probs=True)
    for i in (0, 8191, 16384, 16900, rows - 20):
        part = sv.sv_sample_logits(z[i:i + 20].clone(), u[i:i + 20].clone(), 0.8, 100, 0.9, want_probs=True)
        for name in ("tokens", "prob", "kept", "probs"):
            assert torch.equal(getattr(r, name)[i:i + 20], getattr(part, name)), (name, i)
