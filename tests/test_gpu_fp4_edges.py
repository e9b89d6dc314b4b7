"""4-bit operands where a CTA walks many rows, where a pair forms two row tiles
from one tile of W, and at more elements than 32 bits count."""
import numpy as np
import pytest
import torch

import draft_ref as R
import fp4_shapes as S
import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ quantisation

def _rows_of(t, rows, d, block):
    """Values, scales and row scales of some rows of t, in 64 bits."""
    i = torch.from_numpy(rows).to(DEV)
    v = R.unpack(t.values[i].cpu().numpy())
    sc = t.scales.view(torch.uint8)[i // 128, :, i % 32, i % 128 // 32].reshape(len(rows), -1)[:, :-(-d // block)].cpu()
    if block == 16:
        return v, sc.contiguous().view(torch.float8_e4m3fn).double().numpy(), t.row_scales[i].cpu().double().numpy()
    return v, 2.0 ** (sc.double().numpy() - 127), None


# sizes by the warps of a row (1, 2, 4, 8, 8 with more octets than a lane keeps): each CTA takes several rows of its
# own after the other; whole octets and others
MANY = [(9001, 64), (9001, 66), (3000, 2000), (3000, 1990), (2500, 4096), (1300, 8192), (1300, 9000), (1300, 9002)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,d", MANY)
def test_many_rows_of_a_cta(block, dtype, M, d):
    """Rows whose sizes differ by many octaves, so that another row's maximum or values would show: all of them
    against calls of 128 rows, a share of them against the plain form."""
    g = torch.Generator(device=DEV).manual_seed(M + d)
    x = (torch.randn((M, d), generator=g, device=DEV) * torch.exp2(torch.randint(-30, 31, (M, 1), generator=g, device=DEV))).to(dtype)
    t = sv.sv_quantize_fp4(x, block)
    for i in range(0, M, 128):
        p = sv.sv_quantize_fp4(x[i:i + 128], block)
        assert torch.equal(t.values[i:i + 128], p.values), i
        assert torch.equal(t.scales[i // 128].view(torch.uint8), p.scales[0].view(torch.uint8)), i
        if block == 16:
            assert torch.equal(t.row_scales[i:i + 128], p.row_scales), i
    rows = np.unique(np.concatenate([np.arange(M - 40, M), np.arange(0, M, 61)]))
    v, s, gs = R.quantize(x[torch.from_numpy(rows).to(DEV)].double().cpu().numpy(), block)
    hv, hs, hg = _rows_of(t, rows, d, block)
    assert np.array_equal(hv, v) and np.array_equal(hs, s)
    if block == 16:
        assert np.array_equal(hg, gs)


def test_quantized_and_read_back_behind_2_to_the_31():
    """540000 rows of 4096: more values than 32 bits count."""
    M, d = 540000, 4096
    x = torch.empty((M, d), dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    for i in range(0, M, 30000):
        x[i:i + 30000] = torch.randn((30000, d), generator=g, device=DEV)
    for block in (16, 32):
        t = sv.sv_quantize_fp4(x, block)
        back = sv.sv_dequantize_fp4(t)
        for i in (0, 262144 * 2, 539904):
            p = sv.sv_quantize_fp4(x[i:i + 128].clone(), block)
            assert torch.equal(t.values[i:i + 128], p.values)
            assert torch.equal(t.scales[i // 128].view(torch.uint8), p.scales[0].view(torch.uint8))
            assert torch.equal(back[i:i + 128], sv.sv_dequantize_fp4(p))


# ------------------------------------------------------------------ the LM head

def _operand(M, d, block, seed, exact):
    r = np.random.default_rng(seed)
    nb = -(-d // block)
    if exact:  # products are multiples of 2^-8 and their sums below 2^14: exact in fp32, in any order
        v = r.choice(np.array([-1.0, -0.5, 0.0, 0.5, 1.0]), (M, d))
        s = r.choice([0.5, 1.0, 2.0], (M, nb))
        g = r.choice([0.25, 1.0, 2.0], M)
    else:
        v = R.E2M1[r.integers(0, 8, (M, d))] * r.choice([-1.0, 1.0], (M, d))
        s = R.round_e4m3(np.exp(r.normal(0, 1, (M, nb)))) if block == 16 else 2.0 ** r.integers(-4, 5, (M, nb))
        g = np.float32(np.exp(r.normal(0, 1, M))).astype(np.float64)
    return v, s, g if block == 16 else None


def _full(v, s, g, block):
    f = torch.from_numpy(v).to(DEV) * torch.from_numpy(s).to(DEV).repeat_interleave(block, 1)[:, :v.shape[1]]
    return f if g is None else f * torch.from_numpy(np.asarray(g)).to(DEV)[:, None]


@pytest.mark.parametrize("exact", [True, False], ids=["exact", "random"])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,V,d", S.LONE + S.PAIR + S.TWO)
def test_head_shapes(M, V, d, block, exact):
    """Each shape of the product, d of seven stages and more, so that a unit's ring comes round inside a tile and
    from a tile to the next."""
    if not exact and (M, V, d) not in (S.PAIR[0], S.TWO[0], S.TWO[1]):
        V = V // 4 + V % 4    # (few sizes are enough of the sums' roundings)
    h, w = _operand(M, d, block, M + d, exact), _operand(V, d, block, V + d, exact)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    z = sv.sv_lm_head_logits_fp4(R.to_device(sv, *h, block), R.to_device(sv, *w, block), status=status)
    a, b = _full(*h, block), _full(*w, block)
    want = a @ b.T
    assert int(status.item()) == 0
    if exact:
        assert torch.equal(z, want.float().to(BF))
    else:
        # half a bf16 step; fp32 sums of d products in any order and the two roundings of the factors, twice over for
        # sums that are cut off instead of rounded
        tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -7) + 2 * (d + 4) * 2.0 ** -24 * (a.abs() @ b.abs().T)
        assert ((z.double() - want).abs() <= tol).all()


def test_head_behind_2_to_the_31():
    """17000 x 131072 logits: stores behind element 2^31, against calls of those rows alone; an odd vocabulary's plain
    stores likewise."""
    M, d = 17000, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn((M, d), generator=g, device=DEV)
    for V in (131072, 131077):
        w = sv.sv_quantize_fp4(torch.randn((V, d), generator=g, device=DEV))
        z = sv.sv_lm_head_logits_fp4(sv.sv_quantize_fp4(x), w)
        for i in (0, 16300, M - 60):
            part = sv.sv_lm_head_logits_fp4(sv.sv_quantize_fp4(x[i:i + 60].contiguous()), w)
            # (sums of 64 products: one MMA, the same in every shape)
            assert torch.equal(z[i:i + 60], part), i
