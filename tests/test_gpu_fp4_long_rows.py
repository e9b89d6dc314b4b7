"""Rows so long that the offsets of their scales pass 32 bits."""
import pytest
import torch

import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("block,more", [(16, 4096 + 66), (32, 4096 + 64)])
def test_row_whose_scales_pass_2_to_the_31(block, more):
    """One row of 2^28 (blocks of 32: 2^29) values and some more, against calls of its parts as rows of 4096, which
    have the same row scale because each holds the row's maximum.  The buffers' surroundings stay as they were."""
    L, d = 4096, (1 << (28 if block == 16 else 29)) + more
    n = d // L
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.empty((1, d), dtype=torch.bfloat16, device=DEV)
    for i in range(0, d, 1 << 26):
        x[0, i:i + (1 << 26)] = torch.randn(min(1 << 26, d - i), generator=g, device=DEV)
    x[0, ::L] = 9.0
    kt = -(-d // (4 * block))
    values = torch.full((64 + d // 2 + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full(((1 << 16) + kt * 512 + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    out = sv.Fp4Tensor(values[64:-64].view(1, d // 2), scales[1 << 16:-512].view(
        torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu).view(1, kt, 32, 4, 4),
        torch.empty(1, device=DEV) if block == 16 else None)
    sv.sv_quantize_fp4(x, block, out=out)
    assert (values[:64] == 0xA5).all() and (values[-64:] == 0xA5).all()
    assert (scales[:1 << 16] == 0xA5).all() and (scales[-512:] == 0xA5).all()
    tiles = out.scales.view(torch.uint8)[0]                         # [kt, 32, 4, 4]
    per = L // (4 * block)
    assert not tiles[:, 1:].any() and not tiles[:, :, 1:].any()     # rows 1 .. 127 of the tiles
    for i in range(0, n, 1 << 13):                                  # parts of 8192 rows of 4096
        m = min(1 << 13, n - i)
        p = sv.sv_quantize_fp4(x[0, i * L:(i + m) * L].view(m, L), block)
        assert torch.equal(out.values[0, i * L // 2:(i + m) * L // 2].view(m, L // 2), p.values), i
        rows = torch.arange(m, device=DEV)
        want = p.scales.view(torch.uint8)[rows // 128, :, rows % 32, rows % 128 // 32]      # [m, per, 4]
        assert torch.equal(tiles[i * per:(i + m) * per, 0, 0].reshape(m, per, 4), want), i
        if block == 16:
            assert (p.row_scales == out.row_scales).all()
    rest = sv.sv_quantize_fp4(x[:, n * L:].contiguous(), block)
    assert torch.equal(out.values[:, n * L // 2:], rest.values)
    assert torch.equal(tiles[n * per:, 0, 0], rest.scales.view(torch.uint8)[0, :, 0, 0])
    back = sv.sv_dequantize_fp4(out)
    assert torch.equal(back[:, n * L:], sv.sv_dequantize_fp4(rest))
    m = 1 << 12
    p = sv.sv_quantize_fp4(x[0, (n - m) * L:n * L].view(m, L), block)
    assert torch.equal(back[0, (n - m) * L:n * L].view(m, L), sv.sv_dequantize_fp4(p))
