"""The draft step's host side at its limits, without a GPU."""
import pytest

from speculative_decoding_sampling_gb300 import _native as N

FAKE = 1 << 40   # a plausible device address, never dereferenced
MAX_ROWS, MAX_D = (1 << 31) - 128, (1 << 31) - 1026     # (d is even)


@pytest.mark.parametrize("block", [16, 32])
def test_sizes_that_are_refused_have_no_scales(block):
    """sv_fp4_scale_bytes is 0 exactly where quantisation and reading back refuse the sizes."""
    L = N.lib()
    rs = FAKE if block == 16 else None
    for rows, d in ((MAX_ROWS + 1, 64), ((1 << 31) - 1, 64), (1 << 31, 64), (4, MAX_D + 2), (4, (1 << 31) - 2)):
        assert L.sv_fp4_scale_bytes(rows, d, block) == 0
        assert L.sv_quantize_fp4(FAKE, N.SV_BF16, rows, d, block, FAKE, FAKE, rs, None) == N.SV_EUNSUPPORTED
        assert L.sv_dequantize_fp4(FAKE, FAKE, rs, rows, d, block, FAKE, N.SV_BF16, None) == N.SV_EUNSUPPORTED
    for rows, d in ((MAX_ROWS, 64), (4, MAX_D), (1, 2)):
        assert L.sv_fp4_scale_bytes(rows, d, block) == -(-rows // 128) * -(-d // (4 * block)) * 512
        # (in range: refused for its pointer, not for its size)
        assert L.sv_quantize_fp4(FAKE + 1, N.SV_BF16, rows, d, block, FAKE, FAKE, rs, None) == N.SV_EINVAL
        assert L.sv_dequantize_fp4(FAKE, FAKE, rs, rows, d, block, FAKE + 1, N.SV_BF16, None) == N.SV_EINVAL
