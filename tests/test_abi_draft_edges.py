"""The draft step's host side at its limits, without a GPU."""
import os
import subprocess
import sys

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


def test_a_torch_without_e8m0_has_everything_but_blocks_of_32():
    code = """
import torch
del torch.float8_e8m0fnu
import speculative_decoding_sampling_gb300 as sv
assert callable(sv.spec_verify) and callable(sv.sv_lm_head_logits_fp4)

class OnDevice(torch.Tensor):   # what the checks ask of a CUDA tensor
    is_cuda = True

x = torch.zeros(2, 64).as_subclass(OnDevice)
try:
    sv.sv_quantize_fp4(x, 32)
except TypeError as e:
    assert "float8_e8m0fnu" in str(e), e
else:
    raise AssertionError("taken")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
