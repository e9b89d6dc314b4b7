"""The draft step's entry points without a GPU: host checks reject bad
arguments before any launch, and the binding refuses bad tensors."""
import ctypes

import pytest
import torch

import speculative_decoding_sampling_gb300 as sv
from speculative_decoding_sampling_gb300 import _native as N

FAKE = 1 << 40   # a plausible device address, never dereferenced
NAN, INF = float("nan"), float("inf")


def _call(fn, base, kw):
    a = dict(base, **kw)
    return getattr(N.lib(), fn)(*[ctypes.c_float(a[n]) if isinstance(a[n], float) else a[n] for n in base])


def _ids(d):
    return ",".join(f"{k}={v}" for k, v in d.items())


QUANT = dict(x=FAKE, xt=N.SV_BF16, rows=4, d=100, block=16, v=FAKE, scales=FAKE, rs=FAKE, stream=None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(v=None), dict(scales=None), dict(rs=None), dict(block=32), dict(rows=-1), dict(d=0), dict(d=1),
    dict(d=99), dict(d=-2), dict(xt=2), dict(xt=9), dict(block=0), dict(block=8), dict(block=64), dict(x=FAKE + 1),
    dict(xt=N.SV_FP32, x=FAKE + 2), dict(scales=FAKE + 8), dict(rs=FAKE + 2),
], ids=_ids)
def test_quantize_host_checks(kw):
    assert _call("sv_quantize_fp4", QUANT, kw) == N.SV_EINVAL


BACK = dict(v=FAKE, scales=FAKE, rs=FAKE, rows=4, d=100, block=16, out=FAKE, ot=N.SV_BF16, stream=None)


@pytest.mark.parametrize("kw", [
    dict(v=None), dict(scales=None), dict(rs=None), dict(out=None), dict(block=32), dict(block=17), dict(rows=-1),
    dict(d=0), dict(d=3), dict(ot=2), dict(out=FAKE + 1), dict(ot=N.SV_FP32, out=FAKE + 2), dict(rs=FAKE + 1),
], ids=_ids)
def test_dequantize_host_checks(kw):
    assert _call("sv_dequantize_fp4", BACK, kw) == N.SV_EINVAL


def test_form_sizes():
    for fn, base in (("sv_quantize_fp4", QUANT), ("sv_dequantize_fp4", BACK)):
        assert _call(fn, base, dict(rows=0, v=None, scales=None)) == N.SV_OK
        assert _call(fn, base, dict(rows=1 << 31)) == N.SV_EUNSUPPORTED
        assert _call(fn, base, dict(d=(1 << 31) - 2)) == N.SV_EUNSUPPORTED
    size = N.lib().sv_fp4_scale_bytes
    assert size(1, 2, 16) == 512 and size(128, 64, 16) == 512 and size(129, 64, 16) == 1024
    assert size(128, 66, 16) == 1024 and size(128, 128, 32) == 512 and size(300, 1000, 32) == 3 * 8 * 512
    assert size(0, 64, 16) == 0 and size(-1, 64, 16) == 0 and size(4, 63, 16) == 0 and size(4, 64, 24) == 0


HEAD = dict(h=FAKE, hs=FAKE, hr=FAKE, w=FAKE, ws=FAKE, wr=FAKE, block=16, M=256, d=4096, V=1000, out=FAKE, status=None,
            stream=None)


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(hs=None), dict(hr=None), dict(w=None), dict(ws=None), dict(wr=None), dict(out=None), dict(block=32),
    dict(block=32, hr=None), dict(block=32, wr=None), dict(block=64), dict(M=-1), dict(d=0), dict(d=16), dict(d=48),
    dict(V=0), dict(h=FAKE + 8), dict(hs=FAKE + 8), dict(w=FAKE + 8), dict(ws=FAKE + 4), dict(hr=FAKE + 2),
    dict(wr=FAKE + 1), dict(out=FAKE + 1), dict(status=FAKE + 2),
], ids=_ids)
def test_head_host_checks(kw):
    assert _call("sv_lm_head_logits_fp4", HEAD, kw) == N.SV_EINVAL


def test_head_sizes():
    assert _call("sv_lm_head_logits_fp4", HEAD, dict(V=N.SV_MAX_V + 1)) == N.SV_EUNSUPPORTED
    assert _call("sv_lm_head_logits_fp4", HEAD, dict(M=(1 << 30) + 1)) == N.SV_EUNSUPPORTED
    assert _call("sv_lm_head_logits_fp4", HEAD, dict(d=(1 << 20) + 32)) == N.SV_EUNSUPPORTED
    assert _call("sv_lm_head_logits_fp4", HEAD, dict(M=0, h=None)) == N.SV_OK
    # more tiles of logits, or of scales, than are counted in 32 bits
    assert _call("sv_lm_head_logits_fp4", HEAD, dict(M=1 << 30, V=N.SV_MAX_V)) == N.SV_EUNSUPPORTED
    assert _call("sv_lm_head_logits_fp4", HEAD, dict(M=1 << 30, V=64, d=1 << 20)) == N.SV_EUNSUPPORTED


SAMPLE = dict(z=FAKE, zt=N.SV_BF16, u=FAKE, T=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=4, V=1000, tokens=FAKE, prob=None,
              kept=None, probs=None, status=None, stream=None)


@pytest.mark.parametrize("kw", [
    dict(z=None), dict(u=None), dict(tokens=None), dict(rows=-1), dict(V=0), dict(zt=2), dict(T=0.0), dict(T=-1.0),
    dict(T=NAN), dict(T=INF), dict(T=1e-35), dict(T=1e35), dict(top_p=0.0), dict(top_p=-0.5), dict(top_p=NAN),
    dict(min_p=-0.1), dict(min_p=1.5), dict(min_p=NAN), dict(z=FAKE + 1), dict(zt=N.SV_FP32, z=FAKE + 2), dict(u=FAKE + 2),
    dict(tokens=FAKE + 1), dict(prob=FAKE + 2), dict(kept=FAKE + 2), dict(probs=FAKE + 1), dict(status=FAKE + 1),
], ids=_ids)
def test_sample_host_checks(kw):
    assert _call("sv_sample_logits", SAMPLE, kw) == N.SV_EINVAL


def test_sample_sizes():
    assert _call("sv_sample_logits", SAMPLE, dict(rows=0, z=None, u=None, tokens=None)) == N.SV_OK
    assert _call("sv_sample_logits", SAMPLE, dict(V=N.SV_MAX_V + 1)) == N.SV_EUNSUPPORTED
    assert _call("sv_sample_logits", SAMPLE, dict(rows=1 << 30)) == N.SV_EUNSUPPORTED


def _form(rows=4, d=64, block=16, **kw):
    f = dict(values=torch.zeros((rows, d // 2), dtype=torch.uint8),
             scales=torch.zeros((-(-rows // 128), -(-d // (4 * block)), 32, 4, 4), dtype=torch.uint8).view(
                 torch.float8_e4m3fn if block == 16 else torch.float8_e8m0fnu),
             row_scales=torch.ones(rows) if block == 16 else None)
    f.update(kw)
    return sv.Fp4Tensor(**f)


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 64)
    for call in (lambda: sv.sv_quantize_fp4(x), lambda: sv.sv_dequantize_fp4(_form()),
                 lambda: sv.sv_lm_head_logits_fp4(_form(), _form()), lambda: sv.sv_sample_logits(x, torch.zeros(2), 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sv.sv_quantize_fp4(x.half()), lambda: sv.sv_sample_logits(x.half(), torch.zeros(2), 1.0),
                 lambda: sv.sv_dequantize_fp4(_form(), torch.float16),
                 lambda: sv.sv_dequantize_fp4(_form(values=torch.zeros((4, 32)))),
                 lambda: sv.sv_lm_head_logits_fp4(_form(scales=torch.zeros(1)), _form())):
        with pytest.raises(TypeError):
            call()
