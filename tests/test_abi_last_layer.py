"""The last-layer entry points without a GPU: host checks reject bad
arguments before any launch, and the binding refuses bad tensors."""
import ctypes

import pytest
import torch

import speculative_decoding_sampling_gb300 as sv
from speculative_decoding_sampling_gb300 import _native as N

FAKE = 1 << 40   # a plausible device address, never dereferenced
NAN, INF = float("nan"), float("inf")


def _call(fn, names, base, kw):
    a = dict(base, **kw)
    return getattr(N.lib(), fn)(*[ctypes.c_float(a[n]) if isinstance(a[n], float) else a[n] for n in names])


NORM = dict(x=FAKE, xt=N.SV_BF16, res=FAKE, rt=N.SV_FP32, post=None, gate=None, gate_rows=1, pre=FAKE, wt=N.SV_BF16,
            offset=0.0, rs=1.0, bs=1.0, eps=1e-6, M=6, d=512, rout=FAKE, h=FAKE, ht=N.SV_BF16, scales=None,
            stream=None)


def _norm(**kw):
    return _call("sv_block_norm", list(NORM), NORM, kw)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(res=None), dict(pre=None), dict(rout=None), dict(h=None), dict(M=-1), dict(d=0), dict(d=-8),
    dict(xt=2), dict(xt=7), dict(rt=2), dict(wt=2), dict(ht=3), dict(ht=N.SV_E4M3), dict(scales=FAKE),
    dict(ht=N.SV_E4M3, scales=FAKE + 2), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(rs=INF), dict(bs=NAN),
    dict(offset=NAN), dict(gate=FAKE, gate_rows=0), dict(gate=FAKE, gate_rows=4), dict(gate=FAKE, gate_rows=12),
    dict(x=FAKE + 1), dict(res=FAKE + 2), dict(pre=FAKE + 1), dict(post=FAKE + 1), dict(h=FAKE + 1),
    dict(rout=FAKE + 2), dict(gate=FAKE + 1),
], ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_norm_host_checks(kw):
    assert _norm(**kw) == N.SV_EINVAL


def test_norm_sizes():
    assert _norm(d=N.SV_MAX_D + 1) == N.SV_EUNSUPPORTED
    assert _norm(M=1 << 31) == N.SV_EUNSUPPORTED
    assert _norm(M=0, x=None, res=None) == N.SV_OK


QUANT = dict(x=FAKE, xt=N.SV_BF16, rows=4, d=100, block=1, v=FAKE, scales=FAKE, stream=None)


def _quant(**kw):
    return _call("sv_quantize_fp8", list(QUANT), QUANT, kw)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(v=None), dict(scales=None), dict(rows=-1), dict(d=0), dict(xt=2), dict(block=0), dict(block=64),
    dict(x=FAKE + 1), dict(xt=N.SV_FP32, x=FAKE + 2), dict(scales=FAKE + 1),
], ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_quantize_host_checks(kw):
    assert _quant(**kw) == N.SV_EINVAL


def test_quantize_sizes():
    assert _quant(rows=0, x=None) == N.SV_OK
    assert _quant(rows=1 << 31) == N.SV_EUNSUPPORTED
    assert _quant(rows=(1 << 31) - 1, d=1 << 20) == N.SV_EUNSUPPORTED  # more blocks than one launch has


HEAD = dict(h=FAKE, hs=FAKE, w=FAKE, ws=FAKE, M=256, d=4096, V=1000, out=FAKE, status=None, stream=None)


def _head(**kw):
    return _call("sv_lm_head_logits_fp8", list(HEAD), HEAD, kw)


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(hs=None), dict(w=None), dict(ws=None), dict(out=None), dict(M=-1), dict(d=0), dict(d=8),
    dict(d=24), dict(V=0), dict(h=FAKE + 8), dict(w=FAKE + 8), dict(hs=FAKE + 2), dict(ws=FAKE + 2),
    dict(out=FAKE + 1), dict(status=FAKE + 2),
], ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_head_host_checks(kw):
    assert _head(**kw) == N.SV_EINVAL


def test_head_sizes():
    assert _head(V=N.SV_MAX_V + 1) == N.SV_EUNSUPPORTED
    assert _head(M=(1 << 30) + 1) == N.SV_EUNSUPPORTED
    assert _head(M=0, h=None) == N.SV_OK
    # more tiles, or steps of them, than are counted in 32 bits
    assert _head(M=1 << 30, V=N.SV_MAX_V) == N.SV_EUNSUPPORTED
    assert _head(M=1 << 24, V=N.SV_MAX_V, d=(1 << 31) - 16) == N.SV_EUNSUPPORTED


VERIFY = dict(h=FAKE, hs=FAKE, w=FAKE, ws=FAKE, d=256, q=FAKE, tok=FAKE, u=FAKE, T=1.0, B=4, K=3, V=1000, logits=FAKE,
              out=FAKE, n=FAKE, flags=None, prob=None, mass=None, status=None, wsp=FAKE, ws_bytes=1 << 24, stream=None)


def _verify(**kw):
    return _call("spec_verify_lm_head_fp8", list(VERIFY), VERIFY, kw)


@pytest.mark.parametrize("kw", [
    dict(h=None), dict(hs=None), dict(w=None), dict(ws=None), dict(logits=None), dict(u=None), dict(out=None),
    dict(tok=None), dict(n=None), dict(d=40), dict(B=-1), dict(K=-1), dict(T=0.0), dict(T=NAN), dict(ws_bytes=64),
    dict(wsp=None), dict(wsp=FAKE + 16), dict(h=FAKE + 4), dict(logits=FAKE + 1), dict(status=FAKE + 1),
], ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_verify_host_checks(kw):
    assert _verify(**kw) == N.SV_EINVAL


def test_verify_sizes():
    assert _verify(B=0) == N.SV_OK
    assert _verify(V=N.SV_MAX_V + 1) == N.SV_EUNSUPPORTED
    assert _verify(B=1 << 40) == N.SV_EUNSUPPORTED
    for B, K, V in ((1, 0, 1), (8, 4, 32000), (256, 8, 151936)):
        need = sv.sv_lm_head_fp8_workspace_bytes(B, K, V)
        # the verification's workspace plus at least one pair per row and 256 ids
        assert need >= sv.sv_workspace_bytes(B, K, V) + B * (K + 1) * -(-V // 256) * 8 and need % 256 == 0
        assert _verify(B=B, K=K, V=V, ws_bytes=need - 1) == N.SV_EINVAL
    assert sv.sv_lm_head_fp8_workspace_bytes(-1, 8, 100) == 0
    assert sv.sv_lm_head_fp8_workspace_bytes(1, 8, 0) == 0
    assert sv.sv_lm_head_fp8_workspace_bytes(1 << 40, 8, 100) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 64)
    w = torch.zeros(64)
    f8 = torch.zeros(2, 64, dtype=torch.float8_e4m3fn)
    for call in (lambda: sv.sv_block_norm(x, x, w), lambda: sv.sv_quantize_fp8(x),
                 lambda: sv.sv_lm_head_logits_fp8(f8, x, f8, x),
                 lambda: sv.spec_verify_lm_head_fp8(f8, x, f8, x, None, x, x, 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sv.sv_block_norm(x.half(), x, w), lambda: sv.sv_block_norm(x, x, w.half()),
                 lambda: sv.sv_block_norm(x, x, w, hidden_dtype=torch.float16), lambda: sv.sv_quantize_fp8(x.half()),
                 lambda: sv.sv_quantize_fp8(f8), lambda: sv.sv_lm_head_logits_fp8(x, x, f8, x),
                 lambda: sv.sv_lm_head_logits_fp8(f8, x, x, x)):
        with pytest.raises(TypeError):
            call()
