"""PyTorch binding of the C ABI: argument marshalling only.

Every step of the verification runs in the CUDA kernels of
libspecverify.so; this module checks shapes and dtypes, allocates outputs
and the workspace through PyTorch, and passes raw device pointers and the
current CUDA stream.  The function names are those of the C ABI.
"""
from __future__ import annotations

import threading
from dataclasses import dataclass

import torch

from . import _native as N


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(sv_status_string(code))


def sv_status_string(code: int) -> str:
    return N.lib().sv_status_string(int(code)).decode()


def sv_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(N.lib().sv_workspace_bytes(int(B), int(K), int(V)))


def sv_kernel_launches(logits_dtype: torch.dtype, dense: bool, B: int, K: int, V: int) -> int:
    """Kernels one spec_verify call with these arguments launches on the
    current device (2 or 3; 0 for B == 0)."""
    import ctypes
    dt = N.SV_BF16 if logits_dtype == torch.bfloat16 else N.SV_FP32
    if logits_dtype not in (torch.bfloat16, torch.float32):
        raise SpecVerifyError(N.SV_EINVAL)
    n = ctypes.c_int32(-1)
    rc = N.lib().sv_kernel_launches(dt, 1 if dense else 0, int(B), int(K), int(V), ctypes.byref(n))
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return int(n.value)


def sv_filter_logits(logits: torch.Tensor, temperature: float, top_k: int = 0, top_p: float = 1.0, *,
                     out: torch.Tensor | None = None, kept: torch.Tensor | None = None,
                     status: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Top-k / top-p filtering of logit rows (last axis = V) at `temperature`:
    every id outside the kept set becomes -inf.  `out` may be `logits`
    itself (in place).  Returns (filtered logits, kept ids per row)."""
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise SpecVerifyError(N.SV_EINVAL)
    if not logits.is_cuda or not logits.is_contiguous() or logits.dim() < 1:
        raise ValueError("logits must be a contiguous CUDA tensor")
    V = logits.shape[-1]
    rows = logits.numel() // V if V else 0
    if out is None:
        out = torch.empty_like(logits)
    if out.shape != logits.shape or out.dtype != logits.dtype or not out.is_contiguous() \
            or out.device != logits.device:
        raise ValueError("out must match logits")
    if kept is None:
        kept = torch.empty(logits.shape[:-1], dtype=torch.int32, device=logits.device)
    if kept.numel() != rows or kept.dtype != torch.int32 or not kept.is_contiguous() \
            or kept.device != logits.device:
        raise ValueError("kept must be a contiguous int32 tensor with one entry per row on the logits' device")
    if status is not None:
        _check(status, "status", torch.int32, (1,), logits.device)
    dt = N.SV_BF16 if logits.dtype == torch.bfloat16 else N.SV_FP32
    stream = torch.cuda.current_stream(logits.device).cuda_stream
    rc = N.lib().sv_filter_logits(logits.data_ptr(), dt, rows, V, float(temperature), int(top_k),
                                  float(top_p), out.data_ptr(), kept.data_ptr(),
                                  None if status is None else status.data_ptr(), stream)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out, kept


_ws_local = threading.local()  # of each host thread: {(device index, raw stream): workspace}


def default_workspace(device: torch.device, nbytes: int, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """A zero-filled workspace of at least `nbytes` on `device` for the calls
    on `stream` (default: the current one) that do not pass their own.  Each
    stream and host thread has one, allocated, cleared and used on that stream
    only: the kernels leave it zero-filled, so calls in the stream's order may
    share it, and calls that may overlap never do (a call is several launches,
    which another thread's may come between).  While the stream is being
    captured, a new one that belongs to the graph, which clears it."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    current = torch.cuda.current_stream(idx)
    if stream is None:
        stream = current
    if stream != current or idx != torch.cuda.current_device():
        with torch.cuda.stream(stream):
            return _workspace_here(idx, stream.cuda_stream, nbytes)
    return _workspace_here(idx, stream.cuda_stream, nbytes)


def _workspace_here(idx: int, raw_stream: int, nbytes: int) -> torch.Tensor:
    """default_workspace of the current stream and device."""
    capturing = torch.cuda.is_current_stream_capturing()
    mine, key = _ws_local.__dict__, (idx, raw_stream)
    ws = None if capturing else mine.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=f"cuda:{idx}")
        if not capturing:
            mine[key] = ws
    return ws


@dataclass
class SpecVerifyResult:
    out_tokens: torch.Tensor            # int32 [B, K+1], -1 padded
    num_emitted: torch.Tensor           # int32 [B]
    accept_flags: torch.Tensor          # int8  [B, K]
    accept_prob: torch.Tensor | None    # fp32  [B, K]
    residual_mass: torch.Tensor | None  # fp32  [B]
    status: torch.Tensor | None         # int32 [1], OR of SV_BAD_* bits


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, dtype, shape, device, host_ok: bool = False):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device and not (host_ok and _pinned(t)):
        raise ValueError(f"{name}: expected device {device}" + (" or page-locked host memory" if host_ok else "")
                         + f", got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _exec_device(target_logits: torch.Tensor) -> torch.device:
    """The GPU a call runs on: the logits' own, or the current one for
    page-locked host logits."""
    if target_logits.is_cuda:
        return target_logits.device
    if _pinned(target_logits):
        return torch.device("cuda", torch.cuda.current_device())
    raise ValueError("target_logits must be a CUDA tensor or page-locked host memory")


def _pinned(t: torch.Tensor) -> bool:
    """A page-locked CPU tensor: mapped into every device's address space, so
    the kernels read it in place (only the bytes they touch cross the link)."""
    return t.device.type == "cpu" and t.is_pinned()


def _call(fn_name: str, target_logits, draft_probs, draft_tokens, uniforms,
          temperature, out_tokens, num_emitted, accept_flags, accept_prob,
          residual_mass, status, workspace, stream, stats=None):
    dev = _exec_device(target_logits)
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, K+1, V]")
    B, K1, V = target_logits.shape
    K = K1 - 1
    if K < 0:
        raise ValueError("target_logits needs K+1 >= 1 rows per sequence")
    if target_logits.dtype == torch.bfloat16:
        dt = N.SV_BF16
    elif target_logits.dtype == torch.float32:
        dt = N.SV_FP32
    else:
        raise TypeError("target_logits must be bfloat16 or float32")
    if not target_logits.is_contiguous():
        raise ValueError("target_logits must be contiguous")
    if draft_probs is not None:
        _check(draft_probs, "draft_probs", torch.float32, (B, K, V), dev, host_ok=True)
    if draft_tokens is None:
        if K > 0:
            raise ValueError("draft_tokens required when K > 0")
    else:
        _check(draft_tokens, "draft_tokens", torch.int32, (B, K), dev, host_ok=True)
    _check(uniforms, "uniforms", torch.float32, (B, K + 1), dev, host_ok=True)
    for name, t, dtype, shape in (("out_tokens", out_tokens, torch.int32, (B, K + 1)),
                                  ("num_emitted", num_emitted, torch.int32, (B,)),
                                  ("accept_flags", accept_flags, torch.int8, (B, K)),
                                  ("accept_prob", accept_prob, torch.float32, (B, K)),
                                  ("residual_mass", residual_mass, torch.float32, (B,)),
                                  ("status", status, torch.int32, (1,))):
        if t is not None:
            _check(t, name, dtype, shape, dev)
    need = sv_workspace_bytes(B, K, V)
    if need == 0 and B > 0:
        raise SpecVerifyError(N.SV_EUNSUPPORTED)
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    if workspace is None:
        if fn_name != "spec_verify" and torch.cuda.is_current_stream_capturing():
            raise ValueError("workspace: the two stages of a captured call need one that both are given")
        workspace = default_workspace(dev, need, stream)
    elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes on {dev}")
    args = [target_logits.data_ptr(), dt, _ptr(draft_probs), _ptr(draft_tokens),
            uniforms.data_ptr(), float(temperature), B, K, V, _ptr(out_tokens),
            _ptr(num_emitted), _ptr(accept_flags), _ptr(accept_prob),
            _ptr(residual_mass), _ptr(status), workspace.data_ptr(),
            workspace.numel() * workspace.element_size()]
    if stats is not None:
        _check(stats, "stats", torch.int64, (N.stats_words(K),), dev)
        fn_name = "spec_verify_stats"
        args.append(stats.data_ptr())
    rc = getattr(N.lib(), fn_name)(*args, stream.cuda_stream)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)


def _outputs(target_logits, want_probs, out):
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = _exec_device(target_logits)
    o = dict(out or {})
    o.setdefault("out_tokens", torch.empty((B, K + 1), dtype=torch.int32, device=dev))
    o.setdefault("num_emitted", torch.empty((B,), dtype=torch.int32, device=dev))
    o.setdefault("accept_flags", torch.empty((B, K), dtype=torch.int8, device=dev))
    if want_probs:
        o.setdefault("accept_prob", torch.empty((B, K), dtype=torch.float32, device=dev))
        o.setdefault("residual_mass", torch.empty((B,), dtype=torch.float32, device=dev))
    o.setdefault("accept_prob", None)
    o.setdefault("residual_mass", None)
    o.setdefault("status", None)
    return o


def spec_verify(target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
                draft_tokens: torch.Tensor | None, uniforms: torch.Tensor,
                temperature: float, *, want_probs: bool = True,
                out: dict | None = None, status: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None,
                stats: torch.Tensor | None = None) -> SpecVerifyResult:
    """Verify a batch of drafts against target logits on the GPU.

    target_logits [B, K+1, V] bf16/fp32; draft_probs [B, K, V] fp32 or None
    (one-hot drafts); draft_tokens [B, K] int32; uniforms [B, K+1] fp32 in
    [0, 1) with uniforms[:, K] the final draw; temperature > 0.  The inputs
    may be CUDA tensors or page-locked (pinned) CPU tensors, which the
    kernels read in place: a pinned draft_probs sends only the rows the
    draws use (the rejected ones) and the drafted entries over the link.
    `out` may supply preallocated output tensors by name; `status` an int32
    [1] device tensor that receives SV_BAD_* bits; `stats` an int64
    [SV_STATS_WORDS(K)] device tensor the verdicts add the call's acceptance
    counters to (spec_verify_stats).  Runs asynchronously on `stream`
    (default: the current stream).  Without a `workspace` the call takes
    default_workspace's, which calls on other streams or from other host
    threads do not share; in a captured graph that is one of the graph's own,
    which every replay clears."""
    o = _outputs(target_logits, want_probs, out)
    if status is not None:
        o["status"] = status
    _call("spec_verify", target_logits, draft_probs, draft_tokens, uniforms,
          temperature, o["out_tokens"], o["num_emitted"], o["accept_flags"],
          o["accept_prob"], o["residual_mass"], o["status"], workspace, stream, stats)
    return SpecVerifyResult(o["out_tokens"], o["num_emitted"], o["accept_flags"],
                            o["accept_prob"], o["residual_mass"], o["status"])


def sv_verify_rows(target_logits, draft_probs, draft_tokens, uniforms,
                   temperature, *, out: dict, workspace: torch.Tensor,
                   stream=None) -> None:
    """First stage of spec_verify (see the C header); `out` as returned in
    the fields of a SpecVerifyResult."""
    _call("sv_verify_rows", target_logits, draft_probs, draft_tokens, uniforms,
          temperature, out["out_tokens"], out["num_emitted"],
          out.get("accept_flags"), out.get("accept_prob"),
          out.get("residual_mass"), out.get("status"), workspace, stream)


def sv_sample_survivors(target_logits, draft_probs, draft_tokens, uniforms,
                        temperature, *, out: dict, workspace: torch.Tensor,
                        stream=None) -> None:
    """Second stage of spec_verify; must follow sv_verify_rows on the same
    stream, workspace and inputs."""
    _call("sv_sample_survivors", target_logits, draft_probs, draft_tokens,
          uniforms, temperature, out["out_tokens"], out["num_emitted"],
          out.get("accept_flags"), out.get("accept_prob"),
          out.get("residual_mass"), out.get("status"), workspace, stream)


# ------------------------------------------------------------- LM head

def sv_lm_head_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(N.lib().sv_lm_head_workspace_bytes(int(B), int(K), int(V)))


def _lm_check(hidden, lm_head):
    if hidden.dtype != torch.bfloat16 or lm_head.dtype != torch.bfloat16:
        raise TypeError("hidden and lm_head must be bfloat16")
    if not (hidden.is_cuda and lm_head.is_cuda and hidden.is_contiguous() and lm_head.is_contiguous()):
        raise ValueError("hidden and lm_head must be contiguous CUDA tensors")
    if hidden.device != lm_head.device or lm_head.dim() != 2 or hidden.shape[-1] != lm_head.shape[1]:
        raise ValueError("lm_head must be [V, d] on the hidden states' device, d their last dimension")


def sv_lm_head_logits(hidden: torch.Tensor, lm_head: torch.Tensor, *, out: torch.Tensor | None = None,
                      status: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """logits = hidden @ lm_head.T on the tensor cores, bf16 out: hidden
    [..., d] bf16, lm_head [V, d] bf16 -> [..., V] bf16.  status: optional
    int32 [1] device tensor that receives SV_INTERNAL_TIMEOUT."""
    _lm_check(hidden, lm_head)
    V, d = lm_head.shape
    M = hidden.numel() // d if d else 0
    if out is None:
        out = torch.empty(hidden.shape[:-1] + (V,), dtype=torch.bfloat16, device=hidden.device)
    if out.dtype != torch.bfloat16 or out.numel() != M * V or not out.is_contiguous() or out.device != hidden.device:
        raise ValueError("out must be a contiguous bf16 [..., V] tensor on the hidden states' device")
    if status is not None:
        _check(status, "status", torch.int32, (1,), hidden.device)
    stream = stream or torch.cuda.current_stream(hidden.device)
    rc = N.lib().sv_lm_head_logits(hidden.data_ptr(), lm_head.data_ptr(), M, d, V, out.data_ptr(),
                                   _ptr(status), stream.cuda_stream)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out


def spec_verify_lm_head(hidden: torch.Tensor, lm_head: torch.Tensor, draft_probs: torch.Tensor | None,
                        draft_tokens: torch.Tensor, uniforms: torch.Tensor, temperature: float, *,
                        logits_out: torch.Tensor | None = None, want_probs: bool = True,
                        workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """spec_verify on logits computed in the same step by the target's LM
    head: hidden [B, K+1, d] bf16, lm_head [V, d] bf16.  Returns
    (SpecVerifyResult, logits [B, K+1, V] bf16).  workspace as for
    spec_verify."""
    _lm_check(hidden, lm_head)
    if hidden.dim() != 3:
        raise ValueError("hidden must be [B, K+1, d]")
    B, K1, d = hidden.shape
    K = K1 - 1
    V = lm_head.shape[0]
    dev = hidden.device
    if logits_out is None:
        logits_out = torch.empty((B, K1, V), dtype=torch.bfloat16, device=dev)
    if logits_out.shape != (B, K1, V) or logits_out.dtype != torch.bfloat16 or not logits_out.is_contiguous():
        raise ValueError("logits_out must be a contiguous bf16 [B, K+1, V] tensor")
    if draft_probs is not None:
        _check(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _check(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _check(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    need = sv_lm_head_workspace_bytes(B, K, V)
    if need == 0 and B > 0:
        raise SpecVerifyError(N.SV_EUNSUPPORTED)
    stream = stream or torch.cuda.current_stream(dev)
    if workspace is None:
        workspace = default_workspace(dev, need, stream)
    elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes on {dev}")
    res = SpecVerifyResult(
        out_tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
        num_emitted=torch.empty((B,), dtype=torch.int32, device=dev),
        accept_flags=torch.empty((B, K), dtype=torch.int8, device=dev),
        accept_prob=torch.empty((B, K), dtype=torch.float32, device=dev) if want_probs else None,
        residual_mass=torch.empty((B,), dtype=torch.float32, device=dev) if want_probs else None,
        status=status)
    if status is not None:
        _check(status, "status", torch.int32, (1,), dev)
    rc = N.lib().spec_verify_lm_head(
        hidden.data_ptr(), lm_head.data_ptr(), d, _ptr(draft_probs), draft_tokens.data_ptr(),
        uniforms.data_ptr(), float(temperature), B, K, V, logits_out.data_ptr(), res.out_tokens.data_ptr(),
        res.num_emitted.data_ptr(), res.accept_flags.data_ptr(), _ptr(res.accept_prob),
        _ptr(res.residual_mass), _ptr(status), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), stream.cuda_stream)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return res, logits_out


# ------------------------------------------------------------- the last layer in 8-bit floating point

_BLOCK = 128  # values along d (and ids of the output embedding) that share a scale
_DTYPES = {torch.bfloat16: N.SV_BF16, torch.float32: N.SV_FP32, torch.float8_e4m3fn: N.SV_E4M3}
_F8, _F32 = torch.float8_e4m3fn, torch.float32


def _dtype(t: torch.Tensor, name: str, fp8: bool = False) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None or (dt == N.SV_E4M3) != fp8:
        raise TypeError(f"{name}: expected {'float8_e4m3fn' if fp8 else 'bfloat16 or float32'}, got {t.dtype}")
    return dt


def _cuda(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.device


def _need(t: torch.Tensor, name: str, dtype, shape, dev: torch.device):
    """_check, without its cost where nothing is wrong (these calls are a few
    microseconds of host time in all)."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check(t, name, dtype, shape, dev)


class _Streams:
    """Enter `stream` and its device: the tensors made inside belong to it."""

    def __init__(self, dev: torch.device, stream: torch.cuda.Stream | None):
        stream = stream or torch.cuda.current_stream(dev)
        if stream.device != dev:
            raise ValueError(f"stream: expected a stream of {dev}, got one of {stream.device}")
        self.raw = stream.cuda_stream
        self.ctx = torch.cuda.stream(stream)

    def __enter__(self) -> int:
        self.ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


class _Current:
    """The same for the current stream of the current device: nothing to do."""

    def __enter__(self) -> int:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())

    def __exit__(self, *exc):
        pass


_CURRENT = _Current()


def _on(dev: torch.device, stream: torch.cuda.Stream | None):
    if stream is None and dev.index == torch.cuda.current_device():
        return _CURRENT
    return _Streams(dev, stream)


def _blocks(n: int) -> int:
    return -(-n // _BLOCK)


def _fits(d: int):
    """A row's length is a 32-bit integer in the C ABI."""
    if d > 0x7FFFFFFF:
        raise SpecVerifyError(N.SV_EUNSUPPORTED)


def sv_quantize_fp8(x: torch.Tensor, block_rows: int = 1, *, out: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """e4m3 values of x [..., d] (bf16 / fp32) with one fp32 scale per block
    of block_rows x 128: 1 for activations (scales [..., ceil(d / 128)]),
    128 for a weight matrix [V, d] (scales [ceil(V / 128), ceil(d / 128)]).
    Returns (values, scales); `out` and `scales` may be preallocated."""
    dt = _dtype(x, "x")
    dev = _cuda(x, "x")
    shape = x.shape
    if block_rows not in (1, _BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    if len(shape) < 1 or shape[-1] < 1 or (block_rows != 1 and len(shape) != 2):
        raise ValueError("x must be [..., d], and [V, d] for blocks of 128 rows")
    d = shape[-1]
    _fits(d)
    rows = x.numel() // d
    sshape = (shape[:-1] if block_rows == 1 else (_blocks(rows),)) + (_blocks(d),)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=_F8, device=dev)
        else:
            _need(out, "out", _F8, shape, dev)
        if scales is None:
            scales = torch.empty(sshape, dtype=_F32, device=dev)
        else:
            _need(scales, "scales", _F32, sshape, dev)
        rc = N.lib().sv_quantize_fp8(x.data_ptr(), dt, rows, d, block_rows, out.data_ptr(), scales.data_ptr(), s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out, scales


@dataclass
class BlockNormResult:
    hidden: torch.Tensor          # [..., d] bf16 / fp32 / e4m3: the LM head's input
    scales: torch.Tensor | None   # [..., ceil(d / 128)] fp32 (e4m3 hidden)
    residual: torch.Tensor        # [..., d]: the residual stream after the block


def sv_block_norm(x: torch.Tensor, residual: torch.Tensor, norm_weight: torch.Tensor, *,
                  post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                  residual_scale: float = 1.0, branch_scale: float = 1.0, weight_offset: float = 0.0,
                  eps: float = 1e-6, hidden_dtype: torch.dtype = torch.bfloat16,
                  residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  scales: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> BlockNormResult:
    """The norms around the target's last block, from its output x [..., d]
    and the residual stream [..., d] to the LM head's input:

        a = x (or its RMS norm times post_weight + weight_offset)
        r = residual_scale * residual + branch_scale * gate * a
        h = RMS norm of r times norm_weight + weight_offset

    x and residual are bf16 or fp32; the weights [d] share a type, bf16 or
    fp32; gate has x's type and is [d] or [G, ..., d] with G gate rows in
    all, each for the same number of consecutive rows of x (one per sequence
    for [B, 1, d]).  hidden_dtype bfloat16, float32 or float8_e4m3fn (with
    scales as from sv_quantize_fp8).  residual_out may be `residual` (in
    place)."""
    xt, rt, wt = _dtype(x, "x"), _dtype(residual, "residual"), _dtype(norm_weight, "norm_weight")
    ht = _DTYPES.get(hidden_dtype)
    if ht is None:
        raise TypeError("hidden_dtype must be bfloat16, float32 or float8_e4m3fn")
    dev = _cuda(x, "x")
    shape = x.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("x must be [..., d]")
    d = shape[-1]
    _fits(d)
    M = x.numel() // d
    _need(residual, "residual", residual.dtype, shape, dev)
    _need(norm_weight, "norm_weight", norm_weight.dtype, (d,), dev)
    if post_weight is not None:
        _need(post_weight, "post_weight", norm_weight.dtype, (d,), dev)
    gate_rows = 1
    if gate is not None:
        if gate.dim() < 1 or gate.shape[-1] != d or gate.numel() == 0:
            raise ValueError("gate must be [..., d] with at least one row")
        _need(gate, "gate", x.dtype, gate.shape, dev)
        gate_rows = gate.numel() // d
        if M % gate_rows:
            raise ValueError(f"gate: {gate_rows} rows do not divide the {M} rows of x")
    if scales is not None and ht != N.SV_E4M3:
        raise ValueError("scales belong to a float8_e4m3fn hidden")
    with _on(dev, stream) as s:
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _need(residual_out, "residual_out", residual.dtype, shape, dev)
        if out is None:
            out = torch.empty(shape, dtype=hidden_dtype, device=dev)
        else:
            _need(out, "out", hidden_dtype, shape, dev)
        sp = None
        if ht == N.SV_E4M3:
            sshape = shape[:-1] + (_blocks(d),)
            if scales is None:
                scales = torch.empty(sshape, dtype=_F32, device=dev)
            else:
                _need(scales, "scales", _F32, sshape, dev)
            sp = scales.data_ptr()
        rc = N.lib().sv_block_norm(x.data_ptr(), xt, residual.data_ptr(), rt, _ptr(post_weight), _ptr(gate), gate_rows,
                                   norm_weight.data_ptr(), wt, weight_offset, residual_scale, branch_scale, eps, M, d,
                                   residual_out.data_ptr(), out.data_ptr(), ht, sp, s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return BlockNormResult(out, scales, residual_out)


def _lm_fp8_check(hidden, hidden_scales, lm_head, lm_head_scales) -> torch.device:
    _dtype(hidden, "hidden", fp8=True)
    _dtype(lm_head, "lm_head", fp8=True)
    dev = _cuda(hidden, "hidden")
    shape, wshape = hidden.shape, lm_head.shape
    if len(wshape) != 2 or len(shape) < 1 or shape[-1] != wshape[1]:
        raise ValueError("lm_head must be [V, d], d the hidden states' last dimension")
    V, d = wshape
    _fits(V)
    _fits(d)
    nb = _blocks(d)
    _need(lm_head, "lm_head", _F8, wshape, dev)
    _need(hidden_scales, "hidden_scales", _F32, shape[:-1] + (nb,), dev)
    _need(lm_head_scales, "lm_head_scales", _F32, (_blocks(V), nb), dev)
    return dev


def sv_lm_head_logits_fp8(hidden: torch.Tensor, hidden_scales: torch.Tensor, lm_head: torch.Tensor,
                          lm_head_scales: torch.Tensor, *, out: torch.Tensor | None = None,
                          status: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """sv_lm_head_logits on e4m3 operands with block scales: hidden [..., d]
    with hidden_scales [..., ceil(d / 128)], lm_head [V, d] with
    lm_head_scales [ceil(V / 128), ceil(d / 128)] (sv_block_norm and
    sv_quantize_fp8 make both) -> [..., V] bf16.  status: optional int32 [1]
    device tensor that receives SV_INTERNAL_TIMEOUT."""
    dev = _lm_fp8_check(hidden, hidden_scales, lm_head, lm_head_scales)
    V, d = lm_head.shape
    M = hidden.numel() // d if d else 0
    oshape = hidden.shape[:-1] + (V,)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(oshape, dtype=torch.bfloat16, device=dev)
        else:
            _need(out, "out", torch.bfloat16, oshape, dev)
        rc = N.lib().sv_lm_head_logits_fp8(hidden.data_ptr(), hidden_scales.data_ptr(), lm_head.data_ptr(),
                                           lm_head_scales.data_ptr(), M, d, V, out.data_ptr(), _ptr(status), s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out


def sv_lm_head_fp8_workspace_bytes(B: int, K: int, V: int) -> int:
    return int(N.lib().sv_lm_head_fp8_workspace_bytes(int(B), int(K), int(V)))


def spec_verify_lm_head_fp8(hidden: torch.Tensor, hidden_scales: torch.Tensor, lm_head: torch.Tensor,
                            lm_head_scales: torch.Tensor, draft_probs: torch.Tensor | None,
                            draft_tokens: torch.Tensor, uniforms: torch.Tensor, temperature: float, *,
                            logits_out: torch.Tensor | None = None, want_probs: bool = True,
                            workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """spec_verify_lm_head on e4m3 operands with block scales: hidden
    [B, K+1, d], hidden_scales [B, K+1, ceil(d / 128)], lm_head and
    lm_head_scales as for sv_lm_head_logits_fp8.  Returns (SpecVerifyResult,
    logits [B, K+1, V] bf16).  workspace as for spec_verify."""
    dev = _lm_fp8_check(hidden, hidden_scales, lm_head, lm_head_scales)
    if hidden.dim() != 3 or hidden.shape[1] < 1:
        raise ValueError("hidden must be [B, K+1, d]")
    B, K1, d = hidden.shape
    K = K1 - 1
    V = lm_head.shape[0]
    if draft_probs is not None:
        _need(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
    _need(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    _need(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    need = sv_lm_head_fp8_workspace_bytes(B, K, V)
    if need == 0 and B > 0:
        raise SpecVerifyError(N.SV_EUNSUPPORTED)
    with _on(dev, stream) as s:
        if logits_out is None:
            logits_out = torch.empty((B, K1, V), dtype=torch.bfloat16, device=dev)
        _need(logits_out, "logits_out", torch.bfloat16, (B, K1, V), dev)
        if workspace is None:
            workspace = _workspace_here(dev.index, s, need)
        elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace must hold {need} bytes on {dev}")
        res = SpecVerifyResult(
            out_tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
            num_emitted=torch.empty((B,), dtype=torch.int32, device=dev),
            accept_flags=torch.empty((B, K), dtype=torch.int8, device=dev),
            accept_prob=torch.empty((B, K), dtype=torch.float32, device=dev) if want_probs else None,
            residual_mass=torch.empty((B,), dtype=torch.float32, device=dev) if want_probs else None,
            status=status)
        rc = N.lib().spec_verify_lm_head_fp8(
            hidden.data_ptr(), hidden_scales.data_ptr(), lm_head.data_ptr(), lm_head_scales.data_ptr(), d,
            _ptr(draft_probs), draft_tokens.data_ptr(), uniforms.data_ptr(), float(temperature), B, K, V,
            logits_out.data_ptr(), res.out_tokens.data_ptr(), res.num_emitted.data_ptr(), res.accept_flags.data_ptr(),
            _ptr(res.accept_prob), _ptr(res.residual_mass), _ptr(status), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return res, logits_out


# ------------------------------------------------------------- the draft's step in 4-bit floating point

_E8M0 = getattr(torch, "float8_e8m0fnu", None)  # younger than every other type here: without it, no blocks of 32
_SCALE_TYPES = {torch.float8_e4m3fn: 16}        # values of a block, by its scales' type
if _E8M0 is not None:
    _SCALE_TYPES[_E8M0] = 32


@dataclass
class Fp4Tensor:
    """A tensor [..., d] in microscaled 4-bit form.  The scales' type says
    which: float8_e4m3fn (a scale for 16 values, and row_scales) or
    float8_e8m0fnu (a scale for 32 values, no row_scales)."""
    values: torch.Tensor              # uint8 [..., d / 2]: column 2i in the low half of byte i
    scales: torch.Tensor              # [ceil(rows / 128), ceil(blocks / 4), 32, 4, 4]: tiles of 128 rows x 4 blocks
    row_scales: torch.Tensor | None   # fp32 [...]


def _fp4_check(t: Fp4Tensor, name: str) -> tuple[torch.device, int, int, int]:
    """(device, block, rows, d) of t."""
    v, sc, rs = t.values, t.scales, t.row_scales
    block = _SCALE_TYPES.get(sc.dtype)
    if block is None:
        raise TypeError(f"{name}.scales: expected float8_e4m3fn or float8_e8m0fnu, got {sc.dtype}")
    if v.dtype is not torch.uint8:
        raise TypeError(f"{name}.values: expected uint8, got {v.dtype}")
    dev = _cuda(v, name)
    shape = v.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"{name}.values must be [..., d / 2]")
    half = shape[-1]
    d = 2 * half
    _fits(d)
    rows = v.numel() // half
    _need(sc, name, sc.dtype, _fp4_scale_shape(rows, d, block), dev)
    if (rs is None) != (block == 32):
        raise ValueError(f"{name}.row_scales: blocks of 16 have them, blocks of 32 do not")
    if rs is not None:
        _need(rs, name, _F32, shape[:-1], dev)
    return dev, block, rows, d


def _fp4_scale_shape(rows: int, d: int, block: int) -> tuple[int, ...]:
    return -(-rows // 128), -(-d // (4 * block)), 32, 4, 4


def sv_quantize_fp4(x: torch.Tensor, block: int = 16, *, out: Fp4Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> Fp4Tensor:
    """x [..., d] (bf16 / fp32, d even) in microscaled 4-bit form: e2m1
    values, a scale for each block of 16 (e4m3, beside a power of two for
    each row) or 32 consecutive values (a power of two, e8m0).  `out`: one of
    the same shape and block to write into."""
    dt = _dtype(x, "x")
    dev = _cuda(x, "x")
    shape = x.shape
    if block not in (16, 32):
        raise ValueError("block must be 16 or 32")
    if block == 32 and _E8M0 is None:
        raise TypeError("blocks of 32 need a torch that has float8_e8m0fnu")
    if len(shape) < 1 or shape[-1] < 2 or shape[-1] % 2:
        raise ValueError("x must be [..., d], d even")
    d = shape[-1]
    _fits(d)
    rows = x.numel() // d
    with _on(dev, stream) as s:
        if out is None:
            st = torch.float8_e4m3fn if block == 16 else _E8M0
            out = Fp4Tensor(torch.empty(shape[:-1] + (d // 2,), dtype=torch.uint8, device=dev),
                            torch.empty(_fp4_scale_shape(rows, d, block), dtype=st, device=dev),
                            torch.empty(shape[:-1], dtype=_F32, device=dev) if block == 16 else None)
        else:
            odev, oblock, _, _ = _fp4_check(out, "out")
            if odev != dev or oblock != block or out.values.shape != shape[:-1] + (d // 2,):
                raise ValueError("out must be of x's shape and device and of this block")
        rc = N.lib().sv_quantize_fp4(x.data_ptr(), dt, rows, d, block, out.values.data_ptr(), out.scales.data_ptr(),
                                     _ptr(out.row_scales), s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out


def sv_dequantize_fp4(t: Fp4Tensor, dtype: torch.dtype = torch.bfloat16, *, out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """What t stands for, [..., d] in bfloat16 or float32."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("dtype must be bfloat16 or float32")
    dev, block, rows, d = _fp4_check(t, "t")
    shape = t.values.shape[:-1] + (d,)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _need(out, "out", dtype, shape, dev)
        rc = N.lib().sv_dequantize_fp4(t.values.data_ptr(), t.scales.data_ptr(), _ptr(t.row_scales), rows, d, block,
                                       out.data_ptr(), _DTYPES[dtype], s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out


def sv_lm_head_logits_fp4(hidden: Fp4Tensor, lm_head: Fp4Tensor, *, out: torch.Tensor | None = None,
                          status: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """sv_lm_head_logits on operands in microscaled 4-bit form, both of the
    same block: hidden [..., d], lm_head [V, d] -> [..., V] bf16; d a
    multiple of 32.  status: optional int32 [1] device tensor that receives
    SV_INTERNAL_TIMEOUT."""
    dev, block, M, d = _fp4_check(hidden, "hidden")
    wdev, wblock, V, wd = _fp4_check(lm_head, "lm_head")
    if wdev != dev or wblock != block or wd != d or lm_head.values.dim() != 2:
        raise ValueError("lm_head must be [V, d] on the hidden states' device, d their last dimension, of the same block")
    _fits(V)
    oshape = hidden.values.shape[:-1] + (V,)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(oshape, dtype=torch.bfloat16, device=dev)
        else:
            _need(out, "out", torch.bfloat16, oshape, dev)
        rc = N.lib().sv_lm_head_logits_fp4(hidden.values.data_ptr(), hidden.scales.data_ptr(), _ptr(hidden.row_scales),
                                           lm_head.values.data_ptr(), lm_head.scales.data_ptr(), _ptr(lm_head.row_scales),
                                           block, M, d, V, out.data_ptr(), _ptr(status), s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return out


@dataclass
class SampleResult:
    tokens: torch.Tensor              # int32 [...]
    prob: torch.Tensor                # fp32 [...]: the tokens' probabilities
    kept: torch.Tensor                # int32 [...]: ids the filters kept
    probs: torch.Tensor | None        # fp32 [..., V]: the processed distribution
    status: torch.Tensor | None       # int32 [1], OR of SV_BAD_ROW and SV_BAD_U


def sv_sample_logits(logits: torch.Tensor, uniforms: torch.Tensor, temperature: float, top_k: int = 0,
                     top_p: float = 1.0, min_p: float = 0.0, *, want_probs: bool = False,
                     out: dict | None = None, status: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> SampleResult:
    """One token for each row of logits [..., V] (bf16 / fp32) at
    `temperature`, by inverse CDF from uniforms [...] (fp32 in [0, 1)), among
    the ids that top-k, top-p (of the top-k set's mass) and min-p (of the
    largest probability) keep.  want_probs: also the processed distribution,
    spec_verify's draft_probs.  `out` may supply preallocated outputs by
    name (tokens, prob, kept, probs); `status` an int32 [1] device tensor that
    receives SV_BAD_* bits."""
    dt = _dtype(logits, "logits")
    dev = _cuda(logits, "logits")
    shape = logits.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("logits must be [..., V]")
    V = shape[-1]
    _fits(V)
    lead = shape[:-1]
    rows = logits.numel() // V
    _need(uniforms, "uniforms", _F32, lead, dev)
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
    top_k = min(max(int(top_k), 0), 0x7FFFFFFF)  # (more than every row has, for what a 32-bit number does not hold)
    with _on(dev, stream) as s:
        tokens = prob = kept = probs = None
        if out:
            tokens, prob, kept, probs = (out.get(k) for k in ("tokens", "prob", "kept", "probs"))
            for t, name, dtype, oshape in ((tokens, "tokens", torch.int32, lead), (prob, "prob", _F32, lead),
                                           (kept, "kept", torch.int32, lead), (probs, "probs", _F32, shape)):
                if t is not None:
                    _need(t, name, dtype, oshape, dev)
        if tokens is None:
            tokens = torch.empty(lead, dtype=torch.int32, device=dev)
        if prob is None:
            prob = torch.empty(lead, dtype=_F32, device=dev)
        if kept is None:
            kept = torch.empty(lead, dtype=torch.int32, device=dev)
        if probs is None and want_probs:
            probs = torch.empty(shape, dtype=_F32, device=dev)
        rc = N.lib().sv_sample_logits(logits.data_ptr(), dt, uniforms.data_ptr(), float(temperature), top_k, float(top_p),
                                      float(min_p), rows, V,
                                      tokens.data_ptr(), prob.data_ptr(), kept.data_ptr(), _ptr(probs), _ptr(status), s)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return SampleResult(tokens, prob, kept, probs, status)


# ------------------------------------------------------------- trees

@dataclass
class TreeResult:
    out_tokens: torch.Tensor           # [B, N] int32: the accepted path's tokens, the final token, then -1
    out_nodes: torch.Tensor            # [B, N] int32: the accepted path's node ids, then -1
    num_emitted: torch.Tensor          # [B] int32
    accept_prob: torch.Tensor | None   # [B, N] fp32: min(1, r(x)/q(x)) of each tested node, -1 otherwise
    status: torch.Tensor | None = None


def sv_tree_workspace_bytes(B: int, nodes: int, V: int) -> int:
    return int(N.lib().sv_tree_workspace_bytes(int(B), int(nodes), int(V)))


def spec_verify_tree(logits: torch.Tensor, draft_probs: torch.Tensor, parent: torch.Tensor, tokens: torch.Tensor,
                     uniforms: torch.Tensor, temperature: float, *, want_probs: bool = True,
                     workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> TreeResult:
    """Verification of a candidate tree (multi-step speculative sampling):
    logits [B, N, V] bf16 / fp32 (row i: the target after node i's path),
    draft_probs [B, N, V] fp32 (row i: the draft distribution of node i's
    children), parent / tokens [B, N] int32, uniforms [B, N] fp32.  workspace
    as for spec_verify."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, N, V]")
    B, Nn, V = logits.shape
    dev = logits.device
    dt = N.SV_BF16 if logits.dtype == torch.bfloat16 else (N.SV_FP32 if logits.dtype == torch.float32 else None)
    if dt is None:
        raise TypeError("logits must be bfloat16 or float32")
    _check(logits, "logits", logits.dtype, (B, Nn, V), dev)
    _check(draft_probs, "draft_probs", torch.float32, (B, Nn, V), dev)
    _check(parent, "parent", torch.int32, (B, Nn), dev)
    _check(tokens, "tokens", torch.int32, (B, Nn), dev)
    _check(uniforms, "uniforms", torch.float32, (B, Nn), dev)
    need = sv_tree_workspace_bytes(B, Nn, V)
    if need == 0 and B > 0:
        raise SpecVerifyError(N.SV_EUNSUPPORTED)
    stream = stream or torch.cuda.current_stream(dev)
    if workspace is None:
        workspace = default_workspace(dev, need, stream)
    elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must hold {need} bytes on {dev}")
    if status is not None:
        _check(status, "status", torch.int32, (1,), dev)
    res = TreeResult(out_tokens=torch.empty((B, Nn), dtype=torch.int32, device=dev),
                     out_nodes=torch.empty((B, Nn), dtype=torch.int32, device=dev),
                     num_emitted=torch.empty((B,), dtype=torch.int32, device=dev),
                     accept_prob=torch.empty((B, Nn), dtype=torch.float32, device=dev) if want_probs else None,
                     status=status)
    rc = N.lib().spec_verify_tree(
        logits.data_ptr(), dt, draft_probs.data_ptr(), parent.data_ptr(), tokens.data_ptr(), uniforms.data_ptr(),
        float(temperature), B, Nn, V, res.out_tokens.data_ptr(), res.out_nodes.data_ptr(),
        res.num_emitted.data_ptr(), _ptr(res.accept_prob), _ptr(status), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), stream.cuda_stream)
    if rc != N.SV_OK:
        raise SpecVerifyError(rc)
    return res
