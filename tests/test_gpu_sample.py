"""The draw of tokens on the GPU against a plain 64-bit form: filters, ties,
masks, sizes, refusals by status, and a whole draft step into the
verification."""
import numpy as np
import pytest
import torch

import draft_ref as R
import speculative_decoding_sampling_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# a decision this near an id's boundary (relative to the mass it is a part of) may fall on either side: the masses are
# right to 2^-28 and the boundaries are sums of them
NEAR = 2.0 ** -28


def _logits(rows, V, dtype, sigma=3.0, bias=0.0, seed=0):
    r = np.random.default_rng(seed)
    z = r.normal(0, sigma, (rows, V)) - bias * np.log(np.arange(1, V + 1))
    return torch.from_numpy(z).to(dtype)


def _check(z, u, T, top_k=0, top_p=1.0, min_p=0.0, *, view=None):
    zd = z.to(DEV) if view is None else view
    ud = torch.as_tensor(u, dtype=F32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = sv.sv_sample_logits(zd, ud.to(DEV), T, top_k, top_p, min_p, want_probs=True, status=status)
    only = sv.sv_sample_logits(zd, ud.to(DEV), T, top_k, top_p, min_p)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(only.tokens, r.tokens) and torch.equal(only.kept, r.kept) and torch.equal(only.prob, r.prob)
    probs, tokens = r.probs.cpu().double().numpy(), r.tokens.cpu().numpy()
    for i in range(z.shape[0]):
        token, keep, q, margin = R.sample(z[i].double().numpy(), float(ud[i]), T, top_k, top_p, min_p)
        if margin < NEAR:
            continue
        # q: exp2 in fp32 of a rounded argument of up to 64 (2^-18) and three roundings; ids below 2^-126 are 0
        assert int(r.kept[i]) == keep.sum(), (i, int(r.kept[i]), keep.sum())
        assert (np.abs(probs[i] - q) <= 2.0 ** -17 * q + 2.0 ** -126).all()
        assert not probs[i][~keep].any()
        assert tokens[i] == token, (i, tokens[i], token)
        # the mass as a whole multiple of 2^-40 of the largest
        assert abs(float(r.prob[i]) - q[token]) <= 2.0 ** -23 * q[token] + 2.0 ** -40 * q.max()


FILTERS = [dict(), dict(top_k=1), dict(top_k=50), dict(top_p=0.9), dict(top_p=0.999), dict(top_p=1e-6),
           dict(min_p=0.05), dict(min_p=1.0), dict(min_p=1e-9), dict(top_k=40, top_p=0.8), dict(top_k=2000, top_p=0.95, min_p=0.01),
           dict(top_k=5, min_p=0.3), dict(top_p=0.7, min_p=0.2), dict(top_k=100000, top_p=0.5)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("filt", FILTERS, ids=lambda f: ",".join(f"{k}={v}" for k, v in f.items()) or "none")
def test_filters(dtype, filt):
    for V, T, sigma, bias in ((3001, 0.8, 3.0, 1.1), (32000, 1.0, 3.0, 0.0), (50257, 0.6, 4.0, 0.0)):
        z = _logits(6, V, dtype, sigma, bias, seed=V)
        u = np.random.default_rng(V + 1).random(6, dtype=np.float32)
        u[0] = 0.0
        u[1] = 1 - 2.0 ** -24
        _check(z, u, T, **filt)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 33, 255, 500, 1023, 4097, 16385, 32003, 65537, 128256, 151936])
def test_sizes(dtype, V):
    rows = 3
    z = _logits(rows, V, dtype, 2.0, seed=V)
    u = np.random.default_rng(V).random(rows, dtype=np.float32)
    _check(z, u, 0.9)
    _check(z, u, 0.9, top_k=max(1, V // 3), top_p=0.9)
    _check(z, u, 0.9, top_p=0.95, min_p=0.001)


@pytest.mark.parametrize("rows", [1, 2, 37, 300, 400])
def test_row_counts(rows):
    z = _logits(rows, 5000, BF, 3.0, seed=rows)
    u = np.random.default_rng(rows).random(rows, dtype=np.float32)
    _check(z, u, 0.7, top_k=100, top_p=0.9)
    _check(z, u, 0.7, top_k=900, top_p=0.95)
    _check(z, u, 0.7, top_p=0.99)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_flat_and_tied_rows(dtype):
    """All ids equal, a few values, cuts inside the equal ones: the ids in order."""
    V = 9000
    r = np.random.default_rng(3)
    for z in (np.zeros((4, V)), r.choice([0.0, 1.0, -1.0], (4, V)), np.full((4, V), -3.5)):
        zt = torch.from_numpy(z).to(dtype)
        u = np.array([0.0, 0.3, 0.77, 0.9999], np.float32)
        for f in (dict(), dict(top_k=1), dict(top_k=2345), dict(top_p=0.37), dict(top_k=5000, top_p=0.61),
                  dict(min_p=1.0), dict(top_k=V), dict(top_k=V + 7, top_p=0.5)):
            _check(zt, u, 1.0, **f)
    z = torch.zeros((1, V), dtype=dtype)
    z[0, ::2] = -0.0                              # the same logit
    _check(z, np.array([0.5004], np.float32), 1.0, top_k=4501)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_masked_rows(dtype):
    V = 4000
    z = _logits(6, V, dtype, 3.0, seed=5)
    lowest = torch.finfo(dtype).min
    z[0, 100:] = -np.inf
    z[1, :] = -np.inf
    z[1, 3999] = 1.0                              # one id left
    z[2, 50:] = lowest                            # masked by the type's lowest value
    z[3, :] = lowest                              # ... all of them: equal, kept
    z[4, 1:] = -np.inf
    z[5, ::3] = -np.inf
    u = np.array([0.2, 0.9, 0.5, 0.5, 0.99, 0.1], np.float32)
    for f in (dict(), dict(top_k=60), dict(top_k=2000), dict(top_p=0.9), dict(min_p=0.1), dict(top_k=300, top_p=0.99, min_p=1e-3)):
        _check(z, u, 1.0, **f)


@pytest.mark.parametrize("T", [1e-4, 0.05, 5.0, 300.0])
def test_temperatures(T):
    """From one id that has all the mass to a flat row (windows that hold everything)."""
    for dtype in (BF, F32):
        z = _logits(3, 6000, dtype, 3.0, seed=8)
        u = np.array([0.1, 0.5, 0.95], np.float32)
        for f in (dict(), dict(top_k=3000), dict(top_p=0.9), dict(top_k=4000, top_p=0.9)):
            _check(z, u, T, **f)


def test_large_and_small_logits():
    for scale in (1e-30, 1e3, 1e30):
        z = (_logits(3, 3000, F32, 3.0, seed=2) * scale).to(F32)
        u = np.array([0.1, 0.5, 0.95], np.float32)
        for f in (dict(), dict(top_k=50), dict(top_p=0.9)):
            _check(z, u, 1.0, **f)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_long_rows(dtype):
    """Slices past a list's 16-bit entries, and rows too long for shared memory."""
    for V in (600001, (1 << 21) - 3):
        z = _logits(2, V, dtype, 3.0, seed=V)
        u = np.array([0.3, 0.8], np.float32)
        _check(z, u, 0.7)
        _check(z, u, 0.7, top_k=500, top_p=0.9)
        _check(z, u, 0.7, top_p=0.8)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_unaligned_base(dtype):
    rows, V = 4, 5003
    z = _logits(rows, V, dtype, 3.0, seed=4)
    u = np.array([0.1, 0.4, 0.6, 0.9], np.float32)
    for off in (1, 3):
        buf = torch.zeros(rows * V + 8, dtype=dtype, device=DEV)
        view = buf[off:off + rows * V].view(rows, V)
        view.copy_(z)
        _check(z, u, 0.8, top_p=0.9, view=view)
        _check(z, u, 0.8, view=view)


def test_bad_rows_and_uniforms_are_reported_and_stay_alone():
    V = 3000
    z = _logits(7, V, F32, 3.0, seed=6)
    z[1, 17] = float("nan")
    z[2, 5] = float("inf")
    z[3, :] = -float("inf")
    u = torch.tensor([0.5, 0.5, 0.5, 0.5, 1.0, float("nan"), 0.25])
    for f in (dict(), dict(top_k=10, top_p=0.9)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = sv.sv_sample_logits(z.to(DEV), u.to(DEV), 0.9, want_probs=True, status=status, **f)
        assert int(status.item()) == sv.SV_BAD_ROW | sv.SV_BAD_U
        tokens = r.tokens.cpu().tolist()
        assert tokens[1:6] == [-1] * 5 and not r.prob[1:6].any()
        assert not r.probs[1:4].any() and not r.kept[1:4].any()
        for i in (0, 4, 5, 6):
            token, keep, q, _ = R.sample(z[i].numpy(), 0.0 if i in (4, 5) else float(u[i]), 0.9, **f)
            assert int(r.kept[i]) == keep.sum() and np.abs(r.probs[i].cpu().numpy() - q).max() < 1e-6
            if i in (0, 6):
                assert tokens[i] == token
    status.zero_()
    sv.sv_sample_logits(z[:1].to(DEV), torch.tensor([-0.1], device=DEV), 0.9, status=status)
    assert int(status.item()) == sv.SV_BAD_U


def test_given_outputs_leading_dims_and_no_rows():
    z = _logits(12, 1000, BF, seed=1).view(3, 4, 1000).to(DEV)
    u = torch.rand((3, 4), device=DEV)
    o = dict(tokens=torch.full((3, 4), 7, dtype=torch.int32, device=DEV), probs=torch.full((3, 4, 1000), 2.0, device=DEV))
    r = sv.sv_sample_logits(z, u, 0.8, 20, out=o)
    assert r.tokens is o["tokens"] and r.probs is o["probs"] and r.prob.shape == (3, 4)
    assert torch.equal(r.probs.gather(-1, r.tokens.long()[..., None]).squeeze(-1) > 0, torch.ones((3, 4), dtype=torch.bool, device=DEV))
    e = sv.sv_sample_logits(z[:0], u[:0], 0.8)
    assert e.tokens.shape == (0, 4)


@pytest.mark.parametrize("rows,V", [(3, 4099), (330, 4099), (2, 151936)])
def test_nothing_is_written_beside_the_outputs(rows, V):
    z = _logits(rows, V, BF, 3.0, seed=rows)
    z[1] = float("nan")
    buf = {"tokens": torch.full((rows + 2,), -77, dtype=torch.int32, device=DEV),
           "kept": torch.full((rows + 2,), -77, dtype=torch.int32, device=DEV),
           "prob": torch.full((rows + 2,), -77.0, device=DEV), "probs": torch.full((rows * V + 2 * 64,), -77.0, device=DEV)}
    o = {k: v[1:-1] for k, v in buf.items() if k != "probs"}
    o["probs"] = buf["probs"][64:-64].view(rows, V)
    zd, u = z.to(DEV), torch.rand(rows, device=DEV)
    before = zd.clone()
    for f in (dict(), dict(top_k=50), dict(top_k=600, top_p=0.9), dict(top_p=0.99), dict(min_p=0.1)):
        sv.sv_sample_logits(zd, u, 0.8, out=o, **f)
        for k, v in buf.items():
            edge = 64 if k == "probs" else 1
            assert (v[:edge] == -77).all() and (v[-edge:] == -77).all() and not (o[k] == -77).any(), k
    assert torch.equal(zd.view(torch.int16), before.view(torch.int16))


def test_rows_do_not_depend_on_the_batch():
    z = _logits(200, 4000, BF, seed=12).to(DEV)
    u = torch.rand(200, device=DEV)
    a = sv.sv_sample_logits(z, u, 0.8, 0, 0.9, want_probs=True)
    for i in (0, 99, 199):
        b = sv.sv_sample_logits(z[i:i + 1], u[i:i + 1], 0.8, 0, 0.9, want_probs=True)
        assert torch.equal(a.tokens[i:i + 1], b.tokens) and torch.equal(a.probs[i:i + 1], b.probs)
        assert torch.equal(a.prob[i:i + 1], b.prob) and torch.equal(a.kept[i:i + 1], b.kept)


@pytest.mark.parametrize("filt", FILTERS + [dict(top_k=700), dict(top_k=900, top_p=0.97), dict(top_p=0.98, min_p=1e-4)],
                         ids=lambda f: ",".join(f"{k}={v}" for k, v in f.items()) or "none")
@pytest.mark.parametrize("dtype,V", [(BF, 4099), (BF, 50001), (F32, 12000)], ids=["bf16-4099", "bf16-50001", "fp32-12000"])
def test_large_batches(dtype, V, filt):
    """Many rows (CTAs of another size, another division of the work) against the same rows in small calls, which the
    plain form above checks: bit for bit.  Among them flat, tied, masked and bad rows."""
    rows = 330
    z = _logits(rows, V, dtype, 3.0, seed=V)
    z[3], z[4, :] = 0.0, -1.25
    z[5] = (z[5] / 3).round()                     # a few values, many times each
    z[6, 20:] = -np.inf
    z[7] = z[7].sort(descending=True).values      # the largest in one CTA
    z[8, 0] = 200.0                               # all mass in one id
    z[9] *= 0.05
    z[10, 7], z[11, :] = float("nan"), -np.inf
    z[13], z[14] = -50.0, -50.0
    z[13, 1:1 + 600 * (V // 700):V // 700] = 5.0  # more equal ids than are ranked, fewer than one CTA settles
    z[14, :700] = torch.linspace(3.0, 3.02, 700).to(dtype)   # as many in one bin or two
    zd = z.to(DEV)
    u = torch.from_numpy(np.random.default_rng(V).random(rows, dtype=np.float32)).to(DEV)
    u[12] = 1.0
    a = sv.sv_sample_logits(zd, u, 0.8, filt.get("top_k", 0), filt.get("top_p", 1.0), filt.get("min_p", 0.0), want_probs=True)
    for i in range(0, rows, 30):
        b = sv.sv_sample_logits(zd[i:i + 30], u[i:i + 30], 0.8, filt.get("top_k", 0), filt.get("top_p", 1.0),
                                filt.get("min_p", 0.0), want_probs=True)
        for name in ("tokens", "prob", "kept", "probs"):
            assert torch.equal(getattr(a, name)[i:i + 30], getattr(b, name)), (name, i)


def test_distribution_of_draws():
    """Uniforms on a fine grid: each id is drawn as often as its probability says, to one count."""
    V, n = 50, 4096
    z = _logits(1, V, F32, 2.0, seed=7)
    u = (torch.arange(n, dtype=F32) + 0.5) / n
    r = sv.sv_sample_logits(z.expand(n, V).contiguous().to(DEV), u.to(DEV), 1.0, 0, 0.95)
    counts = np.bincount(r.tokens.cpu().numpy(), minlength=V)
    q = R.sample(z[0].numpy(), 0.5, 1.0, 0, 0.95)[2]
    assert np.abs(counts - n * q).max() <= 1.0 + 1e-3


def test_streams_and_graph():
    z = _logits(16, 8000, BF, seed=3).to(DEV)
    u = torch.rand(16, device=DEV)
    want = sv.sv_sample_logits(z, u, 0.8, 50, 0.9, want_probs=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = sv.sv_sample_logits(z, u, 0.8, 50, 0.9, want_probs=True, stream=side)
    b = sv.sv_sample_logits(z, u, 0.8, 50, 0.9, want_probs=True)
    torch.cuda.synchronize()
    for r in (a, b):
        assert torch.equal(r.tokens, want.tokens) and torch.equal(r.probs, want.probs)
    zz, uu = z.clone(), u.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = sv.sv_sample_logits(zz, uu, 0.8, 50, 0.9, want_probs=True)
    for seed in (1, 2):
        zz.copy_(_logits(16, 8000, BF, seed=seed))
        uu.copy_(torch.rand(16))
        g.replay()
        e = sv.sv_sample_logits(zz, uu, 0.8, 50, 0.9, want_probs=True)
        assert torch.equal(r.tokens, e.tokens) and torch.equal(r.probs, e.probs)


def test_draft_step_into_verification():
    """Hidden states to 4 bits, the draft's head, tokens and q with the target's filters; the target's logits (its own
    head, in e4m3) filtered alike; verification.  With the draft as its own target every token is accepted."""
    B, K, V, d = 8, 4, 4000, 256
    g = torch.Generator(device=DEV).manual_seed(5)
    w = torch.randn((V, d), generator=g, device=DEV) * (3 / d ** 0.5)
    w4 = sv.sv_quantize_fp4(w.to(BF))
    h = torch.randn((B, K + 1, d), generator=g, device=DEV)
    T, top_k, top_p = 0.8, 50, 0.9
    z = torch.empty((B, K + 1, V), dtype=BF, device=DEV)
    tokens, q = torch.empty((B, K), dtype=torch.int32, device=DEV), torch.empty((B, K, V), device=DEV)
    for k in range(K + 1):      # position by position, as a draft does
        z[:, k] = sv.sv_lm_head_logits_fp4(sv.sv_quantize_fp4(h[:, k].contiguous()), w4)
        if k < K:
            r = sv.sv_sample_logits(z[:, k].contiguous(), torch.rand(B, generator=g, device=DEV), T, top_k, top_p,
                                    want_probs=True)
            tokens[:, k], q[:, k] = r.tokens, r.probs
            assert torch.equal(r.probs.gather(-1, r.tokens.long()[:, None])[:, 0] > 0, r.prob > 0)
    both = sv.sv_lm_head_logits_fp4(sv.sv_quantize_fp4(h), w4)
    assert torch.equal(both, z)                   # all positions at once are the same product
    filt, kept = sv.sv_filter_logits(z, T, top_k, top_p)
    u = torch.rand((B, K + 1), generator=g, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    res = sv.spec_verify(filt, q, tokens, u * (1 - 1e-4), T, status=status)
    assert int(status.item()) == 0
    assert (res.num_emitted == K + 1).all() and torch.equal(res.out_tokens[:, :K], tokens)
    # another target: its own head in e4m3
    w8, ws = sv.sv_quantize_fp8(w, 128)
    h8, hs = sv.sv_quantize_fp8(h)
    zt = sv.sv_lm_head_logits_fp8(h8, hs, w8, ws)
    filt, _ = sv.sv_filter_logits(zt, T, top_k, top_p)
    res = sv.spec_verify(filt, q, tokens, u, T, status=status)
    assert int(status.item()) == 0 and (res.num_emitted >= 1).all()
    p = torch.softmax(filt.double() / T, -1)
    a = (p[:, :K].gather(-1, tokens.long()[..., None]) / q.double().gather(-1, tokens.long()[..., None])).squeeze(-1).clamp(max=1)
    assert (res.accept_prob.double() - a).abs().max() < 1e-5
