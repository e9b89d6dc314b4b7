"""The LM head on e4m3 operands with block scales, the verification fused
behind it, and the last layer run together, through the binding."""
import numpy as np
import pytest
import torch

import last_layer_ref as R
import speculative_decoding_sampling_gb300 as sv
import synth
from oracle import parity
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
OUT = ("out_tokens", "num_emitted", "accept_flags", "accept_prob", "residual_mass")


def _dev(ops):
    return [t.to(DEV) for t in ops]


def _logits(ops, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sv.sv_lm_head_logits_fp8(*_dev(ops), status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out.cpu()


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


# (M, V, d): a single token, row counts around the 32-row warps and the 128 /
# 256-row tiles, vocabularies below and above one tile, odd ones (single
# stores), d below one block, ending inside a block, wrapping the ring
SHAPES = [(1, 256, 128), (1, 1, 16), (5, 7, 16), (31, 33, 112), (33, 300, 144), (45, 1001, 1040), (127, 520, 256),
          (128, 5000, 272), (129, 2056, 512), (130, 31, 128), (200, 9999, 144), (256, 777, 1024), (257, 1000, 384),
          (300, 4097, 640), (513, 512, 2048), (40, 20000, 4096), (3, 45000, 64),
          # wide tiles whose rows start at every alignment: vocabularies 3, 1, 6, 4 and 7 above a multiple of 8
          (131, 32003, 144), (260, 40001, 128), (50, 36006, 128), (7, 44004, 16), (129, 65527, 32),
          # a last row tile of at most 128 rows: 1, 33, 64, 65, 128 of them, and 129 (not one)
          (257, 9000, 256), (289, 9001, 384), (320, 12000, 128), (577, 20003, 64), (384, 9504, 640), (641, 30000, 272),
          (385, 9000, 128), (896, 20000, 2176)]


@pytest.mark.parametrize("M,V,d", SHAPES, ids=[f"M{m}_V{v}_d{d}" for m, v, d in SHAPES])
def test_logits(M, V, d):
    ops = R.head_operands(M, V, d, seed=M + V + d)
    z, err = R.head64(*ops)
    assert R.within(_logits(ops), z, err, torch.bfloat16)


@pytest.mark.parametrize("M,V,d", [(1, 777, 512), (64, 4096, 128), (129, 1000, 1040), (300, 640, 320)])
def test_logits_dyadic_bit_exact(M, V, d):
    """Entries 0 and +-1/2 with power-of-two scales: every partial sum is
    exact, so the logits are the exact ones rounded once."""
    ops = R.head_operands(M, V, d, seed=5, dyadic=True)
    z, _ = R.head64(*ops)
    assert torch.equal(_logits(ops), z.float().to(torch.bfloat16))


@pytest.mark.parametrize("M,V", [(3, 1500), (200, 1500), (300, 9000), (384, 9002)])
def test_every_value_and_scale_reaches_its_place(M, V):
    """One non-zero per operand row and scales that differ everywhere: each
    logit is a single product, so an index that is off shows as a wrong one."""
    d = 1168
    nb = R.blocks(d)
    g = torch.Generator().manual_seed(M)
    kk = torch.randint(0, d, (V,), generator=g)
    w = torch.zeros(V, d)
    w[torch.arange(V), kk] = (torch.randint(1, 8, (V,), generator=g) * 0.25)
    h = torch.randint(-8, 9, (M, d), generator=g).float()
    hs = 1 + torch.arange(M * nb).view(M, nb).float() / 4096
    ws = 1 + torch.arange(R.blocks(V) * nb).view(-1, nb).float() / 128
    ops = (h.to(torch.float8_e4m3fn), hs, w.to(torch.float8_e4m3fn), ws)
    z, _ = R.head64(*ops)
    # one product of the two scales (rounded once) and one with the exact inner sum
    assert R.within(_logits(ops), z, 3 * R.U * z.abs(), torch.bfloat16)


# row counts of several 128-row tiles whose waves cost less on single CTAs than
# on pairs, and the same ids a wave below, where pairs take them
@pytest.mark.parametrize("M,V,d", [(257, 20003, 128), (288, 32000, 272), (321, 24006, 1040), (384, 50001, 64),
                                   (513, 20008, 144), (640, 35000, 128), (384, 9700, 272), (384, 12960, 144),
                                   (384, 12961, 144), (1100, 33001, 32)])
def test_logits_over_several_row_tiles(M, V, d):
    test_logits(M, V, d)


@pytest.mark.parametrize("M,V", [(300, 20010), (513, 20003)])
def test_places_over_several_row_tiles(M, V):
    test_every_value_and_scale_reaches_its_place(M, V)


def test_leading_dims_and_empty():
    h, hs, w, ws = _dev(R.head_operands(12, 300, 144, seed=1))
    flat = sv.sv_lm_head_logits_fp8(h, hs, w, ws)
    lead = sv.sv_lm_head_logits_fp8(h.view(4, 3, 144), hs.view(4, 3, 2), w, ws)
    assert lead.shape == (4, 3, 300) and torch.equal(lead.view(12, 300), flat)
    assert sv.sv_lm_head_logits_fp8(h[:0], hs[:0], w, ws).shape == (0, 300)


@pytest.mark.parametrize("M", [6, 140])
def test_nan_and_infinite_scales_stay_in_place(M):
    h, hs, w, ws = R.head_operands(M, 700, 256, seed=2)
    clean = _logits((h, hs, w, ws))
    hs[1, 0] = float("nan")
    ws[2, 1] = float("inf")                     # ids 256..383
    got = _logits((h, hs, w, ws))
    rows = torch.arange(M) != 1
    ids = (torch.arange(700) < 256) | (torch.arange(700) >= 384)
    assert got[1].isnan().all()
    assert torch.equal(got[rows][:, ids], clean[rows][:, ids])
    assert not got[rows][:, ~ids].isfinite().any()


def test_logits_write_only_their_buffer():
    for M, V in ((5, 333), (131, 520), (40, 4099)):
        ops = _dev(R.head_operands(M, V, 208, seed=3))
        keep = [t.clone() for t in ops]
        o, st = Guarded((M, V), torch.bfloat16), Guarded((1,), torch.int32, fill=0)
        sv.sv_lm_head_logits_fp8(*ops, out=o.t, status=st.t)
        torch.cuda.synchronize()
        assert o.guards_intact() and st.guards_intact() and int(st.t.item()) == 0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ops, keep))


@pytest.mark.parametrize("shift", [1, 2, 5])
@pytest.mark.parametrize("M,V", [(5, 40008), (140, 32008), (3, 77)])
def test_logits_at_any_alignment(M, V, shift):
    """An output that starts between 16-byte boundaries (a slice of a larger
    buffer): the same logits, and nothing around them."""
    ops = _dev(R.head_operands(M, V, 80, seed=shift))
    want = sv.sv_lm_head_logits_fp8(*ops)
    buf = torch.full((M * V + 16,), -7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[shift:shift + M * V].view(M, V)
    sv.sv_lm_head_logits_fp8(*ops, out=out)
    assert torch.equal(out, want)
    assert (buf[:shift] == -7).all() and (buf[shift + M * V:] == -7).all()


def test_offsets_past_32_bits():
    """More than 2^31 logits, and more than 2^31 weights: sampled entries."""
    M, V, d = 16500, 131072, 16
    h, hs, w, ws = R.head_operands(M, V, d, seed=8, dyadic=True)
    got = sv.sv_lm_head_logits_fp8(*_dev((h, hs, w, ws)))
    for r0, v0 in ((0, 0), (M - 40, V - 500), (M // 2, V // 2)):
        z, _ = R.head64(h[r0:r0 + 40], hs[r0:r0 + 40], w[v0 // 128 * 128:v0 + 500], ws[v0 // 128:])
        z = z[:, v0 % 128:]
        assert torch.equal(got[r0:r0 + 40, v0:v0 + 500].cpu(), z.float().to(torch.bfloat16))
    del got
    M, V, d = 2, 2097152, 1040
    h, hs, _, _ = R.head_operands(M, 1, d, seed=9, dyadic=True)
    _, _, w, ws = R.head_operands(1, 1280, d, seed=10, dyadic=True)
    wd = torch.zeros((V, d), dtype=torch.uint8, device=DEV)
    wd[-1280:] = w.view(torch.uint8).to(DEV)
    wsd = torch.ones((R.blocks(V), R.blocks(d)), device=DEV)
    wsd[-10:] = ws.to(DEV)
    got = sv.sv_lm_head_logits_fp8(h.to(DEV), hs.to(DEV), wd.view(torch.float8_e4m3fn), wsd)
    z, _ = R.head64(h, hs, w, ws)
    assert torch.equal(got[:, -1280:].cpu(), z.float().to(torch.bfloat16))
    assert int(got[:, :-1280].count_nonzero()) == 0


# ------------------------------------------------------------- fused

def _fused(ops, B, K, q, tokens, u, T, **kw):
    h, hs, w, ws = _dev(ops)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    res, logits = sv.spec_verify_lm_head_fp8(
        h.view(B, K + 1, -1), hs.view(B, K + 1, -1), w, ws, None if q is None else torch.from_numpy(q).to(DEV),
        torch.from_numpy(tokens).to(DEV), torch.from_numpy(u).to(DEV), T, status=status, **kw)
    torch.cuda.synchronize()
    cand = {k: getattr(res, k).cpu().numpy() for k in OUT}
    cand["status"] = int(status.item())
    return cand, logits


FUSED = [(24, 3, 1000, 256), (24, 0, 4097, 128), (17, 8, 32000, 256), (5, 4, 130, 64), (40, 3, 257, 192),
         (1, 0, 500, 128), (1, 4, 32003, 144), (30, 4, 32001, 64), (64, 4, 40000, 64),
         (60, 4, 9000, 128), (96, 3, 9003, 64)]


@pytest.mark.parametrize("onehot", [False, True], ids=["dense", "onehot"])
@pytest.mark.parametrize("B,K,V,d", FUSED, ids=[f"B{b}_K{k}_V{v}_d{d}" for b, k, v, d in FUSED])
def test_fused_verify_against_oracle(orc, B, K, V, d, onehot):
    """Dyadic operands make the logits exact, so the oracle verifies the very
    logits the kernels see."""
    T = 0.8
    ops = R.head_operands(B * (K + 1), V, d, seed=B + 7 * K + V, dyadic=True)
    z, _ = R.head64(*ops)
    z = z.float().to(torch.bfloat16).view(B, K + 1, V)
    q, tokens, u = synth.drafts_for(z.double().numpy(), T, 1.0, seed=V + K, onehot_p=0.6 if onehot else None)
    cand, logits = _fused(ops, B, K, q, tokens, u, T)
    assert cand["status"] == 0
    assert torch.equal(logits.cpu(), z)
    rep = parity.compare(orc, _bits(z), q, tokens, u, T, cand)
    assert rep.ok(), rep.summary()


@pytest.mark.parametrize("B,K,V,d", [(32, 4, 5000, 512), (12, 8, 9001, 144), (3, 2, 40000, 256)])
def test_fused_matches_unfused(B, K, V, d):
    """Any scales: the fused call agrees with spec_verify on the logits it
    wrote (the statistics are merged in another order than the row pass's,
    hence 1e-5 on the probabilities), and those are sv_lm_head_logits_fp8's."""
    T = 0.7
    ops = R.head_operands(B * (K + 1), V, d, seed=77)
    z, _ = R.head64(*ops)
    q, tokens, u = synth.drafts_for(z.view(B, K + 1, V).numpy(), T, 1.0, seed=78)
    cand, logits = _fused(ops, B, K, q, tokens, u, T)
    assert cand["status"] == 0
    assert torch.equal(logits.view(-1, V).cpu(), _logits(ops))
    ref = sv.spec_verify(logits, torch.from_numpy(q).to(DEV), torch.from_numpy(tokens).to(DEV),
                         torch.from_numpy(u).to(DEV), T)
    for k in OUT[:3]:
        assert np.array_equal(cand[k], getattr(ref, k).cpu().numpy()), k
    for k in OUT[3:]:
        assert np.abs(cand[k] - getattr(ref, k).cpu().numpy()).max(initial=0.0) <= 1e-5, k


@pytest.mark.parametrize("B", [4, 60])
def test_fused_bad_row_is_reported(B):
    """A NaN scale in one sequence: that sequence emits nothing, the others
    are as without it."""
    K, V, d, T = 2, 900, 256, 1.0
    h, hs, w, ws = R.head_operands(B * (K + 1), V, d, seed=4, dyadic=True)
    z, _ = R.head64(h, hs, w, ws)
    q, tokens, u = synth.drafts_for(z.view(B, K + 1, V).numpy(), T, 1.0, seed=5)
    clean, _ = _fused((h, hs, w, ws), B, K, q, tokens, u, T)
    hs[1 * (K + 1) + 1, 1] = float("nan")
    got, _ = _fused((h, hs, w, ws), B, K, q, tokens, u, T)
    assert got["status"] == sv.SV_BAD_ROW and got["num_emitted"][1] == 0 and (got["out_tokens"][1] == -1).all()
    others = np.arange(B) != 1
    for k in OUT:
        assert np.array_equal(got[k][others], clean[k][others]), k


@pytest.mark.parametrize("B,K,V,d", [(9, 3, 3000, 128), (50, 3, 700, 128)])
def test_fused_returns_workspace_to_zero(B, K, V, d):
    ops = R.head_operands(B * (K + 1), V, d, seed=12)
    q, tokens, u = synth.drafts_for(np.zeros((B, K + 1, V)), 1.0, 1.0, seed=3)
    ws = Guarded((sv.sv_lm_head_fp8_workspace_bytes(B, K, V),), torch.uint8, fill=0)
    first, _ = _fused(ops, B, K, q, tokens, u, 1.0, workspace=ws.t)
    again, _ = _fused(ops, B, K, q, tokens, u, 1.0, workspace=ws.t)
    assert ws.guards_intact() and int(ws.t.count_nonzero().item()) == 0
    for k in OUT:
        assert np.array_equal(first[k], again[k]), k


def test_fused_captured_graphs_do_not_share_a_workspace():
    """Two captured calls, replayed at once on two streams, and a larger eager
    call between capture and replay (which replaces the shared workspace)."""
    B, K, V, d, T = 8, 3, 4000, 256, 0.9
    sets, graphs = [], []
    for i in range(2):
        ops = R.head_operands(B * (K + 1), V, d, seed=20 + i, dyadic=True)
        z, _ = R.head64(*ops)
        q, tokens, u = synth.drafts_for(z.view(B, K + 1, V).numpy(), T, 1.0, seed=30 + i)
        want, _ = _fused(ops, B, K, q, tokens, u, T)
        h, hs, w, ws = _dev(ops)
        args = (h.view(B, K + 1, d), hs.view(B, K + 1, -1), w, ws, torch.from_numpy(q).to(DEV),
                torch.from_numpy(tokens).to(DEV), torch.from_numpy(u).to(DEV), T)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res, _ = sv.spec_verify_lm_head_fp8(*args)
        sets.append((want, res, args))
        graphs.append(g)
    big = R.head_operands(64 * 9, 6000, 64, seed=3)
    q, tokens, u = synth.drafts_for(np.zeros((64, 9, 6000)), T, 1.0, seed=1)
    _fused(big, 64, 8, q, tokens, u, T)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for want, res, _ in sets:
        for k in OUT:
            assert np.array_equal(want[k], getattr(res, k).cpu().numpy()), k


def test_other_stream():
    ops = _dev(R.head_operands(70, 3000, 512, seed=6))
    want = sv.sv_lm_head_logits_fp8(*ops)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.sv_lm_head_logits_fp8(*ops, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------- together

@pytest.mark.parametrize("B,K", [(1, 0), (2, 4), (40, 4)])
def test_last_layer_together(B, K):
    """From the last block's output to the emitted tokens: norms and
    quantisation, the LM head, then the verification three ways (fused; top-k
    and top-p filtered; and through the unfused logits), with the quantised
    hidden states checked against the 64-bit norms and the logits against the
    64-bit product of the operands that the kernels were given."""
    V, d, T = 5000, 1024, 0.8
    M = B * (K + 1)
    x, res = R.rand((B, K + 1, d), 1, torch.bfloat16), R.rand((B, K + 1, d), 2, torch.float32, 3.0)
    wn, wp = R.rand((d,), 3, torch.bfloat16, 0.1), R.rand((d,), 4, torch.bfloat16, 0.1)
    gate = R.rand((B, 1, d), 5, torch.bfloat16)
    W = R.rand((V, d), 6, torch.bfloat16, 0.09).to(DEV)
    w8, ws = sv.sv_quantize_fp8(W, 128)
    n = sv.sv_block_norm(x.to(DEV), res.to(DEV), wn.to(DEV), post_weight=wp.to(DEV), gate=gate.to(DEV),
                         weight_offset=1.0, hidden_dtype=torch.float8_e4m3fn)
    h64, _, eh, _ = R.norm64(x.view(M, d), res.view(M, d), wn, wp, gate, offset=1.0)
    h8, hs = n.hidden.cpu().view(M, d), n.scales.cpu().view(M, -1)
    sc = R.spread_scales(hs.to(R.F64), 1, M, d)
    assert ((h8.to(R.F64) * sc - h64).abs() <= 2.0 ** -4 * h64.abs() + 2.0 ** -10 * sc + 1.1 * eh + 4 * R.U * h64.abs()).all()
    z, err = R.head64(h8, hs, w8.cpu(), ws.cpu())
    q, tokens, u = synth.drafts_for(z.view(B, K + 1, V).numpy(), T, 0.7, seed=9)
    qd, td, ud = (torch.from_numpy(a).to(DEV) for a in (q, tokens, u))
    fused, logits = sv.spec_verify_lm_head_fp8(n.hidden, n.scales, w8, ws, qd, td, ud, T)
    assert R.within(logits.cpu().view(M, V), z, err, torch.bfloat16)
    split = sv.sv_lm_head_logits_fp8(n.hidden, n.scales, w8, ws)
    assert torch.equal(split, logits)
    plain = sv.spec_verify(split, qd, td, ud, T)
    for k in OUT[:3]:
        assert torch.equal(getattr(fused, k), getattr(plain, k)), k
    filt, kept = sv.sv_filter_logits(split, T, 50, 0.95)
    some = sv.spec_verify(filt, qd, td, ud, T)
    assert int(kept.max()) <= 50 and bool((some.num_emitted >= 1).all())
    last = some.out_tokens.gather(1, some.num_emitted.long()[:, None] - 1)
    row = filt.gather(1, (some.num_emitted.long() - 1)[:, None, None].expand(B, 1, V)).squeeze(1)
    assert bool(row.gather(1, last.long()).isfinite().all())   # the drawn token is one the filter kept


def test_tree_behind_the_fp8_head(orc):
    """A candidate tree verified on logits from the e4m3 head (dyadic, so the
    oracle sees the same logits)."""
    B, V, d, T = 4, 1500, 128, 0.8
    par = np.asarray(synth.TREE_SHAPES["tree16"], np.int32)
    N = len(par)
    ops = R.head_operands(B * N, V, d, seed=40, dyadic=True)
    z, _ = R.head64(*ops)
    zb = z.float().to(torch.bfloat16).view(B, N, V)
    rng = np.random.default_rng(3)
    zq = zb.double().numpy() / T + rng.standard_normal((B, N, V))
    q = np.exp(zq - zq.max(-1, keepdims=True))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    tok = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):
            tok[b, i] = min(V - 1, int(np.searchsorted(np.cumsum(q[b, par[i]].astype(np.float64)), rng.random())))
    u = rng.random((B, N), dtype=np.float32)
    parent = np.tile(par, (B, 1))
    h, hs, w, ws = _dev(ops)
    lg = sv.sv_lm_head_logits_fp8(h.view(B, N, d), hs.view(B, N, -1), w, ws)
    assert torch.equal(lg.cpu(), zb)
    res = sv.spec_verify_tree(lg, *(torch.from_numpy(a).to(DEV) for a in (q, parent, tok, u)), T)
    cand = {k: getattr(res, k).cpu().numpy() for k in ("out_tokens", "out_nodes", "num_emitted", "accept_prob")}
    rep = parity.compare_tree(orc, _bits(zb), q, parent, tok, u, T, cand)
    assert rep.ok(), rep.summary()
