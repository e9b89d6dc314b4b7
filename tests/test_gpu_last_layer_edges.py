"""The last layer's operators where their callers or their numbers leave the
ordinary: several widths of one kernel, from several host threads and in one
graph; values near the ends of the fp32 range; infinite scales."""
import ctypes
import threading

import pytest
import torch

import last_layer_ref as R
import speculative_decoding_sampling_gb300 as sv
from speculative_decoding_sampling_gb300 import _native as N

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float32


def _bits(t):
    t = t.cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ------------------------------------------------------------- one kernel, several widths

def _norm_args(x, res, pre, out, res_out, stream):
    """sv_block_norm's arguments, converted once (bf16 all round)."""
    M, d = x.shape
    vp, f = ctypes.c_void_p, ctypes.c_float
    return (vp(x.data_ptr()), N.SV_BF16, vp(res.data_ptr()), N.SV_BF16, None, None, ctypes.c_int64(1),
            vp(pre.data_ptr()), N.SV_BF16, f(0.0), f(1.0), f(1.0), f(1e-6), ctypes.c_int64(M), d,
            vp(res_out.data_ptr()), vp(out.data_ptr()), N.SV_BF16, None, vp(stream.cuda_stream))


def test_norm_widths_on_several_host_threads():
    """Rows of 4096, 1024 and 8192 values need different amounts of shared
    memory of one kernel: calls from three host threads at once, each on its
    own stream, all succeed and give what the same calls give alone."""
    jobs = []
    for i, d in enumerate((4096, 1024, 8192)):
        x, res, pre = (R.rand(s, 10 * i + k, BF).to(DEV) for k, s in enumerate(((700, d), (700, d), (d,))))
        jobs.append((x, res, pre, sv.sv_block_norm(x, res, pre), torch.empty_like(x), torch.empty_like(x),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(jobs)), [set() for _ in jobs]

    def work(job, seen):
        x, res, pre, _, out, res_out, stream = job
        fn, args = N.lib().sv_block_norm, _norm_args(x, res, pre, out, res_out, stream)
        start.wait()
        for _ in range(4000):
            seen.add(fn(*args))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, codes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert codes == [{N.SV_OK}] * len(jobs)
    for _, _, _, want, out, res_out, _ in jobs:
        assert torch.equal(_bits(out), _bits(want.hidden)) and torch.equal(_bits(res_out), _bits(want.residual))


def test_norm_widths_in_one_graph():
    """Both widths captured into one graph, the second branch on a stream of
    its own that joins before the quantisation; replayed with new inputs."""
    xs = [R.rand((700, d), d, BF).to(DEV) for d in (4096, 1024)]
    ws = [R.rand((d,), d + 1, BF).to(DEV) for d in (4096, 1024)]
    call = lambda i: sv.sv_block_norm(xs[i], xs[i], ws[i], hidden_dtype=BF)  # noqa: E731
    want = [call(0), call(1)]
    sv.sv_quantize_fp8(want[0].hidden)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        a = call(0)
        with torch.cuda.stream(side):
            b = call(1)
        main.wait_stream(side)
        q = sv.sv_quantize_fp8(a.hidden)
        c = call(1)
    for k in range(3):
        for i, x in enumerate(xs):
            x.copy_(R.rand(x.shape, 50 + 2 * k + i, BF))
        g.replay()
        want = [call(0), call(1)]
        wq = sv.sv_quantize_fp8(want[0].hidden)
        torch.cuda.synchronize()
        for got, ref in ((a, want[0]), (b, want[1]), (c, want[1])):
            assert torch.equal(_bits(got.hidden), _bits(ref.hidden))
            assert torch.equal(_bits(got.residual), _bits(ref.residual))
        assert torch.equal(_bits(q[0]), _bits(wq[0])) and torch.equal(q[1], wq[1])


@pytest.mark.parametrize("M", [64, 351, 607, 608])
@pytest.mark.parametrize("d", [1536, 1537])
def test_norm_row_counts_up_to_the_staying_ctas(M, d):
    """Row counts on both sides of the change of kernel, and a width that
    never changes: the same rows within the same bounds."""
    x, res, pre = R.rand((M, d), 1, BF), R.rand((M, d), 2, FP, 3.0), R.rand((d,), 3, BF, 0.3)
    post, gate = R.rand((d,), 4, BF, 0.3), R.rand((1, d), 5, BF)
    h, r, eh, er = R.norm64(x, res, pre, post, gate, offset=1.0)
    dv = lambda t: t.to(DEV)  # noqa: E731
    got = sv.sv_block_norm(dv(x), dv(res), dv(pre), post_weight=dv(post), gate=dv(gate), weight_offset=1.0,
                           hidden_dtype=FP)
    assert R.within(got.residual.cpu(), r, er, FP) and R.within(got.hidden.cpu(), h, eh, FP)


# ------------------------------------------------------------- ends of the range

def _norm(x, res, pre, post=None, gate=None, hidden=FP, **kw):
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    return sv.sv_block_norm(dv(x), dv(res), dv(pre), post_weight=dv(post), gate=dv(gate), hidden_dtype=hidden,
                            branch_scale=kw.get("bs", 1.0))


@pytest.mark.parametrize("M", [5, 700])
@pytest.mark.parametrize("d", [1024, 1000])
def test_norm_factor_before_gate_and_weight(M, d):
    """x times gate times weight past the fp32 range, their product with the
    norm's factor well inside it; and a row whose mean square is past the
    range, which normalises to 0 before the gate."""
    x, res, pre = R.rand((M, d), 1), R.rand((M, d), 2), R.rand((d,), 3)
    post, gate = R.rand((d,), 4) * 1e11, R.rand((M, d), 5) * 1e11
    x[1] *= 1e17
    bs = 1e-16
    h, r, eh, er = R.norm64(x, res, pre, post, gate, bs=bs)
    got = _norm(x, res, pre, post, gate, bs=bs)
    assert R.within(got.residual.cpu(), r, er, FP) and R.within(got.hidden.cpu(), h, eh, FP)
    x[2] = 1e38
    post, gate = post * 1e-11, gate * 1e-11
    got = _norm(x, res, pre, post, gate * 16)
    assert torch.equal(got.residual[2].cpu(), res[2])
    assert got.hidden.isfinite().all()


@pytest.mark.parametrize("M,d", [(M, d) for M in (5, 700) for d in (8192, 4096, 1000, 300, 96, 4101)] + [(5, 20000)])
def test_norm_of_large_rows(M, d):
    """Rows whose sum of squares is past the fp32 range while their mean
    square is inside it, beside ordinary rows, as x (under a post norm) and as
    residual; past the mean square's own range a row normalises to 0."""
    x, res, pre, post = R.rand((M, d), 1), R.rand((M, d), 2), R.rand((d,), 3), R.rand((d,), 4)
    sign = torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0)
    # mean square 3e37: the sum is past 3.4e38 from 12 values on
    x[1], res[3] = 5.5e18 * sign, 5.5e18 * sign.flip(0)
    x[4], res[4] = 4e18 * sign, -4e18 * sign
    h, r, eh, er = R.norm64(x, res, pre, post)
    got = _norm(x, res, pre, post)
    assert R.within(got.residual.cpu(), r, er, FP) and R.within(got.hidden.cpu(), h, eh, FP)
    assert got.hidden[1].count_nonzero() > 0 and got.hidden[3].count_nonzero() > 0
    res[0] = 3e19 * sign                                    # mean square 9e38
    clean = got.hidden[1:].clone()
    got = _norm(x, res, pre, post)
    assert (got.hidden[0] == 0).all() and got.residual[0].isfinite().all()
    assert torch.equal(_bits(got.hidden[1:]), _bits(clean))


@pytest.mark.parametrize("M", [5, 700])
def test_norm_of_tiny_rows_under_a_tiny_eps(M):
    """Values whose squares are near the smallest normal number, with an eps
    that does not hide them."""
    d, eps = 8192, 1e-38
    x, res, pre = torch.zeros(M, d), R.rand((M, d), 2) * 2.0 ** -60, R.rand((d,), 3)
    eps32 = float(torch.tensor(eps))
    h, r, eh, er = R.norm64(x, res, pre, eps=eps32)
    got = sv.sv_block_norm(x.to(DEV), res.to(DEV), pre.to(DEV), eps=eps, hidden_dtype=FP)
    assert R.within(got.residual.cpu(), r, er, FP) and R.within(got.hidden.cpu(), h, eh, FP)


# ------------------------------------------------------------- infinite scales

@pytest.mark.parametrize("M,V,d", [(6, 700, 256), (140, 700, 256), (300, 20003, 144), (1, 130, 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_infinite_scales_give_nan_logits(M, V, d, value):
    """A scale that is not finite makes NaN of the logits it belongs to, and
    of no other; so do two scales whose product is past the fp32 range."""
    h, hs, w, ws = R.head_operands(M, V, d, seed=2)
    clean = sv.sv_lm_head_logits_fp8(*(t.to(DEV) for t in (h, hs, w, ws))).cpu()
    nb, vb = R.blocks(d), R.blocks(V)
    row, wb = M // 2, vb - 1
    hs[row, nb - 1] = value
    ws[wb, 0] = value
    got = sv.sv_lm_head_logits_fp8(*(t.to(DEV) for t in (h, hs, w, ws))).cpu()
    bad = torch.zeros(M, V, dtype=torch.bool)
    bad[row] = True
    bad[:, wb * 128:] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[~bad])
    hs[row, nb - 1], ws[wb, 0] = 3e30, 1.0
    ws[0, nb - 1] = 3e30
    got = sv.sv_lm_head_logits_fp8(*(t.to(DEV) for t in (h, hs, w, ws))).cpu()
    assert got[row, :128].isnan().all()


@pytest.mark.parametrize("B", [4, 60])
@pytest.mark.parametrize("where", ["weights", "hidden"])
def test_fused_reports_infinite_scales(B, where):
    """An infinite scale of a weight block with a single id reaches every
    sequence, one of a hidden row its own: SV_BAD_ROW, nothing emitted."""
    K, V, d = 3, 257, 256
    h, hs, w, ws = R.head_operands(B * (K + 1), V, d, seed=3, dyadic=True)
    if where == "weights":
        ws[2, 1] = float("inf")
    else:
        hs[(K + 1) * 1, 0] = float("inf")
    g = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    res, logits = sv.spec_verify_lm_head_fp8(h.view(B, K + 1, d).to(DEV), hs.view(B, K + 1, 2).to(DEV), w.to(DEV),
                                             ws.to(DEV), None, tokens.to(DEV),
                                             torch.rand((B, K + 1), generator=g).to(DEV), 0.9, status=status)
    assert int(status.item()) == sv.SV_BAD_ROW
    if where == "weights":
        assert logits[..., 256].isnan().all() and logits[..., :256].isfinite().all()
        assert (res.num_emitted == 0).all() and (res.out_tokens == -1).all()
    else:
        assert logits[1, 0].isnan().all()
        assert int(res.num_emitted[1]) == 0 and (res.num_emitted[torch.arange(B) != 1] >= 1).all()


# ------------------------------------------------------------- the widest rows

@pytest.mark.parametrize("d", [2 ** 31 - 8, 2 ** 31 - 1, 2 ** 31 - 129])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_rows_as_wide_as_an_int(d, rows):
    """Widths at the end of 32 bits, three rows: the ends of every row are
    quantised as they are alone, and the scales lie where they belong."""
    nb = R.blocks(d)
    n = d - (nb - 3) * 128                                  # the last three blocks, the last one short
    x = torch.zeros((3, d), dtype=BF, device=DEV)
    head, tail = R.rand((3, 256), 1, BF).to(DEV), R.rand((3, n), 2, BF).to(DEV)
    x[:, :256], x[:, -n:] = head, tail
    v, s = sv.sv_quantize_fp8(x, rows)
    hv, hs = sv.sv_quantize_fp8(head, rows)
    tv, ts = sv.sv_quantize_fp8(tail, rows)
    assert s.shape == (3 if rows == 1 else 1, nb)
    assert torch.equal(s[:, :2], hs) and torch.equal(s[:, -3:], ts)
    assert torch.equal(_bits(v[:, :256]), _bits(hv)) and torch.equal(_bits(v[:, -n:]), _bits(tv))
    mid = v.view(torch.uint8)[:, 256:d - n]
    assert all(int(mid[i].count_nonzero()) == 0 for i in range(3))
    assert (s[:, 2:-3] == torch.tensor(R.AMAX_FLOOR, device=DEV) / 448).all()
