"""Calls without a workspace of their own that overlap: on two streams, from
two host threads, and in two captured graphs that are replayed at once.  Each
gives what it gives alone."""
import threading

import pytest
import torch

import last_layer_ref as R
import speculative_decoding_sampling_gb300 as sv
import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T = 0.9


def _drafts(B, K, V, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.softmax(torch.randn((B, K, V), generator=g), -1)
    tok = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32)
    return q.to(DEV), tok.to(DEV), torch.rand((B, K + 1), generator=g).to(DEV)


def _fp8_head(seed, B=16, K=4, V=20000, d=256):
    h, hs, w, ws = R.head_operands(B * (K + 1), V, d, seed=seed, dyadic=True)
    args = (h.view(B, K + 1, d).to(DEV), hs.view(B, K + 1, -1).to(DEV), w.to(DEV), ws.to(DEV), *_drafts(B, K, V, seed))
    return lambda **kw: sv.spec_verify_lm_head_fp8(*args, T, **kw)[0]


def _bf16_head(seed, B=16, K=4, V=20000, d=256):
    h, W = R.rand((B, K + 1, d), seed, torch.bfloat16), R.rand((V, d), seed + 1, torch.bfloat16, 0.1)
    args = (h.to(DEV), W.to(DEV), *_drafts(B, K, V, seed))
    return lambda **kw: sv.spec_verify_lm_head(*args, T, **kw)[0]


def _verify(seed, B=32, K=4, V=20000):
    logits = R.rand((B, K + 1, V), seed, torch.bfloat16, 3.0).to(DEV)
    args = (logits, *_drafts(B, K, V, seed))
    return lambda **kw: sv.spec_verify(*args, T, **kw)


def _tree(seed, B=16, V=20000):
    par = torch.tensor(synth.TREE_SHAPES["tree16"], dtype=torch.int32)
    N = par.numel()
    q, tok, u = _drafts(B, N, V, seed)
    logits = R.rand((B, N, V), seed, torch.bfloat16, 3.0).to(DEV)
    args = (logits, q, par.expand(B, N).contiguous().to(DEV), tok, u[:, :N].contiguous())
    return lambda **kw: sv.spec_verify_tree(*args, T, **kw)


CALLS = dict(fp8_head=_fp8_head, bf16_head=_bf16_head, verify=_verify, tree=_tree)


def _same(a, b):
    """Token decisions are equal; so are the numbers, bit for bit."""
    for k, v in vars(b).items():
        if v is not None:
            assert torch.equal(getattr(a, k), v), k


def _alone(call):
    r = call()
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("kind", CALLS)
def test_two_streams(kind):
    calls = [CALLS[kind](seed) for seed in (1, 2)]
    want = [_alone(c) for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(40):
        for i, c in enumerate(calls):
            got[i].append(c(stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for r in got[i]:
            _same(r, want[i])
    for c, w in zip(calls, want):
        _same(_alone(c), w)


@pytest.mark.parametrize("kind", CALLS)
@pytest.mark.parametrize("own_streams", [False, True])
def test_two_host_threads(kind, own_streams):
    """On the current stream of both, or on a stream each."""
    calls = [CALLS[kind](seed) for seed in (3, 4)]
    want = [_alone(c) for c in calls]
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        kw = dict(stream=torch.cuda.Stream()) if own_streams else {}
        start.wait()
        for _ in range(40):
            got[i].append(calls[i](**kw))
        torch.cuda.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in (0, 1):
        assert len(got[i]) == 40
        for r in got[i]:
            _same(r, want[i])


@pytest.mark.parametrize("kind", CALLS)
def test_two_captured_graphs(kind):
    calls = [CALLS[kind](seed) for seed in (5, 6)]
    want = [_alone(c) for c in calls]
    graphs, out = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.append(c())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        _same(calls[0](), want[0])       # an eager call beside them
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        _same(o, w)


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_two_stages_in_a_graph_need_a_workspace():
    logits, q, tok, u = (R.rand((2, 3, 500), 1, torch.bfloat16).to(DEV), *_drafts(2, 2, 500, 1))
    out = {k: v for k, v in vars(_alone(lambda: sv.spec_verify(logits, q, tok, u, T))).items()}
    with pytest.raises(ValueError, match="workspace"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            sv.sv_verify_rows(logits, q, tok, u, T, out=out, workspace=None)
    torch.cuda.synchronize()
