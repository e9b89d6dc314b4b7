"""Who shares a default workspace, without a GPU: streams and capture are
stand-ins, the zero fill is on the CPU."""
import contextlib
import threading

import pytest
import torch

from speculative_decoding_sampling_gb300 import binding

DEV = torch.device("cuda", 0)


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw
        self.device = DEV


@pytest.fixture
def cuda(monkeypatch):
    """The current stream of each host thread, whether it is being captured,
    and where each zero fill was queued."""
    class State(threading.local):
        stream, capturing = Stream(1), False

    st, fills, zeros = State(), [], torch.zeros

    @contextlib.contextmanager
    def enter(stream):
        before, st.stream = st.stream, stream
        try:
            yield
        finally:
            st.stream = before

    def fill(*shape, device=None, **kw):
        fills.append(st.stream.cuda_stream)
        return zeros(*shape, **kw)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: st.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: st.capturing)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch, "zeros", fill)
    st.fills = fills
    # a thread of its own: nothing is cached for it yet, and nothing stays behind
    return st, lambda f: _on_thread(f, st)


def _on_thread(f, st):
    out = []

    def body():
        try:
            out.append(f())
        except BaseException as e:  # noqa: BLE001  (handed to the test's thread)
            out.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if isinstance(out[0], BaseException):
        raise out[0]
    return out[0]


def test_streams_do_not_share(cuda):
    st, on_thread = cuda

    def body():
        a = binding.default_workspace(DEV, 1000)
        st.stream = Stream(2)
        b = binding.default_workspace(DEV, 1000)
        assert a.data_ptr() != b.data_ptr()
        assert binding.default_workspace(DEV, 500) is b and st.stream.cuda_stream == 2
        st.stream = Stream(1)
        assert binding.default_workspace(DEV, 1000) is a
        # named while another stream is current: that stream's, filled there
        c = binding.default_workspace(DEV, 1000, Stream(3))
        assert c is not a and c is not b and st.stream.cuda_stream == 1
        assert binding.default_workspace(DEV, 1000, Stream(2)) is b

    on_thread(body)
    assert st.fills == [1, 2, 3]


def test_growth_replaces_one_streams_workspace(cuda):
    st, on_thread = cuda

    def body():
        a, b = binding.default_workspace(DEV, 300), binding.default_workspace(DEV, 300, Stream(2))
        big = binding.default_workspace(DEV, 5000)
        assert big.numel() >= 5000 and a.numel() < 5000 and int(big.count_nonzero()) == 0
        assert binding.default_workspace(DEV, 300) is big
        assert binding.default_workspace(DEV, 300, Stream(2)) is b

    on_thread(body)


def test_host_threads_do_not_share(cuda):
    _, on_thread = cuda
    a = on_thread(lambda: binding.default_workspace(DEV, 1000))
    b = on_thread(lambda: binding.default_workspace(DEV, 1000))   # the same stream
    assert a.data_ptr() != b.data_ptr()


def test_captured_calls_do_not_share(cuda):
    st, on_thread = cuda

    def body():
        st.capturing = True
        a, b = binding.default_workspace(DEV, 1000), binding.default_workspace(DEV, 1000)
        assert a.data_ptr() != b.data_ptr()
        st.capturing = False
        c = binding.default_workspace(DEV, 1000)   # not one whose fill has only been recorded
        assert c is not a and c is not b and binding.default_workspace(DEV, 1000) is c

    on_thread(body)
