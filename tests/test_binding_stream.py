"""The binding's look-up of torch's current stream, on the host: a stand-in for the GPU's part of torch."""
import os
import sys
import threading

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def fb(monkeypatch):
    from binary_basis_lut_amd import build as B
    if B.is_stale():
        B.build()
    from binary_basis_lut_amd import fluxbin

    class Stream:
        cuda_stream = 5

    monkeypatch.setattr(fluxbin, "_raw_stream", None)
    monkeypatch.setattr(fluxbin, "_device", None, raising=False)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 5 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return fluxbin


def test_streams_given_and_current(fb):
    class Stream:
        cuda_stream = 9

    assert fb._stream(7) == 7 and fb._stream(Stream()) == 9
    assert fb._stream(None) == 5 and fb._stream(None) == 5  # before and after the look-up is kept
    assert fb._raw_stream is not None


def test_nothing_is_kept_before_torch_runs_on_a_gpu(fb, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    assert fb._stream(None) == 5 and fb._raw_stream is None


def test_a_thread_that_looks_between_any_two_steps_gets_a_stream(fb):
    """Another thread asks for the stream after every single bytecode step of the first look-up."""
    first, wrong = [], []

    def other():
        try:
            if fb._stream(None) != 5:
                wrong.append("another handle")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    def ask():
        kept = fb._raw_stream, fb._device  # the other thread must not finish the look-up for this one
        t = threading.Thread(target=other)
        t.start()
        t.join()
        fb._raw_stream, fb._device = kept

    def trace(frame, event, arg):
        if frame.f_code is not fb._stream.__code__:
            return None
        frame.f_trace_opcodes = True
        if event == "opcode":
            first.append(frame.f_lasti)
            sys.settrace(None)
            ask()
            sys.settrace(trace)
        return trace

    before = sys.gettrace()
    sys.settrace(trace)
    try:
        assert fb._stream(None) == 5
    finally:
        sys.settrace(before)
    assert len(first) > 10 and not wrong, wrong


def test_a_forked_child_is_refused_as_torch_refuses_it(fb, monkeypatch):
    """The parent's streams mean nothing in a child: there torch itself has to answer again."""
    assert fb._stream(None) == 5 and fb._raw_stream is not None

    def refuse(device=None):
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    pid = os.fork()
    if pid == 0:
        status = 1
        try:
            torch.cuda.is_initialized, torch.cuda.current_stream = lambda: False, refuse  # as torch does in a child
            try:
                fb._stream(None)
            except RuntimeError:
                status = 0
        finally:
            os._exit(status)
    assert os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]) == 0
    assert fb._raw_stream is not None and fb._stream(None) == 5  # the parent goes on as before
