"""CPU tests of where the binding's outputs come from when the caller names a stream: from that stream's memory,
recorded for the stream that the caller goes on with.  Memory of the caller's own stream may still be in use by work
queued there, which a kernel on the named stream does not wait for.  No device is touched: streams, memory and the
library are stand-ins."""
import contextlib
import types

import pytest
import torch

from gated_delta_rule_40_gb300 import kda

CALLER = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=1, name="caller")
SIDE = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=2, name="side")


class _Memory:
    """A tensor's address, the stream it was allocated on and the streams it was recorded for."""

    def __init__(self, shape, dtype, stream):
        self.shape, self.dtype, self.device, self.allocated, self.recorded = shape, dtype, None, stream, []

    def data_ptr(self):
        return 4096

    def numel(self):
        return 1

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def made(monkeypatch):
    """The allocations of a call, in order."""
    log, current = [], [CALLER]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*shape, dtype=None, device=None):
        log.append(_Memory(shape, dtype, current[-1]))
        return log[-1]

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(kda, "_device_of", lambda t: 0)
    monkeypatch.setattr(kda, "_arg", lambda *a: 4096)
    monkeypatch.setattr(kda, "_check", lambda *a, **kw: None)
    lib = types.SimpleNamespace(kda_bwd_workspace_size=lambda *a: 1024)
    for name in kda.declared_symbols():
        if not hasattr(lib, name):
            setattr(lib, name, lambda *a: 0)
    monkeypatch.setattr(kda, "_lib", lib)
    return log


def _tensors(*shapes, dtype=torch.bfloat16):
    return [torch.zeros(s, dtype=dtype) for s in shapes]


def _attn_fwd(stream):
    q, k = _tensors((1, 4, 2, 128), (1, 4, 1, 128))
    kda.kda_attn_fwd(q, k, k, 0.1, stream=stream)


def _attn_paged(stream):
    q, c = _tensors((4, 2, 128), (3, 1, 16, 128))
    i = torch.zeros(2, dtype=torch.int32)
    kda.kda_attn_paged(q, c, c, i[None], i, i, 0.1, stream=stream)


def _page_plan(stream):
    i = torch.zeros(2, dtype=torch.int32)
    kda.kda_page_plan(i, i, i, i[:1], i[:, None], 16, 4, stream=stream)


SERVING = [(_attn_fwd, 2), (_attn_paged, 2), (_page_plan, 5)]


@pytest.mark.parametrize("call,outputs", SERVING)
def test_outputs_come_from_the_stream_that_writes_them(made, call, outputs):
    call(SIDE)
    assert len(made) == outputs
    for m in made:
        assert m.allocated is SIDE and CALLER in m.recorded


def _linear(name, *extra, lead=(1, 4), K=128, state=None, gate=True, **kw):
    """A call of the linear-attention entry points on [*lead, heads, K] inputs."""
    q, v = _tensors((*lead, 2, K), (*lead, 2, K))
    args = [q, q, v] + ([v, torch.zeros(*lead, 2)] if gate else []) + [torch.zeros(2), 0.1, *extra]
    if state is not None:
        args.append(torch.zeros(state))
    return lambda stream: getattr(kda, name)(*args, stream=stream, **kw)


LINEAR = [
    (_linear("kda_fwd"), 2), (_linear("kda_fwd_scalar_gate"), 2), (_linear("kda_fwd_bf16_state"), 2),
    (_linear("kda_fwd_noalloc"), 1), (_linear("kda_la_fwd", gate=False), 2),
    (_linear("kda_decode_step", lead=(3,), state=(3, 2, 128, 128)), 1),
    (_linear("kda_la_decode", lead=(3,), state=(3, 2, 128, 128), gate=False), 1),
    (_linear("kda_decode_tokens", lead=(3, 4), state=(3, 2, 128, 128)), 1),
    (_linear("kda_bwd", torch.zeros((1, 4, 2, 128))), 8)]   # seven gradients and the workspace


@pytest.mark.parametrize("call,outputs", LINEAR)
def test_linear_attention_outputs_come_from_the_stream_that_writes_them(made, call, outputs):
    call(SIDE)
    assert len(made) == outputs
    for m in made:
        assert m.allocated is SIDE and CALLER in m.recorded


@pytest.mark.parametrize("call,outputs", SERVING + LINEAR)
def test_without_a_stream_nothing_is_recorded(made, monkeypatch, call, outputs):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    call(None)
    assert len(made) == outputs
    assert all(m.allocated is CALLER and not m.recorded for m in made)
