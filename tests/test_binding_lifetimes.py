"""What prepared calls and workspaces keep alive and in order, without a GPU (nothing is launched)."""
import gc
import weakref

import pytest
import torch

import sparse_moe_expert_router_amd as moe


def _bank(E=4, H=256, F=128):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    return {"fmt": "bf16", "gate": z(E, F, H), "up": z(E, F, H), "down": z(E, H, F)}


def _few(bank, shared):
    return moe.FewTokenLayer(torch.zeros((4, 256), dtype=torch.bfloat16), 2, bank, shared, max_tokens=4,
                             ws=moe.Workspace(torch.device("cpu")))


def _layer(bank, shared):
    return moe.LayerCall(torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((4, 256), dtype=torch.bfloat16), 2, bank, shared)


@pytest.mark.parametrize("make", [_few, _layer])
def test_a_prepared_call_keeps_the_weights_it_points_to(make):
    """The caller may put other tensors into the dicts afterwards; the call's own stay where its pointers say."""
    bank, shared = _bank(), _bank(E=1)
    call = make(bank, shared)
    for d, st in ((bank, call.st), (shared, call.sh)):
        for name in ("gate", "up", "down"):
            old, at = weakref.ref(d[name]), d[name].data_ptr()
            d[name] = torch.zeros_like(d[name])
            gc.collect()
            assert old() is not None and old().data_ptr() == at == getattr(st, name).w


class _Stream:
    """Stands for a stream: writes down what it is made to wait for."""

    def __init__(self, ptr):
        self.cuda_stream, self.waits = ptr, []

    def wait_stream(self, other):
        self.waits.append(other)


def test_a_few_token_layer_on_another_stream_waits_for_the_one_before(monkeypatch):
    """The workspace was made on, or last used on, another stream, whose work may still use its memory."""
    a, b, capture = _Stream(1), _Stream(2), _Stream(3)
    now = [a]
    calls = []

    class Device:
        def __init__(self, t):
            self.stream = now[0].cuda_stream

        def call(self, name, *args):
            calls.append((now[0], [len(s.waits) for s in (a, b, capture)], args[-1]))

    monkeypatch.setattr(moe._lib, "_Device", Device)
    monkeypatch.setattr(moe._lib, "_current_stream", lambda device: now[0])
    monkeypatch.setattr(moe._lib, "_capturing", lambda device: now[0] is capture)
    few = _few(_bank(), None)
    few.ws_buf = type("Buffer", (), {"record_stream": lambda self, s: None})()
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    few(x)
    assert a.waits == []
    now[0] = b
    few(x), few(x)
    assert b.waits == [a]
    now[0] = a
    few(x)
    assert a.waits == [b] and b.waits == [a]
    now[0] = capture            # a stream under capture must not wait for one that is not
    few(x)
    assert capture.waits == []
    now[0] = a                  # and nothing outside waits for a capture
    few(x)
    assert a.waits == [b]
    assert [s.cuda_stream for s, _, _ in calls] == [p for _, _, p in calls] == [1, 2, 2, 1, 3, 1]
    assert calls[1][1] == [0, 1, 0]     # the wait comes before the call


def test_a_workspace_that_grows_keeps_the_buffer_of_a_captured_call(monkeypatch):
    """A graph goes on using the buffer that its calls were recorded with."""
    capturing = [False]
    monkeypatch.setattr(moe._lib, "_stream_capturing", lambda: capturing[0])
    ws = moe.Workspace(torch.device("cpu"))
    ws._gpu = True                          # asks whether the stream records a graph
    eager = weakref.ref(ws.get(100)[0])
    ws.get(200)
    gc.collect()
    assert eager() is None                  # nothing but the workspace used it
    capturing[0] = True
    in_graph = [weakref.ref(ws.get(n)[0]) for n in (150, 300)]
    capturing[0] = False
    buf, n = ws.get(1000)
    gc.collect()
    assert n == 1000 and all(r() is not None and r() is not buf for r in in_graph)
