"""What the binding does through torch for a call (a temporary workspace, the largest length)
happens on the call's stream, and the workspace is held until the launch."""
import contextlib
import gc
import weakref

import pytest
import torch

import paged_kv_cache_335_b200 as pa


@pytest.fixture
def current(monkeypatch):
    """Stands in for torch.cuda's streams: the list's last entry is the current one."""
    stack = ["current"]

    class Stream:
        def __init__(self, handle=0):
            self.cuda_stream = handle

    class External(Stream):
        pass

    @contextlib.contextmanager
    def on(st):
        stack.append(st.cuda_stream)
        yield
        stack.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(pa, "_dev", lambda t, name, dtype=None: t.data_ptr())
    return stack


@pytest.mark.parametrize("make,want", [(lambda: None, "current"), (lambda: torch.cuda.Stream(64), 64),
                                       (lambda: 48, 48), (lambda: 1, 0), (lambda: 0, 0)])
def test_allocations_and_maxima_are_the_streams(current, monkeypatch, make, want):
    seen = []
    empty, top = torch.empty, torch.Tensor.max
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(("empty", current[-1])), empty(*a, **k))[1])
    monkeypatch.setattr(torch.Tensor, "max", lambda t: (seen.append(("max", current[-1])), top(t))[1])
    stream = make()
    ws, ptr, size = pa._workspace(100, None, "cpu", stream)
    assert size == 100 and ptr == ws.data_ptr()
    assert pa._longest(torch.tensor([3, 9, 4]), stream) == 9
    assert pa._longest_between(torch.tensor([0, 5, 6, 20]), stream) == 14
    assert seen == [("empty", want), ("max", want), ("max", want)]
    assert current == ["current"]


def test_nothing_to_allocate_or_measure(current):
    assert pa._workspace(0, None, "cpu", 48)[1:] == (0, 0)
    assert pa._longest(torch.tensor([], dtype=torch.int32), 48) == 0
    assert pa._longest_between(torch.tensor([7], dtype=torch.int32), 48) == 0
    mine = torch.zeros(256, dtype=torch.uint8)
    assert pa._workspace(100, mine, "cpu", 48) == (mine, mine.data_ptr(), 256)


def test_a_temporary_workspace_lives_until_the_launch(current, monkeypatch):
    """pa_decode_weights: the entry is called while the workspace still exists."""
    refs, alive = [], []
    empty = torch.empty

    def made(*a, **k):
        t = empty(*a, **{**k, "device": "cpu"})
        refs.append(weakref.ref(t))
        return t

    def entry(*args):
        gc.collect()
        alive.append([r() is not None for r in refs])
        return pa.PA_OK

    kc = torch.zeros((4, 1, 16, 64))
    q = torch.zeros((1, 2, 64))
    w = torch.zeros((1, 1, 32))
    tables, lens = torch.zeros((1, 2), dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    out = empty((1, 2, 64))
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(pa, "pa_decode_weights_workspace_size", lambda *a: 4096)
    pa._decode_weights_call(entry, (), out, w, q, kc, kc, tables, lens, 0.1, torch.float32, None, 0, None, 48)
    assert alive == [[True]]
