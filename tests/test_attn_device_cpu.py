"""The attention layers' calls are made with their tensors' device current, whatever the caller's is: PyTorch's default
stream has the handle 0, and a launch on it goes to the current device.  No GPU: the library and the devices are stand-ins."""
import contextlib
import types

import pytest
import torch

import gated_deltanet_decode_gb300 as G

ONE = torch.device("cuda", 1)


class Tensor:
    """What the calls ask of a tensor that the argument checks have passed."""

    def __init__(self, *shape):
        self.shape, self.device, self.dtype = shape, ONE, torch.int32

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def element_size(self):
        return 4

    def dim(self):
        return len(self.shape)


@pytest.fixture
def calls(monkeypatch):
    """(function, current device, stream) of every call into the library; device 0 is current."""
    now, made = [0], []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], torch.device(d).index
        yield
        now[0] = before

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, now[0], a[-1])) or 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(G._lib, "load", lambda *a: Library())
    monkeypatch.setattr(G._lib, "fast", lambda: None)
    monkeypatch.setattr(G, "_raw_stream", lambda dev: ("stream of", dev.index))
    monkeypatch.setattr(G, "_arg", lambda *a: 16)
    monkeypatch.setattr(G, "_ptr", lambda *a: 16)
    monkeypatch.setattr(G, "_token_rows", lambda *a: (16, 128))
    monkeypatch.setattr(G, "_table", lambda t, *a: (16, *t.shape))
    yield made
    assert now == [0]


POOL = types.SimpleNamespace(device=ONE, d=128, hkv=2, dtype=torch.bfloat16, _p=None, _h=None, _code=1)
MOVES = types.SimpleNamespace(src=Tensor(2), dst=Tensor(2), count=Tensor(1), status=Tensor(2),
                              _pointers=lambda n, dev: (16, 16, 16))
Q, T, ROWS = Tensor(3, 4, 128), Tensor(2, 5), Tensor(2)


@pytest.mark.parametrize("name,call", [
    ("attn_prologue", lambda: G.attn_prologue(Q, Q, Q, POOL, None, T, ROWS, Tensor(3), out=Q)),
    ("paged_attention", lambda: G.paged_attention(Q, POOL, T, ROWS, Tensor(3), out=Q, workspace=Tensor(64))),
    ("kv_pages_reserve", lambda: G.kv_pages_reserve(T, ROWS, ROWS, ROWS, 16, status=ROWS)),
    ("kv_pages_fork", lambda: G.kv_pages_fork(T, ROWS, Tensor(9), ROWS, ROWS, 16, MOVES)),
    ("kv_pages_free", lambda: G.kv_pages_free(T, ROWS, Tensor(9), ROWS)),
    ("kv_pages_compact", lambda: G.kv_pages_compact(T, Tensor(2), MOVES, remap=ROWS)),
    ("kv_pages_copy", lambda: G.kv_pages_copy(POOL, MOVES)),
])
def test_calls_go_to_their_tensors_device(calls, name, call):
    call()
    assert calls == [(name, 1, ("stream of", 1))]
