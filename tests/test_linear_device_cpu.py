"""The calls of linear attention and of attention over shared prefixes go to their tensors' device, whatever the current one
is.  No GPU: the library and the devices are stand-ins."""
import types

import pytest
import torch

import gated_deltanet_decode_gb300 as G
from test_attn_device_cpu import ONE, POOL, Q, ROWS, T, Tensor, calls  # noqa: F401 (a fixture)


class Heads(Tensor):
    """Activations [tokens][heads][d], dense."""

    def __init__(self, *shape):
        super().__init__(*shape)
        self.dtype = torch.bfloat16

    def stride(self):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)


STATES = types.SimpleNamespace(tensor=Tensor(9), hk=1, hv=2, dk=64, dv=64, handle=16, _p=None)
QK, V, G1 = Heads(2, 1, 64), Heads(2, 2, 64), Tensor(2)
BOUNDS, PREFIX, CU = Tensor(2), Tensor(2, 2), Tensor(3)


@pytest.mark.parametrize("name,call", [
    ("linear_attention_decode", lambda: G.linear_attention_decode(QK, QK, V, G1, STATES, ROWS, ROWS, out=V)),
    ("linear_attention_prefill", lambda: G.linear_attention_prefill(QK, QK, V, G1, STATES, CU, ROWS, ROWS, out=V, workspace=Tensor(64))),
    ("kv_pages_shared", lambda: G.kv_pages_shared(T, ROWS, CU, BOUNDS, 16, out=PREFIX)),
    ("paged_attention_shared", lambda: G.paged_attention_shared(Q, POOL, T, ROWS, CU, BOUNDS, PREFIX, out=Q, workspace=Tensor(64))),
])
def test_calls_go_to_their_tensors_device(calls, name, call):  # noqa: F811
    assert STATES.tensor.device == ONE
    call()
    assert calls == [(name, 1, ("stream of", 1))]
