"""Linear attention's C entry points refuse bad arguments on the host (no GPU: nothing is launched)."""
import ctypes

import pytest

from gated_deltanet_decode_gb300 import _lib

EINVAL = 1
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    return _lib.load()


@pytest.fixture(scope="module")
def pool(L):
    h = ctypes.c_void_p()
    assert L.gdn_state_pool_wrap(FAKE, 9, _lib.gdn_dims(2, 4, 64, 32), ctypes.byref(h)) == 0
    yield h
    L.gdn_state_pool_destroy(h)


GOOD = dict(q=FAKE, qs=128, k=FAKE, ks=128, v=FAKE, vs=128, g=FAKE, per=1, cu=FAKE, read=FAKE, write=FAKE, scale=1.0, out=FAKE,
            rows=2, tokens=5, in_place=0, ws=FAKE, wb=1 << 40, dtype=BF16)


def decode(L, pool, **k):
    a = dict(GOOD, **k)
    return L.linear_attention_decode(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["g"], a["per"], pool, a["read"],
                                     a["write"], a["scale"], a["out"], a["rows"], a["in_place"], a["dtype"], None)


def prefill(L, pool, **k):
    a = dict(GOOD, **k)
    return L.linear_attention_prefill(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["g"], a["per"], pool, a["cu"], a["read"],
                                      a["write"], a["scale"], a["out"], a["rows"], a["tokens"], a["in_place"], a["ws"], a["wb"],
                                      a["dtype"], None)


BAD = [dict(rows=-1), dict(dtype=2), dict(scale=float("inf")), dict(scale=float("nan")), dict(read=None), dict(write=None),
       dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(out=None), dict(q=FAKE + 2), dict(v=FAKE + 8), dict(out=FAKE + 4),
       dict(qs=120), dict(ks=127), dict(vs=100), dict(qs=129), dict(vs=132)]


@pytest.mark.parametrize("wrong", BAD, ids=lambda w: str(next(iter(w.items()))))
@pytest.mark.parametrize("call", [decode, prefill])
def test_refusals(L, pool, call, wrong):
    assert call(L, pool, **wrong) == EINVAL
    assert L.gdn_last_error()


def test_null_pool_and_prefill_only(L, pool):
    assert decode(L, None) == EINVAL and prefill(L, None) == EINVAL
    assert prefill(L, pool, tokens=-1) == EINVAL
    assert prefill(L, pool, cu=None) == EINVAL
    need = L.linear_attention_prefill_workspace_bytes(pool, 2, 5, BF16)
    if need:
        assert prefill(L, pool, ws=None) == EINVAL and prefill(L, pool, wb=need - 1) == EINVAL and prefill(L, pool, ws=FAKE + 64) == EINVAL


def test_nothing_to_do(L, pool):
    assert decode(L, pool, rows=0, q=None, k=None, v=None, g=None, out=None, read=None, write=None) == 0
    assert prefill(L, pool, rows=0, tokens=0, q=None, k=None, v=None, g=None, out=None, read=None, write=None, cu=None) == 0
    assert L.linear_attention_prefill_workspace_bytes(None, 1, 1, BF16) == 0
