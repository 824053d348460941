"""kv_pages_shared and paged_attention_shared refuse bad arguments on the host (no GPU: nothing is launched)."""
import ctypes

import pytest

from gated_deltanet_decode_gb300 import _lib

EINVAL, EUNSUPPORTED = 1, 4
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    return _lib.load()


@pytest.fixture(scope="module")
def pool(L):
    h = ctypes.c_void_p()
    assert L.kv_page_pool_wrap(FAKE, FAKE, 10, 16, 2, 2, 128, BF16, ctypes.byref(h)) == 0
    yield h
    L.kv_page_pool_destroy(h)


def attention(L, h, **k):
    a = dict(q=FAKE, qs=512, pool=h, layer=0, table=FAKE, mp=4, sl=FAKE, cu=FAKE, bounds=FAKE, groups=1, prefix=FAKE, scale=0.1,
             out=FAKE, hq=4, rows=2, T=2, ws=FAKE, wb=1 << 40, dtype=BF16, stream=None)
    a.update(k)
    return L.paged_attention_shared(*a.values())


@pytest.mark.parametrize("bad", [dict(q=None), dict(pool=None), dict(table=None), dict(sl=None), dict(cu=None), dict(bounds=None),
                                 dict(prefix=None), dict(prefix=FAKE + 4), dict(groups=-1), dict(groups=0), dict(groups=3), dict(out=None), dict(hq=3),
                                 dict(layer=2), dict(rows=-1), dict(T=-1), dict(mp=0), dict(dtype=F32), dict(scale=0.0),
                                 dict(scale=float("nan")), dict(qs=500), dict(ws=None), dict(wb=100), dict(ws=FAKE + 8)])
def test_attention_refusals(L, pool, bad):
    assert attention(L, pool, **bad) == EINVAL
    assert L.gdn_last_error()


def test_workspace(L, pool):
    need = L.paged_attention_shared_workspace_bytes
    assert need(None, 4, 2, 2) == 0 and need(pool, 3, 2, 2) == 0 and need(pool, 4, 0, 2) == 0
    small = need(pool, 4, 2, 2)
    assert small >= 2 * 2 * 4 * (128 * 4 + 8) and need(pool, 4, 2, 200) > small
    assert attention(L, pool, wb=small - 1) == EINVAL
    assert attention(L, pool, T=0, rows=0, groups=0, q=None, table=None, sl=None, cu=None, bounds=None, prefix=None, out=None) == 0


def shared(L, **k):
    a = dict(table=FAKE, rows=3, mp=4, sl=FAKE, cu=FAKE, bounds=FAKE, groups=2, page=16, prefix=FAKE, stream=None)
    a.update(k)
    return L.kv_pages_shared(*a.values())


@pytest.mark.parametrize("bad,code", [(dict(table=None), EINVAL), (dict(sl=None), EINVAL), (dict(cu=None), EINVAL),
                                      (dict(bounds=None), EINVAL), (dict(prefix=None), EINVAL), (dict(prefix=FAKE + 4), EINVAL),
                                      (dict(rows=-1), EINVAL), (dict(mp=0), EINVAL), (dict(groups=4), EINVAL), (dict(groups=0), EINVAL),
                                      (dict(groups=-1), EINVAL), (dict(page=24), EUNSUPPORTED), (dict(mp=2 ** 27), EUNSUPPORTED)])
def test_shared_refusals(L, bad, code):
    assert shared(L, **bad) == code
    assert L.gdn_last_error()


def test_no_rows(L):
    assert shared(L, rows=0, groups=0, table=None, sl=None, cu=None, bounds=None, prefix=None) == 0
