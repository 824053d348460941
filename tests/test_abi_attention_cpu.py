"""CPU-only checks of the attention layers' C ABI: arguments are refused on the host before any CUDA call."""
import ctypes

import pytest

EINVAL, EUNSUPPORTED = 1, 4
FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_decode_gb300 import _lib
    return _lib.load()


def wrap(L, k=FAKE, v=FAKE, pages=10, page=16, layers=2, hkv=2, d=128, dtype=BF16):
    h = ctypes.c_void_p()
    return L.kv_page_pool_wrap(k, v, pages, page, layers, hkv, d, dtype, ctypes.byref(h)), h


def test_pool_geometry(L):
    assert L.kv_page_pool_wrap(FAKE, FAKE, 10, 16, 1, 2, 128, BF16, None) == EINVAL
    assert wrap(L, k=None)[0] == EINVAL and wrap(L, v=None)[0] == EINVAL
    assert wrap(L, k=FAKE + 8)[0] == EINVAL
    assert wrap(L, pages=0)[0] == EINVAL and wrap(L, layers=0)[0] == EINVAL and wrap(L, hkv=0)[0] == EINVAL
    assert wrap(L, dtype=2)[0] == EINVAL
    assert wrap(L, page=24)[0] == EUNSUPPORTED and wrap(L, page=8)[0] == EUNSUPPORTED
    assert wrap(L, d=96)[0] == EUNSUPPORTED
    assert wrap(L, pages=2 ** 30, hkv=4)[0] == EUNSUPPORTED
    rc, h = wrap(L)
    assert rc == 0 and L.kv_page_pool_k(h) == FAKE and L.kv_page_pool_v(h) == FAKE and L.kv_page_pool_num_pages(h) == 10
    assert L.kv_page_pool_destroy(h) == 0 and L.kv_page_pool_destroy(None) == 0
    assert L.kv_page_pool_k(None) is None and L.kv_page_pool_num_pages(None) == 0


def prologue(L, h, **kw):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, pool=h, layer=0, rope=FAKE, pos=64, rot=64, inter=0, qn=None, kn=None,
             eps=1e-6, table=FAKE, mp=4, sl=FAKE, cu=FAKE, out=FAKE, hq=4, rows=1, T=1, dtype=BF16, stream=None)
    a.update(kw)
    return L.attn_prologue(*a.values())


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=None), dict(v=None), dict(pool=None), dict(table=None), dict(sl=None),
                                 dict(cu=None), dict(out=None), dict(out=FAKE + 2), dict(layer=2), dict(layer=-1), dict(hq=3),
                                 dict(hq=0), dict(rows=-1), dict(rows=0), dict(T=-1), dict(mp=0), dict(dtype=F32), dict(dtype=7),
                                 dict(qs=511), dict(qs=516), dict(ks=248), dict(q=FAKE + 2), dict(rot=8), dict(rot=144),
                                 dict(rot=-16), dict(rope=None), dict(rope=FAKE + 4), dict(pos=0), dict(qn=FAKE, eps=-1.0),
                                 dict(kn=FAKE + 4)])
def test_prologue_refusals(L, bad):
    _, h = wrap(L)
    assert prologue(L, h, **bad) == EINVAL
    assert L.gdn_last_error()
    L.kv_page_pool_destroy(h)


def test_nothing_to_do(L):
    _, h = wrap(L)
    assert prologue(L, h, T=0, rows=0, q=None, table=None, sl=None, cu=None) == 0
    assert L.paged_attention(None, 0, h, 0, None, 1, None, None, 1.0, None, 4, 0, 0, None, 0, BF16, None) == 0
    assert L.kv_pages_copy(h, None, None, 0, None, None) == 0
    assert L.kv_pages_reserve(FAKE, 1, 1, FAKE, 1, 16, None, None, 0, None, None) == 0
    assert L.kv_pages_free(FAKE, 1, 1, None, FAKE, 1, None, 0, None) == 0
    assert L.rope_table(None, 16, 0, 1.0, None, None) == 0
    L.kv_page_pool_destroy(h)


@pytest.mark.parametrize("bad", [dict(q=None), dict(qs=8), dict(pool=None), dict(scale=0.0), dict(scale=float("inf")), dict(scale=-1.0),
                                 dict(out=None), dict(out=FAKE + 8), dict(hq=5), dict(layer=2), dict(table=None), dict(rows=0)])
def test_attention_refusals(L, bad):
    _, h = wrap(L)
    a = dict(q=FAKE, qs=512, pool=h, layer=0, table=FAKE, mp=4, sl=FAKE, cu=FAKE, scale=0.1, out=FAKE, hq=4, rows=1, T=1, ws=FAKE,
             wb=1 << 40, dtype=BF16, stream=None)
    a.update(bad)
    assert L.paged_attention(*a.values()) == EINVAL
    L.kv_page_pool_destroy(h)


def test_table_refusals(L):
    _, h = wrap(L)
    assert L.kv_pages_reserve(None, 1, 1, FAKE, 1, 16, FAKE, FAKE, 1, FAKE, None) == EINVAL
    assert L.kv_pages_reserve(FAKE, 1, 1, FAKE, 1, 16, FAKE, FAKE, 4097, FAKE, None) == EINVAL
    assert L.kv_pages_reserve(FAKE, 1, 1, FAKE, 1, 17, FAKE, FAKE, 1, FAKE, None) == EUNSUPPORTED
    assert L.kv_pages_reserve(FAKE, 1, 2 ** 30, FAKE, 1, 16, FAKE, FAKE, 1, FAKE, None) == EUNSUPPORTED
    assert L.kv_pages_reserve(FAKE, 1, 1, FAKE, 1, 16, FAKE, None, 1, FAKE, None) == EINVAL
    assert L.kv_pages_fork(FAKE, 1, 1, FAKE, FAKE, 1, 16, FAKE, FAKE, -1, FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert L.kv_pages_fork(FAKE, 1, 1, FAKE, FAKE, 1, 16, FAKE, FAKE, 1, FAKE, FAKE, None, FAKE, None) == EINVAL
    assert L.kv_pages_fork(FAKE, 1, 1, None, FAKE, 1, 16, FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert L.kv_pages_free(FAKE, 0, 1, FAKE, FAKE, 1, FAKE, 1, None) == EINVAL
    assert L.kv_pages_free(FAKE, 1, 1, FAKE, FAKE, 1, None, 1, None) == EINVAL
    assert L.kv_pages_compact(FAKE, 1, 1, FAKE, 1, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert L.kv_pages_compact(FAKE, 1, 1, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert L.kv_pages_copy(h, FAKE, None, 1, None, None) == EINVAL
    assert L.kv_pages_copy(None, FAKE, FAKE, 1, None, None) == EINVAL
    assert L.kv_pages_copy(h, FAKE, FAKE, -1, None, None) == EINVAL
    for bad in ((8, 4, 1.0), (0, 4, 1.0), (20, 4, 1.0), (16, -1, 1.0), (16, 4, float("nan"))):
        assert L.rope_table(FAKE, *bad, FAKE, None) == EINVAL
    L.kv_page_pool_destroy(h)


def test_rope_frequencies():
    """The scalings' closed forms, on the CPU."""
    import math

    import torch

    from gated_deltanet_decode_gb300 import rope_inv_freq
    plain, one = rope_inv_freq(64, 500000.0)
    assert one == 1.0 and plain.dtype == torch.float64 and plain.shape == (32,)
    assert torch.allclose(plain, 500000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-14)
    assert torch.allclose(rope_inv_freq(64, 500000.0, {"type": "linear", "factor": 8})[0], plain / 8, rtol=1e-14)
    ntk = rope_inv_freq(64, 500000.0, {"type": "ntk", "factor": 8})[0]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 8, rel_tol=1e-12)
    y, m = rope_inv_freq(64, 500000.0, {"type": "yarn", "factor": 8, "original": 8192, "mscale": 1.5})
    assert m == 1.5 and (y <= plain).all() and (y >= plain / 8 - 1e-18).all() and y[0] == plain[0]
    for bad in ((63, 1e4, None), (0, 1e4, None), (64, 1e4, {"type": "other", "factor": 2}), (64, 1e4, {"type": "ntk", "factor": 0})):
        with pytest.raises(ValueError):
            rope_inv_freq(*bad)
