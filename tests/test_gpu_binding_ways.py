"""The attention layers' two bindings, the C++ one and ctypes, make the same calls and raise the same errors."""
import pytest
import torch

from attn_helpers import DEV, Cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["cpp", "ctypes"])
def way(request, gdn, monkeypatch):
    from gated_deltanet_decode_gb300 import _lib
    if request.param == "ctypes":
        monkeypatch.setattr(_lib, "_fast", None)
    elif _lib.fast() is None:
        pytest.skip("the C++ binding was not built")
    return gdn


def results(G):
    c = Cache([77, 0, 300], "bf16", 2, 128, 16, seed=1)
    pool, table, lens, cu = c.pool(G), i32(c.table), i32(c.lens), i32([0, 3, 4, 5])
    g = torch.Generator().manual_seed(5)
    x = torch.randn(5, 12 * 128, generator=g).bfloat16().to(DEV)
    q, k, v = (x[:, a * 128:b * 128].view(5, b - a, 128) for a, b in ((0, 8), (8, 10), (10, 12)))
    w = torch.rand(128, generator=g).to(DEV)
    out = torch.empty(5, 8, 128, dtype=torch.bfloat16, device=DEV)
    a = G.attn_prologue(q, k, v, pool, G.rope_table(64, 400), table, lens, cu, q_norm=w, interleaved=True)
    b = G.attn_prologue(q, k, v, pool, None, table, lens, cu, k_norm=w, out=out)
    assert b is out
    o = G.paged_attention(a, pool, table, lens, cu)
    o2 = torch.empty_like(o)
    ws = torch.empty(G.paged_attention_workspace_bytes(pool, 8, 3, 5), dtype=torch.uint8, device=DEV)
    assert G.paged_attention(b, pool, table, lens, cu, scale=0.2, out=o2, workspace=ws) is o2
    t, refs, n = i32([[3, 5, 7, 0], [0] * 4, [0] * 4]), i32([0, 0, 0, 1, 0, 1, 0, 1, 0, 0]), i32([40, 0, 0])
    m = G.KVPageMoves(2)
    small = G.KVPagePool(10, 16, 2, 128, k=pool.k[:, :10].contiguous(), v=pool.v[:, :10].contiguous())
    assert G.kv_pages_fork(t, n, refs, i32([0, 0]), i32([1, 2]), 16, m) is m
    G.kv_pages_copy(small, m)
    G.kv_pages_free(t, n, refs, i32([0]))
    return [a, b.clone(), o, o2, pool.k, pool.v, t, refs, n, m.src, m.dst, m.count, small.k, small.v]


def test_both_give_the_same(gdn, monkeypatch):
    from gated_deltanet_decode_gb300 import _lib
    if _lib.fast() is None:
        pytest.skip("the C++ binding was not built")
    one = results(gdn)
    monkeypatch.setattr(_lib, "_fast", None)
    for x, y in zip(one, results(gdn)):
        assert torch.equal(x, y)


def test_both_refuse(way):
    c = Cache([20], "bf16", 2, 128, 16)
    pool, table, lens, cu = c.pool(way), i32(c.table), i32(c.lens), i32([0, 1])
    q, k = (torch.zeros(1, h, 128, dtype=torch.bfloat16, device=DEV) for h in (4, 2))
    with pytest.raises(way.GDNError) as e:
        way.paged_attention(q, pool, table, lens, cu, scale=-1.0)
    assert e.value.code == 1 and "scale" in str(e.value)
    with pytest.raises(way.GDNError):
        way.attn_prologue(q, k, k, pool, None, table, lens, cu, layer=5)
    with pytest.raises(TypeError):
        way.paged_attention(q.half(), pool, table, lens, cu)
    with pytest.raises(ValueError):
        way.paged_attention(q, pool, table, lens, i32([0, 1, 2]))
    with pytest.raises(ValueError):
        way.attn_prologue(q, k, q, pool, None, table, lens, cu)
    m = way.KVPageMoves(1)
    with pytest.raises(way.GDNError):
        way.kv_pages_fork(table, lens, i32([0] * 9), i32([0]), i32([0]), 17, m)
    with pytest.raises(ValueError):
        way.kv_pages_free(table, i32([1, 2]), i32([0] * 9), i32([0]))
    with pytest.raises(TypeError):
        way.kv_pages_free(table, lens.long(), i32([0] * 9), i32([0]))
