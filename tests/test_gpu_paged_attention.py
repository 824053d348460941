"""paged_attention on the GPU against its definition in 64 bits: head layouts,
lengths around page and tile edges, padding, masked places that hold NaN,
strides, streams, graphs, and bad tables."""
import numpy as np
import pytest
import torch

from attn_helpers import DEV, TYPES, Cache, attention_ref, check_attention, i32, packed

pytestmark = pytest.mark.gpu


def run(G, c, new, hq, seed=1, scale=None, layer=0, q=None, **kw):
    T = int(sum(new))
    if q is None:
        q = torch.randn(T, hq, c.d, generator=torch.Generator().manual_seed(seed)).to(TYPES[c.dtype])
    out = G.paged_attention(q.to(DEV), c.pool(G), i32(c.table), i32(c.lens), i32(packed(new)), layer=layer, scale=scale,
                            **kw)
    return q, out


HEADS = [(136, 1, 64), (4, 4, 64), (12, 4, 64), (16, 4, 128), (7, 1, 128), (10, 2, 128), (16, 2, 256), (6, 2, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_decode_rows_of_many_lengths(gdn, dtype, hq, hkv, d):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 0, 700]
    c = Cache(lens, dtype, hkv, d, 16, seed=d + hq, poison=float("nan"))
    new = [1] * len(lens)
    q, out = run(gdn, c, new, hq)
    check_attention(out, *attention_ref(c, q, new, d ** -0.5), dtype)
    assert (out[13] == 0).all()
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_chunks_over_a_cache(gdn, dtype, hq, hkv, d, page):
    new = [5, 1, 0, 67, 1, 130, 2]
    lens = [5, 300, 40, 200, 0, 131, 129]
    c = Cache(lens, dtype, hkv, d, page, seed=page + hq, poison=float("nan"))
    q, out = run(gdn, c, new, hq)
    check_attention(out, *attention_ref(c, q, new, d ** -0.5), dtype)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,n,length", [(4, 1, 64, 513, 513), (8, 2, 128, 300, 1500), (2, 1, 256, 257, 900), (1, 1, 128, 600, 601)])
def test_one_long_chunk(gdn, dtype, hq, hkv, d, n, length):
    c = Cache([length], dtype, hkv, d, 32, seed=n, poison=float("nan"))
    q, out = run(gdn, c, [n], hq)
    check_attention(out, *attention_ref(c, q, [n], d ** -0.5), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_contexts_few_rows(gdn, dtype):
    lens, new = [40003, 17, 23001], [1, 1, 3]
    c = Cache(lens, dtype, 2, 128, 64, seed=3, poison=float("nan"))
    q, out = run(gdn, c, new, 8)
    check_attention(out, *attention_ref(c, q, new, 128 ** -0.5), dtype)


def test_many_short_rows(gdn):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 1500).tolist()
    c = Cache(lens, "bf16", 2, 64, 16, seed=5, poison=float("inf"))
    new = [1] * len(lens)
    q, out = run(gdn, c, new, 4)
    check_attention(out, *attention_ref(c, q, new, 0.125), "bf16")


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (8, 2, 256)])
def test_long_and_single_tile_rows_in_turn(gdn, hq, hkv, d):
    """Runs of several rows each, of one key tile and of many: the parts of the kernel that take turns on tiles meet again."""
    rng = np.random.default_rng(d)
    lens = [int(rng.integers(1, 100)) if r % 4 else int(rng.integers(1500, 3000)) for r in range(160)]
    new = [1 if r % 5 else min(70, lens[r]) for r in range(160)]
    c = Cache(lens, "bf16", hkv, d, 16, seed=d, poison=float("nan"))
    q, out = run(gdn, c, new, hq)
    check_attention(out, *attention_ref(c, q, new, d ** -0.5), "bf16")
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_and_large_scores(gdn, dtype):
    """Scores of some hundreds, whose maximum comes late: earlier sums are scaled down to nothing."""
    c = Cache([400, 900], dtype, 1, 128, 16, seed=9)
    q = torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(2)).to(TYPES[dtype])
    k = c.k
    for r, at in ((0, 399), (1, 600)):
        page, slot = c.table[r, at // 16], at % 16
        k[0, page, 0, slot] = 8 * q[r, 0]
    q, out = run(gdn, c, [1, 1], 4, q=q, scale=0.5)
    check_attention(out, *attention_ref(c, q, [1, 1], 0.5), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_later_tokens_of_a_chunk_do_not_reach_earlier_ones(gdn, dtype, bad):
    new, lens = [70, 4], [170, 100]
    c = Cache(lens, dtype, 2, 128, 16, seed=4)
    q, want = run(gdn, c, new, 8)
    for r, at in ((0, 150), (1, 98)):
        page, slot = c.table[r, at // 16], at % 16
        c.k[0, page, :, slot] = bad
        c.v[0, page, :, slot] = bad
    q, out = run(gdn, c, new, 8, q=q)
    early = list(range(0, 50)) + [70, 71]
    ref, mag = attention_ref(c, q, new, 128 ** -0.5)
    check_attention(out[early], ref[early], mag[early], dtype)
    assert not torch.isfinite(out[50:70].float()).all(-1).any() or bad == float("inf")


@pytest.mark.parametrize("hq,hkv,d", [(12, 4, 64), (16, 4, 128), (14, 2, 256), (2, 2, 128)])
def test_fp32_items_of_every_number_of_rows(gdn, hq, hkv, d):
    """Tokens about where the rows of a tile take more or fewer of its warps, in runs of unequal cost."""
    new = [1, 4, 5, 6, 8, 9, 10, 11, 16, 17, 21, 22, 33, 42, 43, 65]
    lens = [n + 37 * (i % 5) + (900 if i % 3 == 0 else 0) for i, n in enumerate(new)]
    c = Cache(lens, "f32", hkv, d, 16, seed=hq, poison=float("nan"))
    q, out = run(gdn, c, new, hq)
    check_attention(out, *attention_ref(c, q, new, d ** -0.5), "f32")
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_values_that_are_not_finite_stay_in_their_columns(gdn, dtype, n):
    """A long row cut into many parts: the columns of V that hold an infinity or a NaN, and no others, show it, for the
    tokens that see it."""
    c = Cache([9001], dtype, 1, 128, 16, seed=n)
    q, want = run(gdn, c, [n], 4)
    late = 9000  # the last token's own key
    for at, col, bad in ((5000, 3, float("inf")), (5001, 3, float("inf")), (8000, 77, float("nan")), (late, 100, float("inf"))):
        c.v[0, c.table[0, at // 16], 0, at % 16, col] = bad
    q, out = run(gdn, c, [n], 4, q=q)
    assert (out[:, :, 3] == float("inf")).all() and torch.isnan(out[:, :, 77]).all()
    assert (out[-1, :, 100] == float("inf")).all() and torch.isfinite(out[:-1, :, 100]).all()
    rest = [x for x in range(128) if x not in (3, 77, 100)]
    ref, mag = attention_ref(c, q, [n], 128 ** -0.5)
    check_attention(out[:, :, rest], ref[:, :, rest], mag[:, :, rest], dtype)


def test_layers_strides_and_given_buffers(gdn):
    c = Cache([77, 130], "bf16", 2, 128, 16, layers=3, seed=6)
    new, hq = [3, 60], 6
    T = sum(new)
    wide = torch.randn(T, (hq + 4) * 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    q = wide[:, :hq * 128].view(T, hq, 128)
    pool = c.pool(gdn)
    out = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((max(16, gdn.paged_attention_workspace_bytes(pool, hq, 2, T)),), 255, dtype=torch.uint8, device=DEV)
    got = gdn.paged_attention(wide.to(DEV)[:, :hq * 128].view(T, hq, 128), pool, i32(c.table), i32(c.lens), i32(packed(new)),
                              layer=2, out=out, workspace=ws)
    assert got is out
    check_attention(out, *attention_ref(c, q, new, 128 ** -0.5, layer=2), "bf16")


def test_same_bits_again_and_on_another_stream(gdn):
    c = Cache([3000, 10, 5000], "bf16", 2, 128, 16, seed=7)
    new = [1, 1, 2]
    q, out = run(gdn, c, new, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, again = run(gdn, c, new, 16, q=q)
    s.synchronize()
    assert torch.equal(out, again)


def test_graph_follows_the_lengths_on_the_device(gdn):
    c = Cache([700, 333], "bf16", 2, 128, 16, seed=8)
    pool, table, q = c.pool(gdn), i32(c.table), torch.randn(2, 8, 128, device=DEV).bfloat16()
    lens, cu = i32([5, 9]), i32([0, 1, 2])
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(16, gdn.paged_attention_workspace_bytes(pool, 8, 2, 2)), dtype=torch.uint8, device=DEV)
    call = lambda: gdn.paged_attention(q, pool, table, lens, cu, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for now in ([700, 333], [1, 0], [130, 300]):
        lens.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        c.lens = now
        check_attention(out, *attention_ref(c, q.cpu(), [1, 1], 128 ** -0.5), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_rows_and_pages_give_zeros_and_set_the_error_word(gdn, dtype):
    lens, new = [50, 300, 40, 90, 20], [1, 40, 3, 1, 1]
    c = Cache(lens, dtype, 2, 128, 16, seed=11)
    good = Cache(lens, dtype, 2, 128, 16, seed=11)
    q = torch.randn(sum(new), 4, 128, generator=torch.Generator().manual_seed(3)).to(TYPES[dtype])
    ref, mag = attention_ref(good, q, new, 128 ** -0.5)
    c.table[1, 17] = c.num_pages + 5     # keys 272 .. 287: tokens 12 .. 39 of the chunk would see them
    c.table[3, 0] = -1
    c.lens = [50, 300, 2, 90, 20]        # row 2: three new tokens, length two
    _, out = run(gdn, c, new, 4, q=q)
    assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
    zero = list(range(13, 41)) + [41, 42, 43, 44]
    fine = [t for t in range(sum(new)) if t not in zero]
    assert (out[zero] == 0).all()
    check_attention(out[fine], ref[fine], mag[fine], dtype)
    c.lens = [50, 300, 40, 90, 16 * c.max_pages + 1]
    c.table[:] = good.table
    _, out = run(gdn, c, new, 4, q=q)
    assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
    assert (out[45] == 0).all()
    check_attention(out[:45], ref[:45], mag[:45], dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_past_32_bit_offsets(gdn, dtype):
    """A pool of over 2^31 elements (2^32 for bf16), whose last pages are used."""
    page, hkv, d, n = 128, 4, 128, 300
    pages = (2 ** 31 if dtype == "f32" else 2 ** 32) // (page * hkv * d) + 8
    k = torch.zeros(1, pages, hkv, page, d, dtype=TYPES[dtype], device=DEV)
    v = torch.zeros_like(k)
    pool = gdn.KVPagePool(pages, page, hkv, d, dtype=TYPES[dtype], k=k, v=v)
    c = Cache([n], dtype, hkv, d, page, seed=12)
    rows = [int(p) for p in c.table[0, :3]]
    at = [pages - 1, 5, pages - 3]
    for a, b in zip(rows, at):
        k[0, b], v[0, b] = c.k[0, a].to(DEV), c.v[0, a].to(DEV)
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(3)).to(TYPES[dtype])
    out = gdn.paged_attention(q.to(DEV), pool, i32([at]), i32([n]), i32([0, 2]))
    check_attention(out, *attention_ref(c, q, [2], d ** -0.5), dtype)


def test_wrong_arguments_are_refused(gdn):
    c = Cache([20], "bf16", 2, 128, 16)
    pool, table, lens, cu = c.pool(gdn), i32(c.table), i32(c.lens), i32([0, 1])
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        gdn.paged_attention(q.float(), pool, table, lens, cu)
    with pytest.raises(ValueError):
        gdn.paged_attention(q.cpu(), pool, table, lens, cu)
    with pytest.raises(ValueError):
        gdn.paged_attention(q, pool, table, lens, i32([0]))
    with pytest.raises(ValueError):
        gdn.paged_attention(q.view(1, 8, 64), pool, table, lens, cu)
    with pytest.raises(TypeError):
        gdn.paged_attention(q, pool, table.long(), lens, cu)
    for bad in (dict(layer=1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(gdn.GDNError):
            gdn.paged_attention(q, pool, table, lens, cu, **bad)
    with pytest.raises(gdn.GDNError):
        gdn.paged_attention(torch.zeros(1, 3, 128, dtype=torch.bfloat16, device=DEV), pool, table, lens, cu)
    with pytest.raises(ValueError):
        gdn.paged_attention(q, pool, table, lens, cu, out=torch.empty(3, device=DEV, dtype=torch.bfloat16))
    assert gdn.paged_attention(q[:0], pool, table, lens, i32([0, 0])).shape == (0, 4, 128)
