"""kv_pages_shared and paged_attention_shared: groups of rows that share their first pages, against the definitions (the
attention in 64 bits, with the tolerances of paged_attention: its parts are the same sums, joined in fp32)."""
import numpy as np
import pytest
import torch

from attn_helpers import DEV, TYPES, Cache, attention_ref, check_attention, i32, packed

pytestmark = pytest.mark.gpu


def shared_by_definition(table, lens, new, bounds, page):
    out = np.zeros((len(lens), 2), np.int32)
    for a, b in zip(bounds, bounds[1:]):
        live = [r for r in range(a, b) if new[r] > 0 and lens[r] >= new[r]]
        n = 0
        if len(live) > 1:
            most = min(min((lens[r] - new[r]) // page for r in live), table.shape[1])
            while n < most and len({int(table[r, n]) for r in live}) == 1:
                n += 1
        out[a:b] = (live[0] if live else a, n)
    return out


class Forked(Cache):
    """groups: (pages shared, [(tokens of its own, new tokens)] by row); a row of no tokens of its own is a padding row, which
    brings its new tokens all the same."""

    def __init__(self, groups, dtype, hkv, d, page, **k):
        self.bounds, lens, self.new = [0], [], []
        for pages, rows in groups:
            lens += [pages * page + own if own else 0 for own, _ in rows]
            self.new += [n for _, n in rows]
            self.bounds.append(len(lens))
        super().__init__(lens, dtype, hkv, d, page, **k)
        for (pages, _), a, b in zip(groups, self.bounds, self.bounds[1:]):
            live = [r for r in range(a, b) if lens[r]]
            for r in live[1:]:
                self.table[r, :pages] = self.table[live[0], :pages]

    def prefix(self):
        return shared_by_definition(self.table, self.lens, self.new, self.bounds, self.page)


def run(G, c, hq, seed=1, scale=None, layer=0, prefix=None, q=None, **k):
    T = int(sum(c.new))
    if q is None:
        q = torch.randn(T, hq, c.d, generator=torch.Generator().manual_seed(seed)).to(TYPES[c.dtype])
    table, lens, cu, bounds = i32(c.table), i32(c.lens), i32(packed(c.new)), i32(c.bounds)
    found = G.kv_pages_shared(table, lens, cu, bounds, c.page)
    assert (found.cpu().numpy() == c.prefix()).all()
    out = G.paged_attention_shared(q.to(DEV), c.pool(G), table, lens, cu, bounds, found if prefix is None else i32(prefix), layer=layer,
                                   scale=scale, **k)
    return q, out


HEADS = [(136, 1, 64), (12, 4, 64), (16, 4, 128), (7, 1, 128), (16, 2, 256), (6, 2, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("page", [16, 128])
def test_decode_of_forked_rows(gdn, dtype, hq, hkv, d, page):
    """Groups of one to nine rows; prefixes of none, one and many pages; padding rows first, within and last; pages that end
    inside a tile; NaN wherever no row has a token."""
    groups = [(0, [(5, 1)]), (3, [(1, 1), (17, 1), (0, 1), (130, 1)]), (40 * 16 // page, [(0, 1)] + [(10 + 31 * i, 1) for i in range(8)]),
              (0, [(200, 1), (3, 1)]), (1, [(2, 1), (2, 1), (0, 1)]), (2, [(0, 1), (0, 1)]), (9, [(40, 1), (0, 1)])]
    c = Forked(groups, dtype, hkv, d, page, seed=d + hq, poison=float("nan"))
    q, out = run(gdn, c, hq)
    check_attention(out, *attention_ref(c, q, c.new, d ** -0.5), dtype)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (8, 2, 256)])
def test_verification_and_chunks(gdn, dtype, hq, hkv, d):
    """Rows of none, one and many new tokens over shared pages; a group whose tokens fill several tiles."""
    groups = [(6, [(9, 4), (70, 70), (30, 1), (12, 0)]), (1, [(150, 130), (180, 150), (0, 3)]), (12, [(4, 4)] * 21)]
    c = Forked(groups, dtype, hkv, d, 32, seed=d, poison=float("nan"))
    q, out = run(gdn, c, hq)
    check_attention(out, *attention_ref(c, q, c.new, d ** -0.5), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(32, 2, 64), (16, 2, 128), (16, 1, 256)])
def test_many_tokens_over_a_long_prefix(gdn, dtype, hq, hkv, d):
    """More tokens and heads than there are places for warps, and items of several parts, own and shared."""
    c = Forked([(60, [(9, 4), (320, 300), (0, 2), (12, 12)]), (0, [(40, 3)])], dtype, hkv, d, 32, seed=d, poison=float("nan"))
    q, out = run(gdn, c, hq)
    assert len(q) * hq > 32 * 152
    check_attention(out, *attention_ref(c, q, c.new, d ** -0.5), dtype)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_prefix_is_divided(gdn, dtype):
    """A shared prefix that every CTA has a part of, and the same with a layer, a scale and given buffers."""
    c = Forked([(1500, [(1, 1), (33, 1), (0, 1), (700, 1)]), (2, [(3, 1)])], dtype, 2, 128, 16, seed=3, layers=2, poison=float("nan"))
    pool_out = torch.full((5, 8, 128), 9.0, dtype=TYPES[dtype], device=DEV)
    ws = torch.full((gdn.paged_attention_shared_workspace_bytes(c.pool(gdn), 8, 5, 5),), 255, dtype=torch.uint8, device=DEV)
    q, out = run(gdn, c, 8, layer=1, scale=0.05, out=pool_out, workspace=ws)
    assert out is pool_out
    check_attention(out, *attention_ref(c, q, c.new, 0.05, layer=1), dtype)


def test_shared_by_less_than_the_tables_have_alike(gdn):
    """A caller's own prefix of fewer pages, and none at all, give the same outputs within rounding."""
    c = Forked([(8, [(20, 1), (3, 2), (50, 1)])], "f32", 2, 64, 16, seed=4)
    for pages in (0, 1, 7):
        q, out = run(gdn, c, 4, prefix=[[0, pages]] * 3)
        check_attention(out, *attention_ref(c, q, c.new, 0.125), "f32")


def test_results_repeat_bit_for_bit(gdn):
    c = Forked([(200, [(1 + 7 * i, 1) for i in range(40)])], "bf16", 2, 128, 16, seed=5)
    q, a = run(gdn, c, 8)
    for _ in range(5):
        assert torch.equal(a, run(gdn, c, 8, q=q)[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite_where_rows_see_them(gdn, dtype):
    """An infinite value in the shared keys reaches every row that weighs it, one in a row's own keys that row alone."""
    c = Forked([(2, [(20, 1), (20, 1), (20, 1)])], dtype, 1, 64, 16, seed=6)
    clean = run(gdn, c, 2)[1]
    c.v[0, c.table[0, 2], 0, 3, 7] = float("inf")          # own: row 0's third page
    out = run(gdn, c, 2)[1]
    assert torch.isinf(out[0, :, 7]).all() and torch.equal(out[1:], clean[1:])
    c.v[0, c.table[0, 2], 0, 3, 7] = 0.0
    c.v[0, c.table[0, 1], 0, 3, 7] = float("nan")          # shared
    out = run(gdn, c, 2)[1]
    assert torch.isnan(out[:, :, 7]).all()
    keep = torch.arange(64, device=DEV) != 7
    assert torch.equal(out[1:][:, :, keep], clean[1:][:, :, keep])


def test_bad_tables(gdn):
    def group():
        return Forked([(4, [(20, 1), (20, 1)]), (2, [(9, 1), (30, 1)])], "bf16", 1, 64, 16, seed=7)

    good = group()
    q, want = run(gdn, good, 2)
    prefix = good.prefix()
    c = group()  # a page outside the pool among the shared ones: the group's rows are zero, the others as they were
    c.table[:2, 1] = c.num_pages
    out = run(gdn, c, 2, q=q)[1]
    assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
    assert (out[:2] == 0).all() and torch.equal(out[2:], want[2:])
    c = group()  # more shared pages than the rows have before their new tokens
    p = prefix.copy()
    p[2:, 1] = 3
    out = run(gdn, c, 2, prefix=p, q=q)[1]
    assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
    assert torch.equal(out[:2], want[:2]) and (out[2] == 0).all()
    for wrong in (np.array([[9, 4]] * 2 + [[2, 2]] * 2), np.array([[0, -1]] * 2 + [[2, 2]] * 2), np.array([[0, 1 << 20]] * 2 + [[2, 2]] * 2)):
        out = run(gdn, group(), 2, prefix=wrong, q=q)[1]
        assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
        assert torch.equal(out[2:], want[2:])


@pytest.mark.parametrize("seed", range(6))
def test_shared_pages_of_random_tables(gdn, seed):
    """Groups of no rows, of one and of hundreds; entries that differ at random places; rows without new tokens."""
    rng = np.random.default_rng(seed)
    page, width = int(rng.choice([16, 64])), int(rng.integers(1, 700))
    sizes = [0, 1, 2, int(rng.integers(3, 40)), 0, int(rng.integers(100, 600)), 5]
    bounds = np.concatenate([[0], np.cumsum(sizes)])
    rows = int(bounds[-1])
    table = np.tile(rng.integers(1, 1000, width), (rows, 1)).astype(np.int32)
    new = rng.integers(0 if seed % 2 else 1, 4, rows)
    lens = np.where(rng.random(rows) < 0.2, 0, rng.integers(1, width * page + 1, rows)) if seed % 3 else np.full(rows, width * page)
    for r in rng.integers(0, rows, 4):
        table[r, rng.integers(0, width)] += 1
    out = torch.full((rows, 2), -7, dtype=torch.int32, device=DEV)
    got = gdn.kv_pages_shared(i32(table), i32(lens), i32(packed(new)), i32(bounds), page, out=out)
    assert got is out
    assert (out.cpu().numpy() == shared_by_definition(table, lens, new, bounds, page)).all()
    assert gdn.get_device_error() == 0


def test_wrong_bounds(gdn):
    table, lens, cu = i32(np.ones((6, 3))), i32([40] * 6), i32(range(7))
    for bounds, want in (([1, 3, 6], {0: (0, 0), 1: (1, 2)}), ([0, 2, 4], {0: (0, 2), 5: (5, 0)}), ([0, 3, 9], {0: (0, 2)}), ([0, 4, 2], {0: (0, 2)})):
        got = gdn.kv_pages_shared(table, lens, cu, i32(bounds), 16).tolist()
        assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE
        for r, x in want.items():
            assert tuple(got[r]) == x


def test_captured_and_on_another_stream(gdn):
    """A step captured once serves rows that grow, and rows that are released."""
    c = Forked([(4, [(20, 1), (5, 1), (9, 1)]), (3, [(2, 1), (40, 1)])], "bf16", 2, 64, 16, seed=8)
    pool, table, cu, bounds = c.pool(gdn), i32(c.table), i32(packed(c.new)), i32(c.bounds)
    lens = i32(c.lens)
    q = torch.randn(5, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    qd = q.to(DEV)

    def step():
        return gdn.paged_attention_shared(qd, pool, table, lens, cu, bounds, gdn.kv_pages_shared(table, lens, cu, bounds, 16))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for released in ([], [0], [0, 2]):
        for r in released:
            c.lens[r] = 0
            c.table[r] = 0
        lens.copy_(i32(c.lens))
        table.copy_(i32(c.table))
        graph.replay()
        check_attention(out, *attention_ref(c, q, c.new, 0.125), "bf16")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, out)


def test_rows_forked_by_the_pool(gdn):
    """fork, copy, reserve, append, attend: the calls of a decoder whose rows are sampled several times."""
    page, d = 16, 64
    g = torch.Generator().manual_seed(9)
    table, lens, refs = i32(np.zeros((5, 8))), i32([0] * 5), i32([0] * 40)
    pool = gdn.KVPagePool(40, page, 2, d)
    gdn.kv_pages_reserve(table, refs, i32([0]), i32([70]), page)
    lens[0] = 70
    x = torch.randn(70, 4, d, generator=g).bfloat16().to(DEV)
    gdn.attn_prologue(x, x[:, :2], x[:, 2:], pool, None, table, lens, i32([0, 70, 70, 70, 70, 70]))
    moves = gdn.KVPageMoves(4)
    gdn.kv_pages_fork(table, lens, refs, i32([0] * 4), i32([1, 2, 3, 4]), page, moves)
    gdn.kv_pages_copy(pool, moves)
    gdn.kv_pages_reserve(table, refs, i32(range(5)), lens + 1, page)
    lens += 1
    x = torch.randn(5, 8, d, generator=g).bfloat16().to(DEV)
    cu, bounds = i32(range(6)), i32([0, 5])
    q = gdn.attn_prologue(x[:, :4], x[:, 4:6], x[:, 6:], pool, None, table, lens, cu)
    prefix = gdn.kv_pages_shared(table, lens, cu, bounds, page)
    assert prefix.tolist() == [[0, 4]] * 5
    a = gdn.paged_attention_shared(q, pool, table, lens, cu, bounds, prefix).double()
    b = gdn.paged_attention(q, pool, table, lens, cu).double()
    assert (a - b).norm() <= 2.0 ** -7 * b.norm()  # two roundings to bf16 each


def test_python_refusals(gdn):
    c = Forked([(2, [(3, 1), (4, 1)])], "bf16", 1, 64, 16)
    pool, table, lens, cu, bounds = c.pool(gdn), i32(c.table), i32(c.lens), i32([0, 1, 2]), i32([0, 2])
    prefix, q = i32(c.prefix()), torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    good = dict(q=q, pool=pool, table=table, seq_len=lens, cu_seqlens=cu, bounds=bounds, prefix=prefix)
    gdn.paged_attention_shared(**good)
    for wrong in (dict(prefix=prefix[:1]), dict(cu_seqlens=cu[:2]), dict(bounds=bounds.cpu()), dict(q=q[:, :, :32]),
                  dict(bounds=i32([0, 1, 2, 2])), dict(scale=-1.0), dict(layer=1), dict(workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises((ValueError, gdn.GDNError)):
            gdn.paged_attention_shared(**{**good, **wrong})
    with pytest.raises(TypeError):
        gdn.paged_attention_shared(**{**good, "prefix": prefix.long()})
    with pytest.raises(gdn.GDNError):
        gdn.kv_pages_shared(table, lens, cu, bounds, 24)
    with pytest.raises(gdn.GDNError):
        gdn.kv_pages_shared(table, lens, cu, i32([0]), 16)
    with pytest.raises(ValueError):
        gdn.kv_pages_shared(table, lens[:1], cu, bounds, 16)


def test_both_bindings_make_the_same_calls(gdn, monkeypatch):
    from gated_deltanet_decode_gb300 import _lib
    if _lib.fast() is None:
        pytest.skip("the C++ binding was not built")
    c = Forked([(6, [(20, 1), (5, 1), (0, 1)])], "bf16", 2, 128, 16, seed=10)
    q, a = run(gdn, c, 8)
    monkeypatch.setattr(_lib, "_fast", None)
    assert torch.equal(a, run(gdn, c, 8, q=q)[1])
