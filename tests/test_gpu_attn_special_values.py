"""paged_attention on the GPU where keys or values are infinite, NaN or at the top of their type's range: against the
definition in 64 bits, in which such a value reaches the tokens that see it and no others."""
import numpy as np
import pytest
import torch

from attn_helpers import DEV, TYPES, Cache, attention_ref, i32, packed

pytestmark = pytest.mark.gpu


def run(G, c, new, hq, seed=1, scale=None, q=None):
    if q is None:
        q = torch.randn(sum(new), hq, c.d, generator=torch.Generator().manual_seed(seed)).to(TYPES[c.dtype])
    return q, G.paged_attention(q.to(DEV), c.pool(G), i32(c.table), i32(c.lens), i32(packed(new)), scale=scale)


def place(c, row, key):
    """Index of a row's key in the pools, without the head and the column."""
    return c.table[row, key // c.page], key % c.page


def check(out, ref, mag, dtype):
    """The tolerances of the parity tests where the definition is finite, and its very values where it is not."""
    o = out.double().cpu()
    fine = torch.isfinite(ref)
    tol = 2.0 ** -8 * (ref.abs() + mag) if dtype == "bf16" else 4e-5 * mag
    assert (torch.isnan(o) == torch.isnan(ref)).all()
    assert (o[torch.isinf(ref)] == ref[torch.isinf(ref)]).all()
    worst = ((o - ref).abs() - tol)[fine].max().item()
    assert worst <= 0, f"out of tolerance by {worst:.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (4, 2, 256)])
def test_items_in_a_row_with_values_that_are_not_finite(gdn, dtype, hq, hkv, d):
    """Prompts of one or two tiles of tokens, several to a run, whose keys are hidden from some of their own tokens: each
    item keeps its own infinities and NaN, whatever the next one finds."""
    rng = np.random.default_rng(d)
    rows = 260
    new = [int(rng.integers(50, 64)) for _ in range(rows)]
    lens = [n + int(rng.integers(0, 40)) for n in new]
    c = Cache(lens, dtype, hkv, d, 16, seed=d, poison=float("nan"))
    for r in range(rows):
        for x in range(int(rng.integers(1, 3))):
            key = int(rng.integers(lens[r] - new[r], lens[r]))
            page, slot = place(c, r, key)
            c.v[0, page, int(rng.integers(0, hkv)), slot, int(rng.integers(0, d))] = (float("inf"), float("nan"), -float("inf"))[r % 3]
    q, out = run(gdn, c, new, hq)
    check(out, *attention_ref(c, q, new, d ** -0.5), dtype)
    assert gdn.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,n", [(4, 2, 64, 70), (8, 1, 128, 5), (4, 1, 128, 100), (2, 1, 256, 40)])
def test_largest_finite_values_stay_with_the_tokens_that_see_them(gdn, dtype, hq, hkv, d, n):
    """V holds the type's largest and lowest value where only the chunk's last tokens see it.  Those tokens are compared in
    fp32; in bf16 a sum before its division may pass the range."""
    c = Cache([130 + n], dtype, hkv, d, 16, seed=d + n)
    top = torch.finfo(TYPES[dtype]).max
    see = [n - 1, n - 3]  # the first tokens that see them
    for x, t in enumerate(see):
        page, slot = place(c, 0, 130 + t)
        c.v[0, page, :, slot, 7 + x] = top if x else -top
    q, out = run(gdn, c, [n], hq)
    ref, mag = attention_ref(c, q, [n], d ** -0.5)
    upto = n if dtype == "f32" else n - 3
    check(out[:upto], ref[:upto], mag[:upto], dtype)
    assert torch.isfinite(ref).all() and gdn.get_device_error() == 0


def test_fp32_keys_at_the_top_of_the_range(gdn):
    """A key's largest value against a query's 2^-120: a score like any other."""
    c = Cache([300], "f32", 1, 64, 16, seed=3)
    top = torch.finfo(torch.float32).max
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(2))
    q[:, :, 9] = 2.0 ** -120
    for key, x in ((17, top), (230, -top), (298, top)):
        page, slot = place(c, 0, key)
        c.k[0, page, 0, slot, 9] = x
    q, out = run(gdn, c, [4], 4, q=q)
    check(out, *attention_ref(c, q, [4], 0.125), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,n", [(4, 2, 64, 70), (8, 1, 128, 5), (4, 1, 128, 100), (2, 1, 256, 40)])
def test_infinite_keys_drop_out_or_leave_nothing(gdn, dtype, hq, hkv, d, n):
    """One infinite element of K gives a score of minus infinity, a weight of zero, or of plus infinity, no result, by the
    query's sign; tokens that do not see the key are as they are without it."""
    c = Cache([130 + n], dtype, hkv, d, 16, seed=d + n + 1)
    for t, x in ((n - 2, float("inf")), (n // 2, -float("inf"))):
        page, slot = place(c, 0, 130 + t)
        c.k[0, page, hkv - 1, slot, 11] = x
    q, out = run(gdn, c, [n], hq)
    ref, mag = attention_ref(c, q, [n], d ** -0.5)
    assert torch.isnan(ref).any() and torch.isfinite(ref[n // 2:]).all(-1).any()
    check(out, ref, mag, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 50])
def test_an_infinite_query_leaves_the_other_heads_and_tokens_alone(gdn, dtype, n):
    c = Cache([3000], dtype, 2, 128, 16, seed=n)
    q = torch.randn(n, 8, 128, generator=torch.Generator().manual_seed(7)).to(TYPES[dtype])
    q[n // 2, 5, 3] = float("inf")
    q, out = run(gdn, c, [n], 8, q=q)
    ref, mag = attention_ref(c, q, [n], 128 ** -0.5)
    assert torch.isnan(ref[n // 2, 5]).all() and torch.isnan(ref).sum() == 128
    check(out, ref, mag, dtype)
