"""paged_attention in fp32 keeps to fp32's precision in norm, not only in its largest error.

The bound.  Scores have a standard deviation of about 2 here.  One is off by the tails' own rounding and the products of
tails that are left out (2^-23 of a term, terms of random signs: 2^-23 of the score's size), by the fp32 additions of its
partial sums (a few times 2^-24 of it) and by the rounding of its distance from the maximum (2^-24 of up to 8), and the
exponential by 2^-22: 4e-7 to 6e-7 of a weight in all.  The weights' errors are independent, so they take the same share of a
result's norm; the products with V add 1e-7.  The bound is 2^-19, 1.9e-6, three times that.  On a mixed batch, operands whose heads
are cut short instead of rounded, or sums left to the tensor cores' truncation, gave 5e-6 and more."""
import pytest
import torch

from attn_helpers import DEV, Cache, attention_ref, i32, packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(12, 4, 64), (16, 4, 128), (8, 1, 128), (16, 2, 256)])
@pytest.mark.parametrize("new,lens", [([1] * 6, [900, 40, 1500, 300, 2000, 7]), ([4, 3, 2], [1000, 350, 3]), ([150, 60], [700, 1200]),
                                      ([1, 1], [9000, 20000])])
def test_error_in_norm(gdn, hq, hkv, d, new, lens):
    c = Cache(lens, "f32", hkv, d, 16, seed=d + sum(new))
    q = 2 * torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(3))
    out = gdn.paged_attention(q.to(DEV), c.pool(gdn), i32(c.table), i32(c.lens), i32(packed(new))).double().cpu()
    ref, _ = attention_ref(c, q, new, d ** -0.5)
    err = ((out - ref).norm() / ref.norm()).item()
    assert err <= 2.0 ** -19, f"{err:.3g} of the result's norm"
