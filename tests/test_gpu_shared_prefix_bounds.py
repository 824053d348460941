"""paged_attention_shared where the division into groups leaves rows out."""
import pytest

from attn_helpers import DEV, i32, packed
from test_gpu_shared_prefix import Forked, run

pytestmark = pytest.mark.gpu


def test_bounds_that_leave_rows_out_are_reported(gdn):
    """The rows of the groups that there are have their results, and a row of no group its own."""
    c = Forked([(3, [(5, 1), (9, 1)]), (2, [(7, 1), (4, 1)])], "bf16", 1, 64, 16, seed=1)
    q, want = run(gdn, c, 2)
    args = (q.to(DEV), c.pool(gdn), i32(c.table), i32(c.lens), i32(packed(c.new)))
    for bounds, prefix in (([0, 2], [[0, 3]] * 2 + [[2, 0], [3, 0]]), ([2, 4], [[0, 0], [1, 0]] + [[2, 2]] * 2), ([1, 4], [[0, 0]] * 4)):
        out = gdn.paged_attention_shared(*args, i32(bounds), i32(prefix))
        assert gdn.get_device_error() == gdn.GDN_DEVERR_BAD_PAGE, bounds
        assert (out.double() - want.double()).norm() <= 2.0 ** -7 * want.double().norm()  # two roundings to bf16 each
