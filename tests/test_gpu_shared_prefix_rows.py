"""paged_attention_shared with more rows and groups than a CTA has threads, which then look at the lengths twice, and
kv_pages_shared over rows that hold tokens and bring none."""
import numpy as np
import pytest

from attn_helpers import attention_ref, check_attention, i32, packed
from test_gpu_shared_prefix import Forked, run, shared_by_definition

pytestmark = pytest.mark.gpu


def groups_of(kind):
    """Every seventh row of the busy batches is padding; of the idle one's 14 rows a group three are live.

    With a key head, a tile and an item a row and group, at 1 unit a tile and 3 an item in bf16 and 4 and 10 in fp32, the busy
    batches are more than the least work a CTA (4 units x 152, 14 x 304) that counts items' begins and ends, the idle one is less."""
    rng = np.random.default_rng(len(kind))
    if kind == "idle":
        return [(int(rng.integers(1, 4)), [(int(rng.integers(1, 20)), 1) if i in (2, 7, 13) else (0, 1) for i in range(14)]) for _ in range(30)]
    return [(int(rng.integers(0, 4)), [(0, 1) if (8 * g + i) % 7 == 5 else (int(rng.integers(1, 40)), 1) for i in range(8)])
            for g in range(60 if kind == "busy" else 110)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["busy", "more", "idle"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (4, 2, 128), (2, 1, 256)])
def test_more_rows_than_threads(gdn, dtype, kind, hq, hkv, d):
    c = Forked(groups_of(kind), dtype, hkv, d, 16, seed=d, poison=float("nan"))
    assert len(c.lens) + len(c.bounds) - 1 > 384
    q, out = run(gdn, c, hq)
    check_attention(out, *attention_ref(c, q, c.new, d ** -0.5), dtype)
    assert gdn.get_device_error() == 0


def test_a_row_without_new_tokens_shares_nothing(gdn):
    """Such a row is not live: it neither leads its group nor ends what the others share."""
    page = 16
    table = np.tile(np.arange(1, 7), (8, 1)).astype(np.int32)
    table[0, 1] = table[3, 2] = table[6, 0] = 9
    lens, new, bounds = [90, 80, 85, 96, 96, 96, 96, 96], [0, 1, 2, 0, 1, 0, 0, 1], [0, 4, 6, 8]
    got = gdn.kv_pages_shared(i32(table), i32(lens), i32(packed(new)), i32(bounds), page)
    assert got.tolist() == [[1, 4]] * 4 + [[4, 0]] * 2 + [[7, 0]] * 2
    assert (got.cpu().numpy() == shared_by_definition(table, lens, new, bounds, page)).all()
    assert gdn.get_device_error() == 0
