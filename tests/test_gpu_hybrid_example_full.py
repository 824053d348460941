"""The example's hybrid decoder when the page pool runs out: the row that gets no pages rests, keeps what it had, and goes on
later as if nothing had been asked."""
import pytest
import torch

from test_gpu_hybrid_example import ex, tokens  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("second", [1, 4])  # a decode step, a chunk
def test_a_row_without_pages_rests(gdn, ex, second):  # noqa: F811
    a, b = ex.Decoder(2, 64, 5), ex.Decoder(2, 64, 40)  # four pages, and enough
    x = tokens(ex, 48 + 16, 5)
    for m in (a, b):
        m.step(x, [48, 16])
    y = tokens(ex, second, 6)
    held = lambda: [a.table, a.length] + [p.tensor for layer in a.gdn.values() for p in layer]  # noqa: E731
    before = [t.clone() for t in held()]
    a.step(torch.cat([y, y]), [second, second])  # neither has room
    assert a.status.tolist() == [gdn.GDN_DEVERR_NO_PAGES] * 2 and gdn.get_device_error() == gdn.GDN_DEVERR_NO_PAGES
    assert all(torch.equal(x, y) for x, y in zip(held(), before))
    for m in (a, b):
        m.release([0])
    for t in range(3):
        z = tokens(ex, second, 20 + t)
        assert torch.equal(a.step(z, [0, second]), b.step(z, [0, second]))
    assert torch.equal(a.length, b.length) and gdn.get_device_error() == 0


def test_a_fork_without_pages_leaves_its_row_empty(gdn, ex):  # noqa: F811
    a, b = ex.Decoder(3, 64, 4), ex.Decoder(3, 64, 4)  # three pages
    x = tokens(ex, 40, 7)
    for m in (a, b):
        m.step(x, [40, 0, 0])
    assert a.fork([0, 0], [1, 2]).tolist() == [gdn.GDN_DEVERR_NO_PAGES] * 2
    assert gdn.get_device_error() == gdn.GDN_DEVERR_NO_PAGES
    for m in (a, b):
        m.release([0])
    y = tokens(ex, 5, 8)
    assert torch.equal(a.step(y, [0, 4, 1]), b.step(y, [0, 4, 1]))
    assert gdn.get_device_error() == 0
