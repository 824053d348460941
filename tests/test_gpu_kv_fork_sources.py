"""kv_pages_fork on the GPU where a source's length is ahead of the pages it holds, or its entries name no page: the fork is
refused as a whole, its rows stay as they were, and the other forks of the call go on."""
import numpy as np
import pytest

from attn_helpers import i32
from test_gpu_kv_pages import BAD, Device, Model

pytestmark = pytest.mark.gpu


class Checked(Model):
    def fork(self, src, dst):
        """The forks whose sources are in order, with the status of the others between."""
        good = [all(0 < p < len(self.refs) for p in self.table[s, : -(-int(self.len[s]) // self.page)]) for s in src]
        status, moves = super().fork([s for s, ok in zip(src, good) if ok], [d for d, ok in zip(dst, good) if ok])
        rest = iter(status)
        return [next(rest) if ok else BAD for ok in good], moves


@pytest.mark.parametrize("max_pages", [9, 1500])  # rows filled in the planning launch, and in one of their own
@pytest.mark.parametrize("tail", [0, 5])
@pytest.mark.parametrize("entry", [0, -1, "pages"])
def test_sources_with_holes(gdn, max_pages, tail, entry):
    page, rows = 16, 24
    m = Checked(rows, max_pages, 40 * 9 + 8, page)
    held = [3, 4, 5, 7, 8, 2, 1, 0]
    lens = [max(0, (h - 1) * page + tail if tail else h * page) for h in held]
    m.reserve(range(8), lens)
    for r, n in enumerate(lens):
        m.len[r] = n
    bad = len(m.refs) if entry == "pages" else entry
    for r, at in ((1, 0), (2, 2), (3, 6), (4, 1)):  # first, middle and last pages
        m.refs[m.table[r, at]] = 0
        m.table[r, at] = bad
    m.len[5] += page  # a length ahead of its pages
    d = Device(m)
    src, dst = [0, 1, 2, 0, 3, 4, 5, 6, 7, 0], list(range(9, 19))
    status, moves = m.fork(src, dst)
    assert status == [0, BAD, BAD, 0, BAD, BAD, BAD, 0, 0, 0]
    mv = gdn.KVPageMoves(len(src))
    mv.src.fill_(9), mv.dst.fill_(9)
    gdn.kv_pages_fork(d.table, d.len, d.refs, i32(src), i32(dst), page, mv)
    assert mv.status.tolist() == status
    n = int(mv.count)
    assert list(zip(mv.src.tolist(), mv.dst.tolist()))[:n] == moves and not mv.src[n:].any() and not mv.dst[n:].any()
    d.same(m)
    assert gdn.get_device_error() == BAD


@pytest.mark.parametrize("n,max_pages", [(1, 400), (33, 70), (700, 40), (4000, 3)])
def test_only_the_rows_with_a_hole_are_refused(gdn, n, max_pages):
    """Any number of forks, of rows of any length, a hole anywhere."""
    rng = np.random.default_rng(n)
    page, sources = 16, max(1, n // 3)
    m = Checked(sources + n, max_pages, 1 + sources * max_pages + n, page)
    lens = [int(rng.integers(0, max_pages * page + 1)) for _ in range(sources)]
    assert not any(m.reserve(range(sources), lens))
    m.len[:sources] = lens
    for r in range(sources):
        if lens[r] and rng.random() < 0.3:
            at = int(rng.integers(0, -(-lens[r] // page)))
            m.refs[m.table[r, at]] = 0
            m.table[r, at] = 0
    d = Device(m)
    src, dst = rng.integers(0, sources, n), sources + rng.permutation(n)
    status, moves = m.fork(src.tolist(), dst.tolist())
    mv = gdn.KVPageMoves(n)
    gdn.kv_pages_fork(d.table, d.len, d.refs, i32(src), i32(dst), page, mv)
    assert mv.status.tolist() == status
    assert list(zip(mv.src.tolist(), mv.dst.tolist()))[: int(mv.count)] == moves
    d.same(m)
    assert gdn.get_device_error() == (BAD if BAD in status else 0)
